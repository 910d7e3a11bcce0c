"""Calls on a stream other than the current one, through the `stream` argument:
what a call allocates for itself belongs to the stream that it runs on."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda):
    lib.qg_device_status(True)
    yield
    assert lib.qg_device_status(True) == 0


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Experts:
    """Indirect rows, many per expert: the sorted rows lie in a workspace."""
    T, topk, E, N, K = 600, 2, 4, 136, 320

    def __init__(self, lib, seed):
        rng = np.random.default_rng(seed)
        self.lib = lib
        qw, sw, zw = C.weights(rng, self.N, self.K, "f32", self.E)
        ids = C.routing(rng, self.T, self.topk, self.E)
        offsets, src, _ = oracle.sort_by_expert(ids, self.E)
        self.packed = C.pack_experts(lib, torch, qw, sw, zw, "f32")
        self.offsets, self.src = _i32(offsets), _i32(src)
        self.x = torch.from_numpy(C.bf16_round(rng.standard_normal((self.T, self.K)))).cuda().to(BF)
        self.y = torch.zeros((self.T * self.topk, self.N), dtype=BF, device="cuda")

    def __call__(self, stream=None):
        self.lib.qgemm_a16w4_bf16_experts(self.x, self.offsets, self.packed, self.y, src=self.src,
                                          topk=self.topk, stream=stream)

    def result(self):
        return [self.y.view(torch.int16)]


class Order:
    """More entries than one CTA sorts: the chunks' counts lie in a workspace."""
    T, topk, E = 3000, 4, 300

    def __init__(self, lib, seed):
        self.lib = lib
        self.ids = _i32(np.random.default_rng(seed).integers(0, self.E, (self.T, self.topk)))
        self.offsets, self.src, self.pos = _i32(np.zeros(self.E + 1)), _i32(np.zeros(self.T * self.topk)), \
            _i32(np.zeros((self.T, self.topk)))

    def __call__(self, stream=None):
        self.lib.qg_sort_by_expert(self.ids, self.offsets, self.src, self.pos, stream=stream)

    def result(self):
        return [self.offsets, self.src, self.pos]


class A8W4:
    """Quantized activations between two kernels lie in a workspace."""
    M, N, K = 96, 200, 512

    def __init__(self, lib, seed):
        rng = np.random.default_rng(seed)
        self.lib = lib
        qw, sw, _ = C.weights(rng, self.N, self.K, "f32")
        self.packed = C.pack(lib, torch, qw, sw, None, "f32")
        self.x = torch.from_numpy(rng.standard_normal((self.M, self.K)).astype(np.float32)).cuda()
        self.bias = torch.zeros(self.N, device="cuda")
        self.y = torch.zeros((self.M, self.N), device="cuda")

    def __call__(self, stream=None):
        self.lib.qgemm_a8w4_f32(self.x, self.packed, self.N, self.bias, -1e30, 1e30, self.y,
                                stream=stream)

    def result(self):
        return [self.y]


CALLS = [Experts, Order, A8W4]


@pytest.mark.parametrize("kind", CALLS)
@pytest.mark.parametrize("raw", [False, True])
def test_workspace_belongs_to_the_calls_stream(lib, monkeypatch, kind, raw):
    """The call may still wait on its stream when it returns: its workspace is
    not handed out to the current one."""
    call = kind(lib, 1)
    call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    seen, real = [], lib._empty_bytes

    def spy(n, device):
        t = real(n, device)
        seen.append((t.data_ptr(), t.numel()))
        return t
    monkeypatch.setattr(lib, "_empty_bytes", spy)
    side = torch.cuda.Stream()
    call(stream=side.cuda_stream if raw else side)
    assert len(seen) == 1, "the call was to need a workspace"
    at, n = seen[0]
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() >= at + n or t.data_ptr() + n <= at for t in others)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", CALLS)
def test_the_default_stream_by_its_handle(lib, kind):
    """Handle 0 is the default stream, not the current one."""
    call = kind(lib, 4)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in call.result()]
    for t in call.result():
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        call(stream=0)
        torch.cuda.default_stream().synchronize()
        assert all(torch.equal(a, b) for a, b in zip(call.result(), want))


def test_packed_weights_of_another_stream(lib, monkeypatch):
    """A matrix packed on another stream: its memory is not handed out before
    that stream, or the current one, is done with it."""
    rng = np.random.default_rng(3)
    qw, sw, _ = C.weights(rng, 264, 1024, "f32")
    q, s = torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda()
    want = lib.pack_w4_g32(q, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    packed = lib.pack_w4_g32(q, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    same = torch.equal(packed, want)  # waits
    at, n = packed.data_ptr(), packed.numel()
    copy = torch.empty_like(packed)
    torch.cuda._sleep(50_000_000)
    copy.copy_(packed)
    del packed
    with torch.cuda.stream(side):
        others = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
        for t in others:
            t.fill_(255)
    assert same and all(t.data_ptr() >= at + n or t.data_ptr() + n <= at for t in others)
    assert torch.equal(copy, want)


@pytest.mark.parametrize("kind", CALLS)
def test_two_calls_on_two_streams(lib, kind):
    """Calls on two explicit streams, neither the current one, many times
    over: the bits of the same calls one after the other."""
    calls = [kind(lib, k) for k in range(2)]
    want = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in call.result()])
        for t in call.result():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for call, stream in zip(calls, streams):
            call(stream=stream)
        junk = torch.full((1 << 21,), 0xFF, dtype=torch.uint8, device="cuda")
        del junk
    torch.cuda.synchronize()
    for call, ref in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(call.result(), ref))


@pytest.mark.parametrize("T,topk,N", [(16, 8, 256), (16, 2, 4096), (130, 4, 520), (700, 4, 64)])
@pytest.mark.parametrize("grad", [False, True])
def test_steps_behind_one_another_share_their_buffers(lib, T, topk, N, grad):
    """Steps of order, spread and sum back to back in one graph, with other ids
    each and the same places and rows: a kernel is resident while the one
    before it still reads the last step's places and writes this step's, and
    must not see the old ones.  Every step's own results are kept."""
    g = torch.Generator(device="cuda").manual_seed(T + N)
    steps, E, S = 24, 64, T * topk
    ids = torch.randint(0, E, (steps, T, topk), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((steps, T, N), generator=g, device="cuda").to(BF)
    w = torch.rand((steps, T, topk), generator=g, device="cuda")
    offsets, src, pos = (torch.empty(n, device="cuda", dtype=torch.int32) for n in (E + 1, S, S))
    pos = pos.view(T, topk)
    xs, dys = torch.empty((S, N), device="cuda", dtype=BF), torch.empty((S, N), device="cuda", dtype=BF)
    wk, dw = torch.empty((T, topk), device="cuda"), torch.empty((steps, T, topk), device="cuda")
    y = torch.empty_like(x)

    def run():
        for k in range(steps):
            lib.qg_sort_by_expert(ids[k], offsets, src, pos)
            lib.qg_spread_rows(x[k], pos, xs)
            if grad:  # of the sum, and the spread's own: two kernels read the places
                lib.qg_combine_rows_grad(x[k], xs, pos, w[k], dys, dw[k])
                lib.qg_combine_rows(dys, pos, y[k])
            else:
                lib.qg_combine_rows(xs, pos, y[k], weights=w[k])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        y.zero_()
        pos.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        xd, wd = x.double(), w.double()
        if grad:
            # products rounded to bf16, f32 sums of topk of them, rounded to bf16
            terms = wd[..., None] * xd[:, :, None]
            A = terms.abs().sum(2)
            assert ((y.double() - terms.sum(2)).abs() <= (2.0 ** -7 + 2.0 ** -14) * A + 1e-30).all()
            # f32 sums of N products
            dots = (xd * xd).sum(-1)
            assert ((dw.double() - dots[..., None]).abs() <= (N + 1) * 2.0 ** -24 * dots[..., None]).all()
        else:
            # f32 sums of topk products, rounded to bf16
            ref, A = wd.sum(2)[..., None] * xd, wd.sum(2)[..., None] * xd.abs()
            assert ((y.double() - ref).abs() <= (2.0 ** -8 + topk * 2.0 ** -22) * A + 1e-30).all()


def test_every_call_on_three_streams_at_once(lib):
    """Few and many rows, dense and per expert, gradients, order and rows, each
    stream in its own order: the bits of the calls one after the other."""
    g = torch.Generator(device="cuda").manual_seed(8)
    rng = np.random.default_rng(8)
    E, N, K, T, topk = 6, 200, 320, 150, 2
    qw, sw, zw = C.weights(rng, N, K, "asym", E)
    packed = C.pack_experts(lib, torch, qw, sw, zw, "asym")

    def lane(k):
        rows = torch.randn((T * topk, K), generator=g, device="cuda").to(BF)
        dys = torch.randn((T * topk, N), generator=g, device="cuda").to(BF)
        ids = torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
        w = torch.rand((T, topk), generator=g, device="cuda")
        o = {"off": _i32(np.zeros(E + 1)), "src": _i32(np.zeros(T * topk)), "pos": _i32(np.zeros((T, topk)))}
        for name, shape in [("few", (9, N)), ("many", (T, N)), ("grad", (T, K)), ("h", (T * topk, N)),
                            ("dx", (T * topk, K)), ("y", (T, N)), ("dh", (T * topk, N)), ("xs", (T * topk, K))]:
            o[name] = torch.zeros(shape, dtype=BF, device="cuda")
        o["dw"] = torch.zeros((T, topk), device="cuda")

        def run(s):
            lib.qg_sort_by_expert(ids, o["off"], o["src"], o["pos"], stream=s)
            lib.qgemm_a16w4_bf16_experts(rows[:T], o["off"], packed, o["h"], src=o["src"], topk=topk,
                                         weights="asym", stream=s)
            lib.qg_combine_rows(o["h"], o["pos"], o["y"], weights=w, stream=s)
            lib.qgemm_a16w4_bf16(rows[:9], packed[k], o["few"], weights="asym", stream=s)
            lib.qgemm_a16w4_bf16(rows[:T], packed[k], o["many"], weights="asym", stream=s)
            lib.qg_combine_rows_grad(o["many"], o["h"], o["pos"], w, o["dh"], o["dw"], stream=s)
            lib.qgemm_a16w4_bf16_grad_x(dys[:T], packed[k], o["grad"], weights="asym", stream=s)
            lib.qgemm_a16w4_bf16_experts_grad_x(o["dh"], o["off"], packed, o["dx"], weights="asym", stream=s)
            lib.qg_spread_rows(o["grad"], o["pos"], o["xs"], stream=s)
        return run, o

    lanes = [lane(k) for k in range(3)]
    want = []
    for run, o in lanes:
        run(None)
        torch.cuda.synchronize()
        want.append({k: t.clone() for k, t in o.items()})
    streams = [torch.cuda.Stream() for _ in lanes]
    for k in range(30):
        for (run, o), s in zip(lanes, streams):
            run(s)
        if k % 10 == 9:
            torch.cuda.synchronize()
            for (_, o), ref in zip(lanes, want):
                for name, t in o.items():
                    assert torch.equal(t, ref[name]), (k, name)
                    t.zero_()
            torch.cuda.synchronize()
