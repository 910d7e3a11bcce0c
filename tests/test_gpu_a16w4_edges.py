"""The weight-only int4 products and the expert rows where indexes, ranges and
addresses are unusual: pairs and many waves of tiles, strides past 32 bits,
ranges and entries that point nowhere, single rows of any length."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16
INVALID = -1


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(BF)


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda):
    lib.qg_device_status(True)
    yield
    assert lib.qg_device_status(True) == 0


# many features: pairs of CTAs, several waves of tiles, every box of rows, a
# half-empty last pair, an odd number of 64-wide blocks
@pytest.mark.parametrize("M,N,K,fmt", [(17, 9600, 192, "f32"), (40, 9500, 128, "bf16"),
                                       (70, 9474, 64, "asym"), (130, 5000, 320, "f32"),
                                       (257, 20000, 64, "bf16"), (600, 6401, 128, "asym")])
def test_pairs_forward(lib, M, N, K, fmt):
    rng = np.random.default_rng(N)
    qw, sw, zw = C.weights(rng, N, K, fmt)
    x = C.bf16_round(rng.standard_normal((M, K)))
    bias = rng.standard_normal(N).astype(np.float32)
    y = torch.empty((M, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16(_bf(x), C.pack(lib, torch, qw, sw, zw, fmt), y, weights=fmt,
                         bias=torch.from_numpy(bias).cuda())
    w = C.real(qw, sw, zw)
    ref = oracle.a16w4(x, w, bias)
    C.assert_close(_np(y), ref, C.tolerance(x.astype(np.float64), w, ref, bias))


@pytest.mark.parametrize("M,N,K,fmt", [(17, 72, 9600, "f32"), (70, 104, 9536, "bf16"),
                                       (300, 200, 6464, "asym"), (257, 64, 20032, "f32")])
def test_pairs_grad(lib, M, N, K, fmt):
    rng = np.random.default_rng(K)
    qw, sw, zw = C.weights(rng, N, K, fmt)
    dy = C.bf16_round(rng.standard_normal((M, N)))
    dx = torch.empty((M, K), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_grad_x(_bf(dy), C.pack(lib, torch, qw, sw, zw, fmt), dx, weights=fmt)
    wt = C.real(qw, sw, zw).T
    ref = oracle.a16w4(dy, wt)
    C.assert_close(_np(dx), ref, C.tolerance(dy.astype(np.float64), wt, ref))


@pytest.mark.parametrize("N", [1, 7, 63, 65, 1001])
def test_single_row_of_any_length(lib, N):
    """The stride of one row says nothing, so a length that is no multiple of
    8 is fine; likewise a row cut out of a wider, odd one."""
    rng = np.random.default_rng(N)
    K = 128
    qw, sw, zw = C.weights(rng, N, K, "f32")
    packed, wt = C.pack(lib, torch, qw, sw, zw, "f32"), C.real(qw, sw, zw).T
    dy = C.bf16_round(rng.standard_normal((1, N)))
    dx = torch.empty((1, K), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_grad_x(_bf(dy), packed, dx)
    ref = oracle.a16w4(dy, wt)
    C.assert_close(_np(dx), ref, C.tolerance(dy.astype(np.float64), wt, ref))
    x = C.bf16_round(rng.standard_normal((1, K)))
    wide = torch.zeros((2, K + 1), dtype=BF, device="cuda")
    wide[0, :K] = _bf(x)[0]
    y = torch.empty((1, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16(wide[:1, :K], packed, y)
    ref = oracle.a16w4(x, wt.T)
    C.assert_close(_np(y), ref, C.tolerance(x.astype(np.float64), wt.T, ref))


@pytest.mark.parametrize("S", [16, 17])
def test_one_matrix_with_offsets(lib, S):
    """E = 1 with a range inside [0, S): both kernels, rows outside it stay."""
    rng = np.random.default_rng(S)
    N, K = 200, 192
    qw, sw, zw = C.weights(rng, N, K, "bf16", 1)
    x = C.bf16_round(rng.standard_normal((S, K)))
    off = torch.tensor([2, S - 1], dtype=torch.int32, device="cuda")
    y = torch.full((S, N), 7.0, dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_experts(_bf(x), off, C.pack_experts(lib, torch, qw, sw, zw, "bf16"), y,
                                 weights="bf16")
    w = C.real(qw, sw, zw)[0]
    ref = oracle.a16w4(x, w)
    y = _np(y)
    C.assert_close(y[2:-1], ref[2:-1], C.tolerance(x.astype(np.float64), w, ref)[2:-1])
    assert (y[:2] == 7.0).all() and (y[-1] == 7.0).all()


@pytest.mark.parametrize("S,ld", [(4, 1 << 30), (20, 1 << 28)])
def test_offsets_past_32_bits(lib, S, ld):
    """Rows, and experts' matrices, more than 2^31 elements and 2^32 bytes apart."""
    rng = np.random.default_rng(S)
    E, N, K = 2, 64, 128
    x_all = torch.empty(((S - 1) * ld + K,), dtype=BF, device="cuda")
    y_all = torch.empty(((S - 1) * ld + N,), dtype=BF, device="cuda")
    x, y = x_all.as_strided((S, K), (ld, 1)), y_all.as_strided((S, N), (ld, 1))
    qw, sw, zw = C.weights(rng, N, K, "f32", E)
    xn = C.bf16_round(rng.standard_normal((S, K)))
    x.copy_(_bf(xn))
    ref = oracle.a16w4(xn, C.real(qw, sw, zw)[0])
    tol = C.tolerance(xn.astype(np.float64), C.real(qw, sw, zw)[0], ref)
    lib.qgemm_a16w4_bf16(x, C.pack(lib, torch, qw[0], sw[0], None, "f32"), y)
    C.assert_close(_np(y), ref, tol)
    # experts, their matrices 2^32 + 2^20 bytes apart
    step = (1 << 32) + (1 << 20)
    one = C.pack(lib, torch, qw[1], sw[1], None, "f32")
    buf = torch.empty((step + one.numel(),), dtype=torch.uint8, device="cuda")
    packed = buf.as_strided((E, one.numel()), (step, 1))
    packed[0].copy_(C.pack(lib, torch, qw[0], sw[0], None, "f32"))
    packed[1].copy_(one)
    half = S // 2
    off = torch.tensor([0, half, S], dtype=torch.int32, device="cuda")
    y.zero_()
    lib.qgemm_a16w4_bf16_experts(x, off, packed, y)
    w = C.real(qw, sw, zw)
    for a, b, e in [(0, half, 0), (half, S, 1)]:
        r = oracle.a16w4(xn[a:b], w[e])
        C.assert_close(_np(y)[a:b], r, C.tolerance(xn[a:b].astype(np.float64), w[e], r))
    # spread and combine over the same rows
    T = S // 2
    pos = torch.arange(S, dtype=torch.int32, device="cuda").flip(0).reshape(T, 2).contiguous()
    t_rows = _bf(xn[:T, :N])
    lib.qg_spread_rows(t_rows, pos, y)
    assert torch.equal(y, t_rows.repeat_interleave(2, 0).flip(0))
    out = torch.empty((T, N), dtype=BF, device="cuda")
    lib.qg_combine_rows(y, pos, out)
    assert torch.equal(out, 2 * t_rows)


BAD = [([-1, 6, 12], [False, True]), ([0, 6, 13], [True, False]), ([7, 6, 12], [False, True]),
       ([0, 13, 12], [False, False])]


@pytest.mark.parametrize("offsets,good", BAD)
@pytest.mark.parametrize("scale", [1, 20])
def test_ranges_that_point_nowhere(lib, offsets, good, scale):
    """Such an expert gets no rows, the others theirs, and the status says so."""
    rng = np.random.default_rng(scale)
    S, E, N, K = 12 * scale, 2, 72, 128
    if scale == 1:
        E, offsets, good = 4, offsets + [offsets[-1]] * 2, good + [True, True]
        if offsets[-1] > S:
            good = good[:2] + [False, False]
    lo = [v * scale for v in offsets]
    qw, sw, zw = C.weights(rng, N, K, "f32", E)
    packed = C.pack_experts(lib, torch, qw, sw, zw, "f32")
    x = C.bf16_round(rng.standard_normal((S, K)))
    dy = C.bf16_round(rng.standard_normal((S, N)))
    off = torch.tensor(lo, dtype=torch.int32, device="cuda")
    w = C.real(qw, sw, zw)
    for grad in (False, True):
        rows, mats = (dy, w.transpose(0, 2, 1)) if grad else (x, w)
        out = torch.full((S, K if grad else N), 7.0, dtype=BF, device="cuda")
        if grad:
            lib.qgemm_a16w4_bf16_experts_grad_x(_bf(dy), off, packed, out)
        else:
            lib.qgemm_a16w4_bf16_experts(_bf(x), off, packed, out)
        assert lib.qg_device_status(True) == INVALID
        out, done = _np(out), np.zeros(S, bool)
        for e in range(E):
            a, b = lo[e], lo[e + 1]
            if good[e] and a < b:
                ref = oracle.a16w4(rows[a:b], mats[e])
                C.assert_close(out[a:b], ref, C.tolerance(rows[a:b].astype(np.float64), mats[e], ref))
                done[a:b] = True
        assert (out[~done] == 7.0).all()


@pytest.mark.parametrize("S", [8, 200])
def test_entries_that_point_nowhere(lib, S):
    """src outside x counts as a row of zeros, a place outside the rows as none."""
    rng = np.random.default_rng(S)
    E, N, K, topk = 2, 64, 128, 2
    T = S // topk
    qw, sw, zw = C.weights(rng, N, K, "f32", E)
    packed, w = C.pack_experts(lib, torch, qw, sw, zw, "f32"), C.real(qw, sw, zw)
    x = C.bf16_round(rng.standard_normal((T, K)))
    src = rng.permutation(S).astype(np.int32)
    src[[0, 3, S - 1]] = [-5, S, 2 ** 31 - 1]
    off = torch.tensor([0, S // 2, S], dtype=torch.int32, device="cuda")
    y = torch.empty((S, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_experts(_bf(x), off, packed, y, src=torch.from_numpy(src).cuda(), topk=topk)
    assert lib.qg_device_status(True) == INVALID
    xs = np.zeros((S, K))
    ok = (src >= 0) & (src < S)
    xs[ok] = x[src[ok] // topk]
    for e, (a, b) in enumerate([(0, S // 2), (S // 2, S)]):
        ref = oracle.a16w4(xs[a:b], w[e])
        C.assert_close(_np(y)[a:b], ref, C.tolerance(xs[a:b], w[e], ref))
    pos = torch.arange(S, dtype=torch.int32, device="cuda").reshape(T, topk).contiguous()
    pos[0, 0], pos[1, 1] = S, 2 ** 31 - 1
    rows = torch.full((S, K), 7.0, dtype=BF, device="cuda")
    lib.qg_spread_rows(_bf(x), pos, rows)
    assert lib.qg_device_status(True) == INVALID
    rows = _np(rows)
    keep = np.ones(S, bool)
    keep[[0, 3]] = False
    assert (rows[~keep] == 7.0).all() and (rows[keep] == np.repeat(x, topk, 0)[keep]).all()
    y1 = torch.empty((T, K), dtype=BF, device="cuda")
    lib.qg_combine_rows(_bf(np.repeat(x, topk, 0)), pos, y1)
    assert lib.qg_device_status(True) == INVALID
    n = np.full((T, 1), 2.0)
    n[:2] = 1.0
    assert (_np(y1) == n * x).all()
    dw = torch.full((T, topk), 7.0, device="cuda")
    lib.qg_combine_rows_grad(_bf(x), _bf(np.repeat(x, topk, 0)), pos, None, None, dw)
    assert lib.qg_device_status(True) == INVALID
    assert float(dw[0, 0]) == 0.0 and float(dw[1, 1]) == 0.0 and float(dw[0, 1]) > 0.0


def _linear(lib, rng, M, N, K):
    qw, sw, zw = C.weights(rng, N, K, "f32")
    packed = C.pack(lib, torch, qw, sw, zw, "f32")
    x = _bf(C.bf16_round(rng.standard_normal((M, K))))
    want = torch.empty((M, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16(x, packed, want)
    return packed, x, want


def test_rows_from_the_call_before(lib):
    """Calls behind one another become resident early; what the one before
    writes is read after it has ended."""
    packed, x, want = _linear(lib, np.random.default_rng(1), 200, 256, 512)
    pos = torch.arange(200, dtype=torch.int32, device="cuda").reshape(200, 1)
    few = torch.empty((8, 256), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16(x[:8], packed, few)
    for _ in range(50):
        xs, y, z = torch.zeros_like(x), torch.zeros_like(want), torch.zeros_like(few)
        lib.qg_spread_rows(x, pos, xs)
        lib.qgemm_a16w4_bf16(xs, packed, y)
        xs.zero_()
        lib.qg_spread_rows(x, pos, xs)
        lib.qgemm_a16w4_bf16(xs[:8], packed, z)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        assert torch.equal(z.view(torch.int16), few.view(torch.int16))


def test_behind_long_work(lib):
    """Behind a call that keeps one SM busy for some 0.1 s, longer than the
    bounded waits of the pipeline: they start to count when it has ended."""
    packed, x, want = _linear(lib, np.random.default_rng(2), 200, 256, 2048)
    N, topk = 1 << 29, 8
    dy = torch.ones((1, N), dtype=BF, device="cuda")
    ys = torch.ones((topk, N), dtype=BF, device="cuda")
    pos = torch.arange(topk, dtype=torch.int32, device="cuda").reshape(1, topk)
    dw = torch.empty((1, topk), device="cuda")
    y, dx = torch.zeros_like(want), torch.empty((200, 2048), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_grad_x(want, packed, dx)
    dx2 = torch.zeros_like(dx)
    lib.qg_combine_rows_grad(dy, ys, pos, None, None, dw)
    lib.qgemm_a16w4_bf16(x, packed, y)
    lib.qg_combine_rows_grad(dy, ys, pos, None, None, dw)
    lib.qgemm_a16w4_bf16_grad_x(want, packed, dx2)
    assert lib.qg_device_status(True) == 0
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    assert torch.equal(dx2.view(torch.int16), dx.view(torch.int16))
    # f32 sums of ones: exact up to 2^24 per thread, and powers of two after it
    assert torch.equal(dw, torch.full_like(dw, float(N)))


@pytest.mark.parametrize("grad", [False, True])
def test_cold_memory(lib, grad):
    """Weights in memory that no kernel has read yet, where tensor copies land
    out of order: the bits of later calls."""
    rng = np.random.default_rng(3)
    E, N, K, S = 64, 1728, 2496, 6000
    cut = np.sort(rng.integers(0, S + 1, E - 1))
    off = torch.tensor([0, *cut.tolist(), S], dtype=torch.int32, device="cuda")
    want = None
    for k in range(6):
        torch.cuda.empty_cache()
        g = torch.Generator(device="cuda").manual_seed(1)
        packed = torch.randint(0, 256, (E, N * K // 2 + N * K // 16), generator=g, device="cuda",
                               dtype=torch.uint8)
        scales = packed[:, N * K // 2:]
        scales.copy_(torch.full((E, N * K // 32), 0.01, dtype=BF, device="cuda").view(torch.uint8))
        rows = torch.randn((S, N if grad else K), generator=g, device="cuda").to(BF)
        out = torch.empty((S, K if grad else N), dtype=BF, device="cuda")
        fresh = torch.empty_like(packed)  # its pages are first touched by the copy engine's writes
        torch.cuda.synchronize()
        fresh.copy_(packed)
        call = lib.qgemm_a16w4_bf16_experts_grad_x if grad else lib.qgemm_a16w4_bf16_experts
        call(rows, off, fresh, out, weights="bf16")
        if want is None:
            again = torch.empty_like(out)
            call(rows, off, fresh, again, weights="bf16")
            want = again.cpu().view(torch.int16)
            del again
        assert torch.equal(out.cpu().view(torch.int16), want), k
        assert lib.qg_device_status(True) == 0
        del packed, scales, rows, out, fresh


# every access width (16, 8, 4 and 2 bytes), by the length or by where the rows
# start, with the experts taken 2, 4 and 8 at a time, many tokens and few
@pytest.mark.parametrize("T,topk", [(200, 1), (200, 2), (170, 4), (160, 5), (151, 11), (5, 2), (3, 9)])
@pytest.mark.parametrize("N,dtype,shift", [(1024, BF, 0), (1020, BF, 0), (1034, BF, 0), (517, BF, 0),
                                           (4091, torch.float16, 0), (512, torch.float16, 1),
                                           (2058, torch.float32, 0), (261, torch.float32, 0),
                                           (2064, BF, 4), (64, torch.float32, 2), (1, BF, 0)])
def test_row_widths(lib, T, topk, N, dtype, shift):
    g = torch.Generator(device="cuda").manual_seed(T * N)
    S = T * topk + 3

    def rows(n):  # rows that start `shift` elements into aligned memory
        flat = torch.randn(n * (N + shift) + shift, generator=g, device="cuda").to(dtype)
        return flat[shift:].view(n, N + shift)[:, :N]

    pos = torch.randperm(S, generator=g, device="cuda")[:T * topk].to(torch.int32).view(T, topk)
    pos[torch.rand((T, topk), generator=g, device="cuda") < 0.2] = -1
    x, ys, dy = rows(T), rows(S), rows(T)
    w = torch.rand((T, topk), generator=g, device="cuda")
    live = pos >= 0
    xs = rows(S)
    before = xs.clone()
    lib.qg_spread_rows(x, pos, xs)
    want = before.clone()
    want[pos[live].long()] = x.repeat_interleave(topk, 0)[live.view(-1)]
    assert torch.equal(xs, want)
    eps = torch.finfo(dtype).eps / 2
    # f32 sums of topk products, one rounding to the rows' type (6e-8: the
    # step of the smallest fp16 values)
    y = rows(T)
    lib.qg_combine_rows(ys, pos, y, weights=w)
    terms = torch.where(live[..., None], w.double()[..., None] * ys.double()[pos.long().clamp(min=0)], 0.0)
    ref, A = terms.sum(1), terms.abs().sum(1)
    inner = topk * 2.0 ** -24 * A
    assert ((y.double() - ref).abs() <= inner + eps * (ref.abs() + inner) + 6e-8).all()
    # products rounded to f32, then to the rows' type; f32 sums of N products
    dys, dw = rows(S), torch.empty_like(w)
    keep = dys.clone()
    lib.qg_combine_rows_grad(dy, ys, pos, w, dys, dw)
    prod = (w.double()[..., None] * dy.double()[:, None])[live]
    at = pos[live].long()
    assert ((dys.double()[at] - prod).abs() <= (eps + 2.0 ** -23) * prod.abs() + 6e-8).all()
    other = torch.ones(S, dtype=torch.bool, device="cuda")
    other[at] = False
    assert torch.equal(dys[other], keep[other])
    dots = torch.where(live[..., None], dy.double()[:, None] * ys.double()[pos.long().clamp(min=0)], 0.0)
    assert ((dw.double() - dots.sum(2)).abs() <= (N + 1) * 2.0 ** -24 * dots.abs().sum(2)).all()


# both sides of every switch between one CTA and chunks of 1024, 2048 and 4096
@pytest.mark.parametrize("T,topk,E", [(255, 8, 64), (256, 8, 64), (257, 8, 64), (1024, 3, 1024), (4096, 8, 60),
                                      (4097, 8, 60), (16384, 8, 1024), (16385, 8, 3), (524288, 8, 256)])
def test_order_across_chunks(lib, T, topk, E):
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-2, E + 2, (T, topk + 3), generator=g, device="cuda", dtype=torch.int32)[:, :topk]
    offsets = torch.empty(E + 1, device="cuda", dtype=torch.int32)
    src = torch.full((T * topk,), -7, device="cuda", dtype=torch.int32)
    pos = torch.empty((T, topk), device="cuda", dtype=torch.int32)
    lib.qg_sort_by_expert(ids, offsets, src, pos)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    want = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device="cuda")).int()
    n = int(want[-1])
    assert torch.equal(offsets, want)
    assert torch.equal(src[:n].long(), order[:n]) and (src[n:] == -7).all()
    places = torch.full((T * topk,), -1, device="cuda", dtype=torch.int32)
    places[order[:n]] = torch.arange(n, device="cuda", dtype=torch.int32)
    assert torch.equal(pos.view(-1), places)
