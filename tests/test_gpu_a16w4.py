"""The weight-only int4 products (bf16 rows) against the float64 oracle,
through the C ABI, with the tolerances derived in tests/a16w4_cases.py."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda):
    lib.qg_device_status(True)
    yield
    assert lib.qg_device_status(True) == 0


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().bfloat16()


def _np(t):
    return t.float().cpu().numpy()


SHAPES = [(1, 14336, 4096), (1, 1, 64), (2, 17, 64), (3, 33, 128), (8, 100, 192), (9, 129, 832),
          (16, 1000, 1024), (17, 64, 2112), (32, 257, 4096), (33, 128, 512), (70, 300, 320),
          (127, 144, 64), (129, 127, 448), (256, 384, 1024), (300, 513, 576), (7, 4097, 256),
          (1, 700, 14336), (64, 2048, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "asym"])
def test_linear_matches_oracle(lib, M, N, K, fmt):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    qw, sw, zw = C.weights(rng, N, K, fmt)
    x = C.bf16_round(rng.standard_normal((M, K)))
    bias = rng.standard_normal(N).astype(np.float32) if N % 2 else None
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16(_bf16(x), C.pack(lib, torch, qw, sw, zw, fmt), y,
                         bias=None if bias is None else torch.from_numpy(bias).cuda(), weights=fmt)
    w = C.real(qw, sw, zw)
    ref = oracle.a16w4(x, w, bias)
    C.assert_close(_np(y), ref, C.tolerance(x.astype(np.float64), w, ref, bias), f"{M}x{N}x{K} {fmt}")


@pytest.mark.parametrize("M,N,K", [(5, 70, 256), (200, 136, 320)])
def test_linear_row_strides_and_margins(lib, M, N, K):
    """Padded rows of x; y at an odd element with an odd pitch: the bytes
    around y's rows stay."""
    rng = np.random.default_rng(11)
    qw, sw, zw = C.weights(rng, N, K, "f32")
    x = C.bf16_round(rng.standard_normal((M, K)))
    xs = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    xs[:, :K] = _bf16(x)
    flat = torch.full((M * (N + 3) + 5,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = flat[1:1 + M * (N + 3)].view(M, N + 3)[:, :N]
    lib.qgemm_a16w4_bf16(xs[:, :K], C.pack(lib, torch, qw, sw, zw, "f32"), y)
    w = C.real(qw, sw, zw)
    ref = oracle.a16w4(x, w)
    C.assert_close(_np(y), ref, C.tolerance(x.astype(np.float64), w, ref))
    flat = _np(flat)
    assert flat[0] == 3.0 and (flat[1:1 + M * (N + 3)].reshape(M, N + 3)[:, N:] == 3.0).all()
    assert (flat[1 + M * (N + 3):] == 3.0).all()


@pytest.mark.parametrize("M", [1, 9, 40, 150])
def test_linear_rows_do_not_mix(lib, M):
    """A row with NaN and infinities changes no other row."""
    rng = np.random.default_rng(M)
    N, K = 130, 512
    qw, sw, zw = C.weights(rng, N, K, "asym")
    packed = C.pack(lib, torch, qw, sw, zw, "asym")
    x = C.bf16_round(rng.standard_normal((M, K)))
    xd = _bf16(x)
    y0 = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16(xd, packed, y0, weights="asym")
    bad = M // 2
    xd[bad, 3] = float("nan")
    xd[bad, 100] = float("inf")
    y1 = torch.empty_like(y0)
    lib.qgemm_a16w4_bf16(xd, packed, y1, weights="asym")
    keep = torch.arange(M, device="cuda") != bad
    assert torch.equal(y0[keep].view(torch.int16), y1[keep].view(torch.int16))
    assert torch.isnan(y1[bad].float()).all()


EXPERTS = [  # T, topk, E, N, K, drop, hot
    (1, 1, 1, 64, 64, 0.0, None), (1, 8, 64, 200, 256, 0.0, None), (8, 8, 64, 130, 512, 0.0, None),
    (5, 2, 9, 65, 192, 0.3, None), (40, 4, 16, 264, 320, 0.1, 3), (3, 1, 1024, 24, 64, 0.0, None),
    (130, 6, 8, 136, 448, 0.2, None), (700, 2, 4, 128, 256, 0.0, 1), (64, 2, 300, 40, 128, 0.0, None),
    (300, 8, 60, 72, 832, 0.4, None)]


def _experts(lib, T, topk, E, N, K, fmt, drop, hot, seed):
    rng = np.random.default_rng(seed)
    qw, sw, zw = C.weights(rng, N, K, fmt, E)
    ids = C.routing(rng, T, topk, E, drop, hot)
    offsets, src, pos = oracle.sort_by_expert(ids, E)
    S = T * topk
    src_d = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    src_d[:len(src)] = torch.from_numpy(src.astype(np.int32)).cuda()
    off_d = torch.from_numpy(offsets.astype(np.int32)).cuda()
    return rng, (qw, sw, zw), C.pack_experts(lib, torch, qw, sw, zw, fmt, gap=48), offsets, src, off_d, src_d


@pytest.mark.parametrize("T,topk,E,N,K,drop,hot", EXPERTS)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "asym"])
@pytest.mark.parametrize("gathered", [True, False])
def test_experts_match_oracle(lib, T, topk, E, N, K, drop, hot, fmt, gathered):
    rng, (qw, sw, zw), packed, offsets, src, off_d, src_d = _experts(
        lib, T, topk, E, N, K, fmt, drop, hot, T + N)
    S = T * topk
    x = C.bf16_round(rng.standard_normal((T if gathered else S, K)))
    bias = rng.standard_normal((E, N)).astype(np.float32) if E % 2 else None
    y = torch.full((S, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16_experts(_bf16(x), off_d, packed, y, src=src_d if gathered else None,
                                 topk=topk, weights=fmt,
                                 bias=None if bias is None else torch.from_numpy(bias).cuda())
    y = _np(y)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        xe = x[src[a:b] // topk] if gathered else x[a:b]
        w = C.real(qw[e], sw[e], None if zw is None else zw[e])
        be = None if bias is None else bias[e]
        ref = oracle.a16w4(xe, w, be)
        C.assert_close(y[a:b], ref, C.tolerance(xe.astype(np.float64), w, ref, be), f"expert {e}")
    assert (y[offsets[E]:] == 7.0).all()      # rows behind the last expert stay


GRADS = [(1, 8, 64), (3, 64, 128), (17, 72, 192), (64, 128, 64), (100, 1000, 832), (129, 136, 448),
         (256, 512, 1024), (300, 520, 576), (513, 2056, 320), (33, 4096, 256)]


@pytest.mark.parametrize("M,N,K", GRADS)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "asym"])
def test_linear_grad_matches_oracle(lib, M, N, K, fmt):
    rng = np.random.default_rng(M + N + K)
    qw, sw, zw = C.weights(rng, N, K, fmt)
    dy = C.bf16_round(rng.standard_normal((M, N)))
    dx = torch.full((M, K + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16_grad_x(_bf16(dy), C.pack(lib, torch, qw, sw, zw, fmt), dx[:, :K], weights=fmt)
    wt = C.real(qw, sw, zw).T
    ref = oracle.a16w4(dy, wt)
    C.assert_close(_np(dx)[:, :K], ref, C.tolerance(dy.astype(np.float64), wt, ref), f"{M}x{N}x{K} {fmt}")
    assert (_np(dx)[:, K:] == 7.0).all()


def test_linear_grad_against_differences(lib):
    """The gradient of sum(y * dy) by central differences of the oracle's y;
    linear in x, so the difference is exact up to its 64-bit rounding and the
    rounding of dx (tolerance of the product)."""
    rng = np.random.default_rng(2)
    M, N, K = 40, 72, 128
    qw, sw, zw = C.weights(rng, N, K, "asym")
    w = C.real(qw, sw, zw)
    dy = C.bf16_round(rng.standard_normal((M, N)))
    x = rng.standard_normal((M, K))
    dx = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16_grad_x(_bf16(dy), C.pack(lib, torch, qw, sw, zw, "asym"), dx, weights="asym")
    tol = C.tolerance(dy.astype(np.float64), w.T, dy.astype(np.float64) @ w)
    for m, k in [(0, 0), (39, 127), (7, 64), (20, 31)]:
        up, dn = x.copy(), x.copy()
        up[m, k] += 0.5
        dn[m, k] -= 0.5
        diff = ((oracle.a16w4(up, w) - oracle.a16w4(dn, w)) * dy).sum()
        assert abs(diff - float(dx[m, k])) <= tol[m, k] + 1e-10


@pytest.mark.parametrize("T,topk,E,N,K,drop,hot", EXPERTS)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "asym"])
def test_experts_grad_matches_oracle(lib, T, topk, E, N, K, drop, hot, fmt):
    rng, (qw, sw, zw), packed, offsets, src, off_d, _ = _experts(
        lib, T, topk, E, N, K, fmt, drop, hot, T + K)
    S = T * topk
    ld = -(-N // 8) * 8
    dy = C.bf16_round(rng.standard_normal((S, N)))
    dyd = torch.full((S, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    dyd[:, :N] = _bf16(dy)
    dx = torch.full((S, K), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16_experts_grad_x(dyd[:, :N], off_d, packed, dx, weights=fmt)
    dx = _np(dx)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            wt = C.real(qw[e], sw[e], None if zw is None else zw[e]).T
            ref = oracle.a16w4(dy[a:b], wt)
            C.assert_close(dx[a:b], ref, C.tolerance(dy[a:b].astype(np.float64), wt, ref), f"expert {e}")
    assert (dx[offsets[E]:] == 7.0).all()


def test_experts_without_any_row(lib):
    """No entry has an expert: nothing is written."""
    rng = np.random.default_rng(5)
    qw, sw, zw = C.weights(rng, 64, 128, "f32", 4)
    packed = C.pack_experts(lib, torch, qw, sw, zw, "f32")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    y = torch.full((6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((6, 128), dtype=torch.bfloat16, device="cuda")
    lib.qgemm_a16w4_bf16_experts(x, off, packed, y)
    assert (y == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(4, 256, 512), (200, 256, 512)])
def test_linear_on_its_own_stream_and_in_a_graph(lib, M, N, K):
    """Two captured graphs of one call replayed on two streams, and the eager
    call, give the same bits."""
    rng = np.random.default_rng(3)
    qw, sw, zw = C.weights(rng, N, K, "f32")
    packed = C.pack(lib, torch, qw, sw, zw, "f32")
    x = _bf16(C.bf16_round(rng.standard_normal((M, K))))
    y = [torch.zeros((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    lib.qgemm_a16w4_bf16(x, packed, y[2])
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.qgemm_a16w4_bf16(x, packed, y[k])
            lib.qgemm_a16w4_bf16(x, packed, y[k])
        graphs.append(g)
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            graphs[k].replay()
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(y[k].view(torch.int16), y[2].view(torch.int16))
