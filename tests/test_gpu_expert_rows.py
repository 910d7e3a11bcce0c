"""Tokens in the order of their experts and back, against the oracle.

Tolerance of combine: topk products and additions in f32, each off by at most
2^-24 of A = sum_j |w ys| (so 2 topk 2^-24 A), then half a step of the row
type.  dw: N products and additions in f32 in some fixed order, at most
(N + 1) 2^-24 sum_n |dy ys|.  dys: one f32 product (2^-24) and half a step."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda):
    lib.qg_device_status(True)
    yield
    assert lib.qg_device_status(True) == 0


def _sort(lib, ids, E):
    T, topk = ids.shape
    d = torch.from_numpy(ids).cuda()
    off = torch.full((E + 1,), 99, dtype=torch.int32, device="cuda")
    src = torch.full((T * topk,), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((T, topk), 99, dtype=torch.int32, device="cuda")
    lib.qg_sort_by_expert(d, off, src, pos)
    return off, src, pos


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 8, 8), (3, 2, 5), (16, 8, 128), (33, 6, 60),
                                      (257, 4, 1024), (2048, 8, 256), (2049, 8, 64), (9000, 2, 7),
                                      (40000, 1, 1000)])
@pytest.mark.parametrize("kind", ["even", "hot", "holes", "none"])
def test_sort_matches_oracle(lib, T, topk, E, kind):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, topk)).astype(np.int32)   # the same expert twice is allowed
    if kind == "hot":
        ids[:] = E // 2
    if kind == "holes":
        ids = rng.integers(-2, E + 2, (T, topk)).astype(np.int32)
        ids[rng.random((T, topk)) < 0.1] = np.iinfo(np.int32).min
        ids[rng.random((T, topk)) < 0.1] = np.iinfo(np.int32).max
    if kind == "none":
        ids[:] = -1
    off, src, pos = (t.cpu().numpy() for t in _sort(lib, ids, E))
    flat = ids.reshape(-1).astype(np.int64)
    live = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(live, flat, E), kind="stable")
    n = int(live.sum())
    ref_off = np.searchsorted(np.where(live, flat, E)[order], np.arange(E + 1))
    np.testing.assert_array_equal(off, ref_off)
    np.testing.assert_array_equal(src[:n], order[:n])
    assert (src[n:] == -7).all()
    ref_pos = np.full(T * topk, -1)
    ref_pos[order[:n]] = np.arange(n)
    np.testing.assert_array_equal(pos.reshape(-1), ref_pos)


def test_sort_matches_the_oracles_definition(lib):
    ids = C.routing(np.random.default_rng(4), 50, 3, 9, drop=0.2)
    off, src, pos = (t.cpu().numpy() for t in _sort(lib, ids, 9))
    r_off, r_src, r_pos = oracle.sort_by_expert(ids, 9)
    np.testing.assert_array_equal(off, r_off)
    np.testing.assert_array_equal(src[:len(r_src)], r_src)
    np.testing.assert_array_equal(pos, r_pos)


def test_sort_of_strided_ids_and_of_nothing(lib):
    wide = torch.randint(0, 12, (70, 9), dtype=torch.int32, device="cuda")
    off = torch.empty(13, dtype=torch.int32, device="cuda")
    src = torch.empty(70 * 4, dtype=torch.int32, device="cuda")
    pos = torch.empty((70, 4), dtype=torch.int32, device="cuda")
    lib.qg_sort_by_expert(wide[:, 2:6], off, src, pos)
    r_off, r_src, r_pos = oracle.sort_by_expert(wide[:, 2:6].cpu().numpy(), 12)
    np.testing.assert_array_equal(off.cpu().numpy(), r_off)
    np.testing.assert_array_equal(src.cpu().numpy(), r_src)
    np.testing.assert_array_equal(pos.cpu().numpy(), r_pos)
    lib.qg_sort_by_expert(torch.empty((0, 4), dtype=torch.int32, device="cuda"), off, src[:0],
                          pos[:0])
    assert (off == 0).all()


ROWS = [(1, 1, 8), (1, 8, 4096), (3, 2, 1), (7, 9, 33), (5, 17, 130), (64, 4, 2056), (300, 6, 515),
        (1500, 8, 256), (40, 1, 10000)]


def _rows(T, topk, N, dtype, seed, margin=0, drop=0.2):
    """pos over a larger set of places, and rows of that dtype."""
    rng = np.random.default_rng(seed)
    S = T * topk + 3
    pos = rng.permutation(S)[:T * topk].astype(np.int32).reshape(T, topk)
    pos[rng.random((T, topk)) < drop] = -1
    w = rng.standard_normal((T, topk)).astype(np.float32)
    def mk(n):
        full = torch.from_numpy(rng.standard_normal((n, N + margin)).astype(np.float32)).cuda().to(DT[dtype])
        return full[:, :N]
    return S, torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(), mk


@pytest.mark.parametrize("T,topk,N", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("margin", [0, 8, 3])
def test_rows_match_oracle(lib, T, topk, N, dtype, margin):
    S, pos, w, mk = _rows(T, topk, N, dtype, T + N, margin)
    x, ys, dy = mk(T), mk(S), mk(T)
    P = pos.cpu().numpy()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    # spread
    xs = mk(S)
    was = xs.clone()
    lib.qg_spread_rows(x, pos, xs)
    want = was.clone()
    for t in range(T):
        for j in range(topk):
            if P[t, j] >= 0:
                want[P[t, j]] = x[t]
    assert torch.equal(xs, want)
    # combine, with and without weights
    for weights in (w, None):
        y = mk(T)
        lib.qg_combine_rows(ys, pos, y, weights=weights)
        wn = None if weights is None else weights.cpu().numpy()
        ref = oracle.combine_rows(f64(ys), P, wn, N)
        A = oracle.combine_rows(np.abs(f64(ys)), P, None if wn is None else np.abs(wn), N)
        inner = 2 * topk * 2.0 ** -24 * A
        assert (np.abs(f64(y) - ref) <= inner + HALF[dtype] * (np.abs(ref) + inner) + 1e-7 * (dtype == "f16")).all()
    # its gradient
    dys, dw = mk(S), torch.full((T, topk), 5.0, device="cuda")
    was = dys.clone()
    lib.qg_combine_rows_grad(dy, ys, pos, w, dys, dw)
    g, r, wn = f64(dy), f64(ys), w.double().cpu().numpy()
    got, gw = f64(dys), dw.double().cpu().numpy()
    used = np.zeros(S, bool)
    for t in range(T):
        for j in range(topk):
            p = P[t, j]
            if p < 0:
                assert gw[t, j] == 0.0
                continue
            used[p] = True
            ref = wn[t, j] * g[t]
            assert (np.abs(got[p] - ref) <= (HALF[dtype] + 2.0 ** -23) * np.abs(ref) + 6e-8 * (dtype == "f16")).all()
            assert abs(gw[t, j] - g[t] @ r[p]) <= (N + 1) * 2.0 ** -24 * (np.abs(g[t]) @ np.abs(r[p]))
    assert torch.equal(dys[torch.from_numpy(~used).cuda()], was[torch.from_numpy(~used).cuda()])
    # one gradient at a time gives the same bits
    dys2, dw2 = was.clone(), torch.empty_like(dw)
    lib.qg_combine_rows_grad(dy, None, pos, w, dys2, None)
    lib.qg_combine_rows_grad(dy, ys, pos, w, None, dw2)
    assert torch.equal(dys2, dys) and torch.equal(dw2, dw)


def test_rows_gradients_against_differences(lib):
    """f32: the gradient of sum(y * c) by central differences in 64 bits."""
    S, pos, w, mk = _rows(6, 3, 20, "f32", 9)
    ys, c = mk(S), mk(6)
    dys, dw = torch.zeros((S, 20), device="cuda"), torch.empty((6, 3), device="cuda")
    lib.qg_combine_rows_grad(c.contiguous(), ys.contiguous(), pos, w, dys, dw)
    P, h = pos.cpu().numpy(), 1e-4
    f = lambda a, b: float((oracle.combine_rows(a, P, b, 20) * c.double().cpu().numpy()).sum())  # noqa: E731
    a0, b0 = ys.double().cpu().numpy(), w.double().cpu().numpy()
    for i, j in [(0, 0), (4, 7), (S - 1, 19), (9, 3)]:
        up, dn = a0.copy(), a0.copy()
        up[i, j] += h
        dn[i, j] -= h
        assert abs((f(up, b0) - f(dn, b0)) / (2 * h) - float(dys[i, j])) < 1e-5
    for i, j in [(0, 0), (3, 2), (5, 1)]:
        up, dn = b0.copy(), b0.copy()
        up[i, j] += h
        dn[i, j] -= h
        assert abs((f(a0, up) - f(a0, dn)) / (2 * h) - float(dw[i, j])) < 1e-4


def test_a_place_outside_is_recorded_and_skipped(lib):
    pos = torch.tensor([[0], [5], [1]], dtype=torch.int32, device="cuda")
    x = torch.arange(12, dtype=torch.float32, device="cuda").view(3, 4)
    xs = torch.full((2, 4), -1.0, device="cuda")
    lib.qg_spread_rows(x, pos, xs)
    assert lib.qg_device_status(True) == -1
    assert torch.equal(xs, torch.stack([x[0], x[2]]))
    y = torch.empty((3, 4), device="cuda")
    lib.qg_combine_rows(xs, pos, y)
    assert lib.qg_device_status(True) == -1
    assert torch.equal(y, torch.stack([x[0], torch.zeros(4, device="cuda"), x[2]]))


def test_sort_spread_combine_in_a_graph_round_trip(lib):
    """Captured and replayed with other ids: combine of two halves gives x back."""
    T, topk, E, N = 200, 2, 32, 96
    ids = torch.randint(0, E, (T, topk), dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    src = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    pos = torch.empty((T, topk), dtype=torch.int32, device="cuda")
    x, xs = torch.randn((T, N), device="cuda"), torch.empty((T * topk, N), device="cuda")
    y, w = torch.empty_like(x), torch.full((T, topk), 0.5, device="cuda")

    def step():
        lib.qg_sort_by_expert(ids, off, src, pos)
        lib.qg_spread_rows(x, pos, xs)
        lib.qg_combine_rows(xs, pos, y, weights=w)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        ids.copy_(torch.randint(0, E, (T, topk), dtype=torch.int32, device="cuda"))
        x.copy_(torch.randn((T, N), device="cuda"))
        g.replay()
        assert torch.equal(y, x)
        assert torch.equal(pos.view(-1)[src.long()], torch.arange(T * topk, device="cuda", dtype=torch.int32))
