"""A gated expert layer over int4 weights, forward and backward, from the calls
that it takes together: order by expert, the two products per expert, the
weighted sum, and their gradients.  Every stage is checked against the float64
formula at the stage's own inputs; the whole chain against differences."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


class Layer:
    """Experts of H -> 2F, gate, F -> H."""

    def __init__(self, lib, rng, E, H, F, fmt, gated=True):
        self.lib, self.E, self.H, self.F, self.fmt, self.gated = lib, E, H, F, fmt, gated
        up = C.weights(rng, 2 * F if gated else F, H, fmt, E)
        down = C.weights(rng, H, F, fmt, E)
        self.up, self.down = C.real(*up), C.real(*down)      # float64 [E][N][K]
        self.up_packed = C.pack_experts(lib, torch, *up, fmt)
        self.down_packed = C.pack_experts(lib, torch, *down, fmt)

    def rows(self, S, N):
        """Rows that nobody has written hold NaN: none may reach a result."""
        return torch.full((S, N), float("nan"), dtype=BF, device="cuda")

    def forward(self, x, ids, weights):
        lib, (T, topk) = self.lib, ids.shape
        S = T * topk
        r = {"x": x, "w": weights}
        r["offsets"] = torch.empty(self.E + 1, dtype=torch.int32, device="cuda")
        r["src"] = torch.full((S,), -1, dtype=torch.int32, device="cuda")
        r["pos"] = torch.empty((T, topk), dtype=torch.int32, device="cuda")
        lib.qg_sort_by_expert(ids, r["offsets"], r["src"], r["pos"])
        r["h"] = self.rows(S, 2 * self.F if self.gated else self.F)
        lib.qgemm_a16w4_bf16_experts(x, r["offsets"], self.up_packed, r["h"], src=r["src"], topk=topk,
                                     weights=self.fmt)
        r["act"] = self.gate(r["h"]) if self.gated else r["h"]
        r["ys"] = self.rows(S, self.H)
        lib.qgemm_a16w4_bf16_experts(r["act"], r["offsets"], self.down_packed, r["ys"], weights=self.fmt)
        r["y"] = torch.empty_like(x)
        lib.qg_combine_rows(r["ys"], r["pos"], r["y"], weights=weights)
        return r

    def backward(self, r, dy):
        lib, S = self.lib, r["ys"].shape[0]
        r["dys"] = self.rows(S, self.H)
        r["dw"] = torch.empty_like(r["w"])
        lib.qg_combine_rows_grad(dy, r["ys"], r["pos"], r["w"], r["dys"], r["dw"])
        r["dact"] = self.rows(S, self.F)
        lib.qgemm_a16w4_bf16_experts_grad_x(r["dys"], r["offsets"], self.down_packed, r["dact"],
                                            weights=self.fmt)
        r["dh"] = self.gate_grad(r["h"], r["dact"]) if self.gated else r["dact"]
        r["dxs"] = self.rows(S, self.H)
        lib.qgemm_a16w4_bf16_experts_grad_x(r["dh"], r["offsets"], self.up_packed, r["dxs"],
                                            weights=self.fmt)
        r["dx"] = torch.empty_like(r["x"])
        lib.qg_combine_rows(r["dxs"], r["pos"], r["dx"])
        return r

    def gate(self, h):
        a, b = h.float().chunk(2, 1)
        return (a * torch.sigmoid(a) * b).to(BF)

    def gate_grad(self, h, d):
        a, b = h.float().chunk(2, 1)
        s, d = torch.sigmoid(a), d.float()
        return torch.cat((d * b * s * (1 + a * (1 - s)), d * a * s), 1).to(BF)


def _inputs(rng, T, topk, E, H, drop):
    ids = C.routing(rng, T, topk, E, drop)
    x = C.bf16_round(rng.standard_normal((T, H)))
    dy = C.bf16_round(rng.standard_normal((T, H)))
    w = rng.random((T, topk)).astype(np.float32)
    return (torch.from_numpy(ids).cuda(), torch.from_numpy(x).cuda().to(BF),
            torch.from_numpy(w).cuda(), torch.from_numpy(dy).cuda().to(BF))


def _check_products(got, rows, w, offsets, label):
    """rows @ w[e]^T of every expert, at the rows' own values."""
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            ref = oracle.a16w4(rows[a:b], w[e])
            C.assert_close(got[a:b], ref, C.tolerance(rows[a:b], w[e], ref), f"{label} expert {e}")


def _check_sum(got, ys, pos, w, label):
    """Sums of topk products in f32 (each step off by 2^-24 of the sum of the
    absolute values at most), rounded to bf16."""
    T, topk = pos.shape
    ref = oracle.combine_rows(ys, pos, w, ys.shape[1])
    A = oracle.combine_rows(np.abs(ys), pos, None if w is None else np.abs(w), ys.shape[1])
    inner = topk * 2.0 ** -24 * A
    C.assert_close(got, ref, inner + 2.0 ** -8 * (np.abs(ref) + inner) + 1e-30, label)


def check(layer, r, ids, dy):
    ids = ids.cpu().numpy()
    offsets, src, pos = oracle.sort_by_expert(ids, layer.E)
    n, topk = int(offsets[-1]), ids.shape[1]
    assert (_np(r["offsets"]) == offsets).all() and (_np(r["pos"]) == pos).all()
    assert (_np(r["src"])[:n] == src).all() and (_np(r["src"])[n:] == -1).all()
    w, dy = _np(r["w"]), _np(dy)
    _check_products(_np(r["h"])[:n], _np(r["x"])[src // topk], layer.up, offsets, "up")
    _check_products(_np(r["ys"])[:n], _np(r["act"])[:n], layer.down, offsets, "down")
    assert np.isnan(_np(r["ys"])[n:]).all()
    ys = np.nan_to_num(_np(r["ys"]))
    _check_sum(_np(r["y"]), ys, pos, w, "y")
    # gradients
    t, j = np.divmod(src, topk)
    ref = w[t, j][:, None] * dy[t]
    # a product rounded to f32, then to bf16
    C.assert_close(_np(r["dys"])[:n], ref, (2.0 ** -8 + 2.0 ** -23) * np.abs(ref) + 1e-30, "dys")
    dots, A = np.zeros(pos.shape), np.zeros(pos.shape)
    dots[t, j], A[t, j] = (dy[t] * ys[:n]).sum(1), np.abs(dy[t] * ys[:n]).sum(1)
    # f32 sums of H products, in whatever order
    C.assert_close(_np(r["dw"]), dots, layer.H * 2.0 ** -24 * A, "dw")
    up_t, down_t = layer.up.transpose(0, 2, 1), layer.down.transpose(0, 2, 1)
    _check_products(_np(r["dact"])[:n], _np(r["dys"])[:n], down_t, offsets, "dact")
    _check_products(_np(r["dxs"])[:n], _np(r["dh"])[:n], up_t, offsets, "dxs")
    _check_sum(_np(r["dx"]), np.nan_to_num(_np(r["dxs"])), pos, None, "dx")
    assert np.isfinite(_np(r["y"])).all() and np.isfinite(_np(r["dx"])).all()


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda):
    lib.qg_device_status(True)
    yield
    assert lib.qg_device_status(True) == 0


# one token, a step of a few, ragged ones on both sides of the kernels' switch
# (4 rows per expert), a long one; some tokens without an expert
CASES = [(1, 2, 8, 128, 64, 0.0), (8, 4, 16, 192, 128, 0.2), (16, 2, 8, 256, 192, 0.0),
         (17, 2, 8, 256, 192, 0.1), (300, 3, 5, 320, 192, 0.3), (6, 3, 4, 64, 64, 1.0),
         (900, 4, 6, 448, 320, 0.0)]


@pytest.mark.parametrize("T,topk,E,H,F,drop", CASES)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "asym"])
def test_layer_forward_and_backward(lib, T, topk, E, H, F, drop, fmt):
    rng = np.random.default_rng(T + H)
    layer = Layer(lib, rng, E, H, F, fmt)
    ids, x, w, dy = _inputs(rng, T, topk, E, H, drop)
    r = layer.backward(layer.forward(x, ids, w), dy)
    check(layer, r, ids, dy)


def test_layer_with_one_expert_for_everybody(lib):
    """Every token on the same expert, twice each: one range holds all rows."""
    rng = np.random.default_rng(4)
    layer = Layer(lib, rng, 16, 128, 64, "f32")
    _, x, w, dy = _inputs(rng, 20, 2, 16, 128, 0.0)
    ids = torch.full((20, 2), 11, dtype=torch.int32, device="cuda")
    r = layer.backward(layer.forward(x, ids, w), dy)
    check(layer, r, ids, dy)


@pytest.mark.parametrize("T", [4, 200])
def test_layer_captured_in_a_graph(lib, T):
    """Forward and backward in one graph, replayed with other tokens and other
    routes on a stream of its own: the bits of the eager calls."""
    rng = np.random.default_rng(T)
    E, H, F, topk = 8, 256, 128, 2
    layer = Layer(lib, rng, E, H, F, "f32")
    static = _inputs(rng, T, topk, E, H, 0.1)
    ids, x, w, dy = static
    layer.backward(layer.forward(x, ids, w), dy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = layer.backward(layer.forward(x, ids, w), dy)
    side = torch.cuda.Stream()
    for _ in range(3):
        new = _inputs(rng, T, topk, E, H, 0.3)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for a, b in zip(static, new):
                a.copy_(b)
            g.replay()
            eager = layer.backward(layer.forward(new[1], new[0], new[2]), new[3])
        torch.cuda.synchronize()
        for k in ("offsets", "pos", "y", "dw", "dx"):
            a, b = captured[k], eager[k]
            assert torch.equal(a.view(torch.int16) if a.dtype == BF else a,
                               b.view(torch.int16) if b.dtype == BF else b), k
        check(layer, eager, new[0], new[3])


@pytest.mark.parametrize("T", [3, 64])
def test_chain_gradient_against_differences(lib, T):
    """Without the gate the layer is linear in x, so central differences of the
    float64 chain are its gradient up to 64-bit rounding.  The bound follows
    the roundings of each stage through the absolute values of the next."""
    rng = np.random.default_rng(9 + T)
    E, H, F, topk = 4, 128, 64, 2
    layer = Layer(lib, rng, E, H, F, "asym", gated=False)
    ids, x, w, dy = _inputs(rng, T, topk, E, H, 0.1)
    r = layer.backward(layer.forward(x, ids, w), dy)
    idn, xn, wn, dyn = ids.cpu().numpy(), _np(x), _np(w), _np(dy)

    def loss(v):
        total = 0.0
        for t in range(T):
            for j in range(topk):
                e = idn[t, j]
                if e >= 0:
                    total += wn[t, j] * (layer.down[e] @ (layer.up[e] @ v[t])) @ dyn[t]
        return total

    bound = np.zeros((T, H))
    for t in range(T):
        for j in range(topk):
            e = idn[t, j]
            if e < 0:
                continue
            d = np.abs(wn[t, j] * dyn[t])[None]
            err = (2.0 ** -8 + 2.0 ** -23) * d
            for m in (layer.down[e].T, layer.up[e].T):
                # magnitude and error of the product of values d off by err
                full = d + err
                err = err @ np.abs(m).T + C.tolerance(full, m, full @ np.abs(m).T)
                d = full @ np.abs(m).T
            bound[t] += (err + topk * 2.0 ** -24 * (d + err))[0]
    dx = _np(r["dx"])
    bound += 2.0 ** -8 * (np.abs(dx) + bound)
    for t, k in [(0, 0), (T - 1, H - 1), (T // 2, 17), (1, 64)]:
        up, dn = xn.copy(), xn.copy()
        up[t, k] += 0.5
        dn[t, k] -= 0.5
        assert abs(loss(up) - loss(dn) - dx[t, k]) <= bound[t, k] + 1e-9
