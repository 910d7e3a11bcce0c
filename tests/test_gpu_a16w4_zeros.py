"""Asymmetric weights whose zero is far larger than the scale, or cancels the
code: each weight is one rounding of s*c + z in f32, then one to bf16.

Tolerance, with w = s*c + z exactly: a weight is off by (2^-8 + 2^-23) |w| at
most, so the sums by that much of A = sum |x w|; the f32 sums add 2^-23 of the
partial sums (at most A) for each of 32 additions in a group and 2^-24 for
K/32 + 16 more, as in a16w4_cases; then half a step of the output."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


def _weights(rng, kind, N, K):
    qw, sw, _ = C.weights(rng, N, K, "f32")
    if kind == "cancel":      # s*c + z is the f32 rounding of s*c alone
        qw = np.repeat(rng.integers(-8, 8, (N, K // 32)), 32, axis=1).astype(np.int8)
        return qw, sw, -(sw * qw[:, ::32].astype(np.float32))
    if kind == "partly":      # one code of each group cancels, the others do not
        return qw, sw, -(sw * rng.integers(-8, 8, sw.shape).astype(np.float32))
    return qw, sw, sw * np.float32(1000.0) * rng.choice([-1.0, 1.0], sw.shape).astype(np.float32)


def _check(y, rows, w):
    ref = rows @ w.T
    A = np.abs(rows) @ np.abs(w).T
    inner = (2.0 ** -8 + 2.0 ** -23 + (64 + w.shape[1] / 32 + 16) * 2.0 ** -24) * A
    C.assert_close(y.double().cpu().numpy(), ref, inner + 2.0 ** -8 * (np.abs(ref) + inner) + 1e-30)


@pytest.mark.parametrize("kind", ["cancel", "partly", "far"])
@pytest.mark.parametrize("M,N,K", [(40, 200, 256), (300, 136, 320), (70, 9474, 64)])
def test_zero_and_code(lib, cuda, kind, M, N, K):
    rng = np.random.default_rng(M + N)
    qw, sw, zw = _weights(rng, kind, N, K)
    packed, w = C.pack(lib, torch, qw, sw, zw, "asym"), oracle.w4_values(qw, sw, zw)
    x = C.bf16_round(rng.standard_normal((M, K))).astype(np.float64)
    y = torch.empty((M, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16(torch.from_numpy(x).cuda().to(BF), packed, y, weights="asym")
    _check(y, x, w)
    ld = -(-N // 8) * 8
    dy = C.bf16_round(rng.standard_normal((M, N))).astype(np.float64)
    dyd = torch.zeros((M, ld), dtype=BF, device="cuda")
    dyd[:, :N] = torch.from_numpy(dy).cuda().to(BF)
    dx = torch.empty((M, K), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_grad_x(dyd[:, :N], packed, dx, weights="asym")
    _check(dx, dy, w.T)
