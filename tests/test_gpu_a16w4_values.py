"""The weight-only int4 products at values that show how they are formed: whole
numbers (exact codes), powers of two as factors, infinities."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16
FORMATS = ["f32", "bf16", "asym"]


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda):
    lib.qg_device_status(True)
    yield
    assert lib.qg_device_status(True) == 0


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(BF)


def _weights(rng, N, K, fmt, E=None):
    qw, sw, zw = C.weights(rng, N, K, fmt, E)
    if fmt == "asym":            # zeros that are no multiple of the scales
        zw = (zw * rng.uniform(0.9, 1.1, zw.shape)).astype(np.float32)
    return qw, sw, zw


@pytest.mark.parametrize("M,N,K", [(1, 700, 256), (2, 1000, 64), (8, 130, 14336), (9, 300, 832), (16, 257, 4096)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("with_bias", [False, True])
def test_few_rows_use_the_codes_exactly(lib, M, N, K, fmt, with_bias):
    rng = np.random.default_rng(M + N)
    qw, sw, zw = _weights(rng, N, K, fmt)
    x = C.integer_rows(rng, M, K)
    bias = rng.standard_normal(N).astype(np.float32) if with_bias else None
    y = torch.empty((M, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16(_bf(x), C.pack(lib, torch, qw, sw, zw, fmt), y, weights=fmt,
                         bias=None if bias is None else torch.from_numpy(bias).cuda())
    ref = oracle.a16w4(x, C.real(qw, sw, zw), bias)
    C.assert_close(y.double().cpu().numpy(), ref, C.exact_codes_tolerance(x.astype(np.float64), qw, sw, zw, ref, bias))


@pytest.mark.parametrize("S,E", [(30, 16), (100, 25), (16, 1)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_few_rows_per_expert_use_the_codes_exactly(lib, S, E, fmt):
    rng = np.random.default_rng(S)
    N, K = 136, 320
    qw, sw, zw = _weights(rng, N, K, fmt, E)
    cut = [0, *sorted(rng.integers(0, S + 1, E - 1).tolist()), S]
    x = C.integer_rows(rng, S, K)
    y = torch.empty((S, N), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_experts(_bf(x), torch.tensor(cut, dtype=torch.int32, device="cuda"),
                                 C.pack_experts(lib, torch, qw, sw, zw, fmt), y, weights=fmt)
    y = y.double().cpu().numpy()
    for e in range(E):
        a, b = cut[e], cut[e + 1]
        if a < b:
            z = None if zw is None else zw[e]
            ref = oracle.a16w4(x[a:b], C.real(qw[e], sw[e], z))
            C.assert_close(y[a:b], ref, C.exact_codes_tolerance(x[a:b].astype(np.float64), qw[e], sw[e], z, ref),
                           f"expert {e}")


@pytest.mark.parametrize("M", [1, 12, 40, 300])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("power", [-60, 100])
def test_powers_of_two_pass_through(lib, M, fmt, power):
    """Rows times 2^power give the bits of the rows' own results times it: no
    sum on the way leaves the range (sum |x| of a group stays below 2^120)."""
    rng = np.random.default_rng(M)
    N, K = 200, 512
    packed = C.pack(lib, torch, *_weights(rng, N, K, fmt), fmt)
    x = _bf(rng.standard_normal((M, K)))
    y, ys = (torch.empty((M, N), dtype=BF, device="cuda") for _ in range(2))
    lib.qgemm_a16w4_bf16(x, packed, y, weights=fmt)
    lib.qgemm_a16w4_bf16(x * 2.0 ** power, packed, ys, weights=fmt)
    assert torch.isfinite(ys).all() and torch.equal(ys, y * 2.0 ** power)


# one infinite value, and nothing else that is not finite, in one row
@pytest.mark.parametrize("M", [1, 8, 16, 17, 40, 150, 300])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_value(lib, M, fmt, sign):
    """Many rows: an infinity of the weight's sign.  Up to 16 rows: infinite or
    NaN, as the header has it (the codes go in as c + 136).  Other rows keep
    their bits."""
    rng = np.random.default_rng(M)
    N, K, k = 136, 320, 77
    qw, sw, zw = _weights(rng, N, K, fmt)
    qw[qw[:, k] == 0, k] = 3     # an infinity times 0 is NaN in the formula
    packed, w = C.pack(lib, torch, qw, sw, zw, fmt), C.real(qw, sw, zw)
    x = _bf(rng.standard_normal((M, K)))
    y, yi = (torch.empty((M, N), dtype=BF, device="cuda") for _ in range(2))
    lib.qgemm_a16w4_bf16(x, packed, y, weights=fmt)
    bad = M // 2
    x[bad, k] = sign * float("inf")
    lib.qgemm_a16w4_bf16(x, packed, yi, weights=fmt)
    keep = torch.arange(M, device="cuda") != bad
    assert torch.equal(yi[keep].view(torch.int16), y[keep].view(torch.int16))
    assert not torch.isfinite(yi[bad]).any()
    if M > 16:
        want = torch.from_numpy(np.sign(w[:, k]) * sign * np.inf).cuda()
        assert torch.equal(yi[bad].double(), want)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("fmt", FORMATS)
def test_an_infinite_gradient(lib, M, fmt):
    rng = np.random.default_rng(M)
    N, K, n = 136, 320, 35
    qw, sw, zw = _weights(rng, N, K, fmt)
    qw[n, qw[n] == 0] = -2
    packed, w = C.pack(lib, torch, qw, sw, zw, fmt), C.real(qw, sw, zw)
    dy = _bf(rng.standard_normal((M, N)))
    dx, dxi = (torch.empty((M, K), dtype=BF, device="cuda") for _ in range(2))
    lib.qgemm_a16w4_bf16_grad_x(dy, packed, dx, weights=fmt)
    bad = M // 2
    dy[bad, n] = float("inf")
    lib.qgemm_a16w4_bf16_grad_x(dy, packed, dxi, weights=fmt)
    keep = torch.arange(M, device="cuda") != bad
    assert torch.equal(dxi[keep].view(torch.int16), dx[keep].view(torch.int16))
    assert torch.equal(dxi[bad].double(), torch.from_numpy(np.sign(w[n]) * np.inf).cuda())
