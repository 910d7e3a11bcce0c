"""The weight-only int4 products at the longest sides that the header allows,
as a reduction and as features, with one row, a few and some more."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16
SIDE = 1 << 24


def _matrix(N, K):
    """A packed matrix of f32 group scales, and its codes and scales."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    u = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand((N, K // 32), generator=g, device="cuda") * 0.01 + 0.002
    b = u.view(N, K // 8, 4)
    codes = torch.cat([b & 15, b >> 4], -1).view(N, K).to(torch.int8) - 8
    return torch.cat([u.view(-1), s.view(torch.uint8).view(-1)]), codes, s


def _sums(rows, codes, s, grad):
    """rows @ W^T (or rows @ W) in 64 bits, with the sums of the squares of the
    terms and of their absolute values, a part of the long side at a time."""
    N, K = codes.shape
    out = [torch.zeros((rows.shape[0], K if grad else N), dtype=torch.float64, device="cuda") for _ in range(3)]
    parts = max(1, N * K >> 26)
    for p in range(parts):
        if N > K:
            a, b = N * p // parts, N * (p + 1) // parts
            w = codes[a:b].double() * s[a:b].double().repeat_interleave(32, 1)
            r, to = (rows[:, a:b], slice(None)) if grad else (rows, slice(a, b))
        else:
            a, b = K // 32 * p // parts * 32, K // 32 * (p + 1) // parts * 32
            w = codes[:, a:b].double() * s[:, a // 32:b // 32].double().repeat_interleave(32, 1)
            r, to = (rows, slice(a, b)) if grad else (rows[:, a:b], slice(None))
        w, r = (w if grad else w.T), r.double()
        out[0][:, to] += r @ w
        out[1][:, to] += (r * r) @ (w * w)
        out[2][:, to] += r.abs() @ w.abs()
    return out


def _assert_close(y, rows, codes, s, grad=False):
    """Rounded weights 6.5 * 2^-8 Q (a16w4_cases), and the f32 sums of the tensor
    cores over R.  A step adds 16 products to the sum and cuts off what lies below
    the sum's last place, 2^-23 of it: towards zero, so these errors add up to
    R/16 * 2^-23 P where P bounds the partial sums.  The products, aligned to the
    sum, are cut too, but by their own random signs: 6.5 sigma of R such errors is
    6.5 sqrt(R) 2^-23 P.  Partial sums of independent terms pass P = 6.5 Q no
    more often than twice the whole sum does (Levy's inequality), below 4e-9.
    The few-row kernel adds its groups by rounded f32 steps, which is less."""
    ref, sq, _ = _sums(rows, codes, s, grad)
    R, Q = rows.shape[1], sq.sqrt()
    inner = 6.5 * 2.0 ** -8 * Q + (R / 16 + 6.5 * R ** 0.5) * 2.0 ** -23 * 6.5 * Q
    assert ((y.double() - ref).abs() <= inner + 2.0 ** -8 * (ref.abs() + inner) + 1e-30).all()


@pytest.mark.parametrize("M", [1, 16, 20])
@pytest.mark.parametrize("N,K", [(3, SIDE), (SIDE, 64)])
@pytest.mark.parametrize("grad", [False, True])
def test_longest_sides(lib, cuda, M, N, K, grad):
    if grad and N == 3:
        N = 8                       # rows of dy in whole 16 bytes
    lib.qg_device_status(True)
    packed, codes, s = _matrix(N, K)
    g = torch.Generator(device="cuda").manual_seed(M)
    rows = torch.randn((M, N if grad else K), generator=g, device="cuda").to(BF)
    out = torch.empty((M, K if grad else N), dtype=BF, device="cuda")
    (lib.qgemm_a16w4_bf16_grad_x if grad else lib.qgemm_a16w4_bf16)(rows, packed, out)
    assert lib.qg_device_status(True) == 0
    _assert_close(out, rows, codes, s, grad)


@pytest.mark.parametrize("E,S", [(1, 20), (2, 40)])
def test_longest_reduction_per_expert(lib, cuda, E, S):
    """No shared reduction here: one CTA takes all of it, within its waits."""
    lib.qg_device_status(True)
    one, codes, s = _matrix(2, SIDE)
    packed = one.repeat(E, 1)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (S // E)
    x = torch.randn((S, SIDE), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF)
    y = torch.empty((S, 2), dtype=BF, device="cuda")
    lib.qgemm_a16w4_bf16_experts(x, off, packed, y)
    assert lib.qg_device_status(True) == 0
    _assert_close(y, x, codes, s)


@pytest.mark.parametrize("M", [1, 16, 20, 150])
@pytest.mark.parametrize("N,K", [(8, SIDE), (SIDE, 64)])
@pytest.mark.parametrize("grad", [False, True])
def test_longest_sides_exactly(lib, cuda, M, N, K, grad):
    """Rows of -1, 0 and 1 and scales of 2^-6: every sum on the way is a whole
    number of 2^-6 below 2^24 of them, exact in f32, so the result is the exact
    sum's nearest bf16 value."""
    if M == 150 and K == SIDE and not grad or M == 150 and N == SIDE and grad:
        M = 40                      # rows of 32 MB
    lib.qg_device_status(True)
    packed, codes, s = _matrix(N, K)
    s.fill_(2.0 ** -6)
    packed[N * K // 2:] = s.view(torch.uint8).view(-1)
    g = torch.Generator(device="cuda").manual_seed(M)
    rows = torch.randint(-1, 2, (M, N if grad else K), generator=g, device="cuda").to(BF)
    out = torch.empty((M, K if grad else N), dtype=BF, device="cuda")
    (lib.qgemm_a16w4_bf16_grad_x if grad else lib.qgemm_a16w4_bf16)(rows, packed, out)
    assert lib.qg_device_status(True) == 0
    ref = _sums(rows, codes, s, grad)[0]
    assert float(ref.abs().max()) < 2.0 ** 17  # far from 2^18: partial sums too
    assert torch.equal(out, ref.to(BF))
