"""The bounded-wait path of the many-row int4 kernel, without a fault.

qg_test_arm_stall(3) makes the next launch of that kernel ask for no rows for a
CTA's second stage, and gives its waits a short limit.  The wait for that stage
runs out; the kernel records QG_ERR_TIMEOUT, waits for the copies and MMAs it
has in flight, frees its tensor memory and returns.  The next call is an
ordinary one with the bits of a call before."""
import numpy as np
import pytest

import a16w4_cases as C

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16
TIMEOUT = -6


def _rows(rng, M, K):
    return torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda().to(BF)


def _run(lib, call, out):
    """Stalled once, then as before."""
    lib.qg_device_status(True)
    call()
    assert lib.qg_device_status(True) == 0
    want = out.clone()
    for _ in range(2):
        lib.qg_test_arm_stall(3)
        call()
        assert lib.qg_device_status(True) == TIMEOUT
        out.zero_()
        call()
        assert lib.qg_device_status(True) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


# CTAs on their own, a reduction shared by clusters of 2 and 8, CTA pairs of two
# stages, and of more with one tile each and with several
@pytest.mark.parametrize("M,N,K", [(200, 300, 320), (64, 256, 512), (64, 256, 4096), (17, 20000, 256),
                                   (300, 14336, 512), (600, 14336, 1024)])
@pytest.mark.parametrize("grad", [False, True])
def test_dense_stalled_then_ordinary(lib, cuda, M, N, K, grad):
    rng = np.random.default_rng(M + N)
    if grad:
        N, K = -(-K // 8) * 8, -(-N // 64) * 64
    qw, sw, zw = C.weights(rng, N, K, "bf16")
    packed = C.pack(lib, torch, qw, sw, zw, "bf16")
    if grad:
        dy, dx = _rows(rng, M, N), torch.empty((M, K), dtype=BF, device="cuda")
        _run(lib, lambda: lib.qgemm_a16w4_bf16_grad_x(dy, packed, dx, weights="bf16"), dx)
    else:
        x, y = _rows(rng, M, K), torch.empty((M, N), dtype=BF, device="cuda")
        _run(lib, lambda: lib.qgemm_a16w4_bf16(x, packed, y, weights="bf16"), y)


# single CTAs and pairs, rows that are gathered first
@pytest.mark.parametrize("N,K", [(136, 512), (4096, 384)])
@pytest.mark.parametrize("grad", [False, True])
def test_experts_stalled_then_ordinary(lib, cuda, N, K, grad):
    rng = np.random.default_rng(N)
    E, S = 4, 600
    if grad:
        N, K = K, -(-N // 64) * 64
    qw, sw, zw = C.weights(rng, N, K, "asym", E)
    packed = C.pack_experts(lib, torch, qw, sw, zw, "asym")
    off = torch.tensor([0, 7, 300, 300, S], dtype=torch.int32, device="cuda")
    rows = _rows(rng, S, N if grad else K)
    out = torch.empty((S, K if grad else N), dtype=BF, device="cuda")
    if grad:
        _run(lib, lambda: lib.qgemm_a16w4_bf16_experts_grad_x(rows, off, packed, out, weights="asym"), out)
    else:
        src = torch.from_numpy(rng.permutation(S).astype(np.int32)).cuda()
        _run(lib, lambda: lib.qgemm_a16w4_bf16_experts(rows, off, packed, out, src=src, topk=1,
                                                       weights="asym"), out)


def test_the_other_kernels_leave_the_stall_armed(lib, cuda):
    """Few rows take another kernel: nothing stalls until the one armed runs."""
    rng = np.random.default_rng(1)
    qw, sw, zw = C.weights(rng, 256, 512, "f32")
    packed = C.pack(lib, torch, qw, sw, zw, "f32")
    x, y = _rows(rng, 64, 512), torch.empty((64, 256), dtype=BF, device="cuda")
    lib.qg_device_status(True)
    lib.qg_test_arm_stall(3)
    lib.qgemm_a16w4_bf16(x[:4], packed, y[:4])
    assert lib.qg_device_status(True) == 0
    lib.qgemm_a16w4_bf16(x, packed, y)
    assert lib.qg_device_status(True) == TIMEOUT
    lib.qgemm_a16w4_bf16(x, packed, y)
    assert lib.qg_device_status(True) == 0
