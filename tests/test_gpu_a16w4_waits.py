"""The bounded waits of the many-row int4 kernel count its own time only."""
import numpy as np
import pytest

import a16w4_cases as C

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


# many stages of the reduction for each CTA: one tile per CTA, its reduction
# shared by a cluster, CTA pairs
@pytest.mark.parametrize("M,N,K", [(200, 256, 8192), (200, 14336, 4096), (600, 2304, 1024)])
@pytest.mark.parametrize("grad", [False, True])
def test_many_stages_behind_long_work(lib, cuda, M, N, K, grad):
    """Behind calls that keep one SM busy for some 0.2 s, longer than a bounded
    wait lasts, on the other SMs: every wait for the call's own copies starts to
    count once that work has ended."""
    rng = np.random.default_rng(M)
    if grad:
        N, K = K, N
    qw, sw, zw = C.weights(rng, N, K, "f32")
    packed = C.pack(lib, torch, qw, sw, zw, "f32")
    rows = torch.from_numpy(rng.standard_normal((M, N if grad else K)).astype(np.float32)).cuda().to(BF)
    call = lib.qgemm_a16w4_bf16_grad_x if grad else lib.qgemm_a16w4_bf16
    want = torch.empty((M, K if grad else N), dtype=BF, device="cuda")
    lib.qg_device_status(True)
    call(rows, packed, want)
    n, topk = 1 << 29, 8
    dy = torch.ones((1, n), dtype=BF, device="cuda")
    ys = torch.ones((topk, n), dtype=BF, device="cuda")
    pos = torch.arange(topk, dtype=torch.int32, device="cuda").reshape(1, topk)
    dw = torch.empty((1, topk), device="cuda")
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    for _ in range(2):
        lib.qg_combine_rows_grad(dy, ys, pos, None, None, dw)
    call(rows, packed, out)
    assert lib.qg_device_status(True) == 0
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
