"""Indirect rows of experts whose offsets are wrong in places: the experts with
a range of their own get all of its rows, whatever the other offsets say."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16
S, TOPK, N, K = 240, 2, 72, 128
# (offsets, the experts that have their range)
OFFSETS = [([140, 120, 240], [1]), ([0, 240, 100], [0]), ([0, 120, -1], [0]), ([-1, 120, 240], [1]),
           ([0, 120, 241], [0]), ([240, 120, 240], [1]), ([300, 0, 100, 900, 240], [1]),
           ([2 ** 31 - 1, -2 ** 31, 7, 239, -2 ** 31], [2]), ([240, 240, 0], [0]),
           ([3, 100, 200], [0, 1]), ([0, 0, 240], [0, 1]), ([0, 240, 240], [0, 1])]


@pytest.mark.parametrize("offsets,good", OFFSETS)
@pytest.mark.parametrize("rows", ["few", "many"])
def test_every_right_range_gets_its_rows(lib, cuda, offsets, good, rows):
    """`few`: enough experts without rows that the other kernel takes the call."""
    rng = np.random.default_rng(len(offsets) + S)
    E = len(offsets) - 1
    if rows == "few":
        offsets = offsets + offsets[-1:] * (60 - E)
        E = 60
    qw, sw, zw = C.weights(rng, N, K, "f32", E)
    packed, w = C.pack_experts(lib, torch, qw, sw, zw, "f32"), C.real(qw, sw, zw)
    x = C.bf16_round(rng.standard_normal((S // TOPK, K)))
    src = rng.permutation(S).astype(np.int32)
    own = np.zeros(S, bool)      # rows of the ranges that hold
    rights = [e for e in range(E) if 0 <= offsets[e] <= offsets[e + 1] <= S]
    for e in rights:
        own[offsets[e]:offsets[e + 1]] = True
    assert set(good) <= set(rights)
    all_right = len(rights) == E
    if all_right:                # nobody's entries are not even looked at
        src[~own] = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, S], (~own).sum())
    need = lib.lib.qgemm_a16w4_bf16_experts_workspace_bytes(E, S, K, 1)
    assert (need > 0) == (rows == "many")
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN as bf16
    y = torch.full((S, N), 7.0, dtype=BF, device="cuda")
    lib.qg_device_status(True)
    lib.qgemm_a16w4_bf16_experts(torch.from_numpy(x).cuda().to(BF), torch.tensor(offsets, dtype=torch.int32,
                                 device="cuda"), packed, y, src=torch.from_numpy(src).cuda(), topk=TOPK,
                                 workspace=ws)
    assert lib.qg_device_status(True) == (0 if all_right else -1)
    y = y.double().cpu().numpy()
    for e in rights:
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            rows_e = x[src[a:b] // TOPK]
            ref = oracle.a16w4(rows_e, w[e])
            C.assert_close(y[a:b], ref, C.tolerance(rows_e.astype(np.float64), w[e], ref), f"expert {e}")
    assert (y[~own] == 7.0).all()
