"""Host-only checks of the weight-only int4 products and the expert order: the
arguments each call refuses, before it touches the device.  Every address
below is made up, so every call has to return before a launch."""
import pytest

qg = pytest.importorskip("gemv_zero_point_b200")
torch = pytest.importorskip("torch")
lib = qg.lib

A = 1 << 20  # an address of any alignment asked for here
INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = -1, -2, -4, -7


def linear(M=4, N=8, K=64, x=A, ldx=64, w=A, fmt=0, bias=None, y=A, ldy=8):
    return lib.qgemm_a16w4_bf16(M, N, K, x, ldx, w, fmt, bias, y, ldy, None)


def linear_grad(M=4, N=8, K=64, dy=A, lddy=8, w=A, fmt=0, dx=A, lddx=64):
    return lib.qgemm_a16w4_bf16_grad_x(M, N, K, dy, lddy, w, fmt, dx, lddx, None)


def experts(E=2, S=4, N=8, K=64, x=A, ldx=64, x_rows=4, src=None, topk=1, offsets=A, w=A, step=4096,
            fmt=0, bias=None, y=A, ldy=8, ws=None, ws_bytes=0):
    return lib.qgemm_a16w4_bf16_experts(E, S, N, K, x, ldx, x_rows, src, topk, offsets, w, step, fmt,
                                        bias, y, ldy, ws, ws_bytes, None)


def experts_grad(E=2, S=4, N=8, K=64, dy=A, lddy=8, offsets=A, w=A, step=4096, fmt=0, dx=A, lddx=64):
    return lib.qgemm_a16w4_bf16_experts_grad_x(E, S, N, K, dy, lddy, offsets, w, step, fmt, dx, lddx,
                                               None)


def sort(T=4, topk=2, E=8, ids=A, ld=2, offsets=A, src=A, pos=A, ws=None, ws_bytes=0):
    return lib.qg_sort_by_expert(T, topk, E, ids, ld, offsets, src, pos, ws, ws_bytes, None)


def spread(T=4, topk=2, S=8, N=16, dtype=1, x=A, ldx=16, pos=A, xs=A, ldxs=16):
    return lib.qg_spread_rows(T, topk, S, N, dtype, x, ldx, pos, xs, ldxs, None)


def combine(T=4, topk=2, S=8, N=16, dtype=1, ys=A, ldys=16, pos=A, weights=None, y=A, ldy=16):
    return lib.qg_combine_rows(T, topk, S, N, dtype, ys, ldys, pos, weights, y, ldy, None)


def combine_grad(T=4, topk=2, S=8, N=16, dtype=1, dy=A, lddy=16, ys=A, ldys=16, pos=A, weights=None,
                 dys=A, lddys=16, dw=A):
    return lib.qg_combine_rows_grad(T, topk, S, N, dtype, dy, lddy, ys, ldys, pos, weights, dys, lddys,
                                    dw, None)


def test_products_refuse_bad_sizes_and_strides():
    for call, in_ld, out_ld in [(linear, "ldx", "ldy"), (linear_grad, "lddy", "lddx"),
                                (experts, "ldx", "ldy"), (experts_grad, "lddy", "lddx")]:
        for bad in [{"N": 0}, {"K": 0}, {"K": -64}, {"fmt": 3}, {"fmt": -1}, {in_ld: 0}, {out_ld: 0},
                    {in_ld: -8}]:
            assert call(**bad) == INVALID, (call.__name__, bad)
        rows = "M" if call in (linear, linear_grad) else "S"
        assert call(**{rows: -1}) == INVALID
        wide = {"K": 96, in_ld: 4096, out_ld: 4096}
        assert call(**wide) == UNSUPPORTED          # K % 64
        side = (1 << 24) + 64
        big = {in_ld: side, out_ld: side}
        assert call(**big, K=side) == UNSUPPORTED
        assert call(**big, N=side) == UNSUPPORTED
        assert call(**{in_ld: 4100, out_ld: 4096}) == MISALIGNED  # rows of 16 bytes
    for call in (experts, experts_grad):
        assert call(E=0) == INVALID and call(E=1025) == UNSUPPORTED
        assert call(step=8 * 32 + 8 * 2 * 4 - 16) == INVALID    # matrices overlap
        assert call(step=4104) == MISALIGNED
        assert call(offsets=None) == INVALID and call(offsets=A + 2) == MISALIGNED
    assert experts(topk=0) == INVALID and experts(x_rows=-1) == INVALID
    assert experts(x_rows=3) == INVALID             # rows in place, fewer than S
    assert experts(x_rows=0, src=A) == INVALID
    assert experts(src=A + 2) == MISALIGNED


def test_products_refuse_missing_and_misaligned_pointers():
    for call, ins, out in [(linear, "x", "y"), (linear_grad, "dy", "dx"), (experts, "x", "y"),
                           (experts_grad, "dy", "dx")]:
        for name in (ins, "w", out):
            assert call(**{name: None}) == INVALID, (call.__name__, name)
        assert call(**{ins: A + 8}) == MISALIGNED
        assert call(w=A + 8) == MISALIGNED
        assert call(**{out: A + 1}) == MISALIGNED
    assert linear(bias=A + 2) == MISALIGNED and experts(bias=A + 1) == MISALIGNED


def test_products_without_rows_do_nothing():
    assert linear(M=0, x=None, w=None, y=None) == 0
    assert linear_grad(M=0, dy=None, w=None, dx=None) == 0
    assert experts(S=0, x=None, w=None, y=None, offsets=None, x_rows=0) == 0
    assert experts_grad(S=0, dy=None, w=None, dx=None, offsets=None) == 0


def test_workspaces():
    ws = lib.qgemm_a16w4_bf16_experts_workspace_bytes
    # a few rows per expert, or rows in place: none; otherwise the sorted rows
    assert ws(64, 64, 256, 1) == 0 and ws(2, 4096, 256, 0) == 0
    assert ws(2, 4096, 256, 1) == 4096 * 256 * 2
    assert ws(0, 4096, 256, 1) == 0 and ws(2, 4096, 100, 1) == 0 and ws(2, -1, 256, 1) == 0
    many = dict(S=4096, src=A, x_rows=4096)
    need = ws(2, 4096, 64, 1)
    assert experts(**many) == WORKSPACE
    assert experts(**many, ws=A, ws_bytes=need - 1) == WORKSPACE
    assert experts(**many, ws=None, ws_bytes=need) == WORKSPACE
    assert experts(**many, ws=A + 128, ws_bytes=need) == MISALIGNED
    sb = lib.qg_sort_by_expert_workspace_bytes
    assert sb(8, 8, 64) == 0 and sb(256, 8, 64) == 0
    assert sb(257, 8, 64) == 3 * 64 * 4              # chunks of 1024 entries
    assert sb(4097, 8, 64) == 17 * 64 * 4            # of 2048
    assert sb(16385, 8, 64) == 33 * 64 * 4           # of 4096
    assert sb(0, 8, 64) == 0 and sb(8, 8, 1025) == 0 and sb(1 << 22, 2, 4) == 0
    assert sort(T=257, topk=8, ld=8, E=64) == WORKSPACE
    assert sort(T=257, topk=8, ld=8, E=64, ws=A, ws_bytes=3 * 64 * 4 - 1) == WORKSPACE
    assert sort(T=257, topk=8, ld=8, E=64, ws=A + 2, ws_bytes=4096) == MISALIGNED


def test_sort_refusals():
    for bad in [{"T": -1}, {"topk": 0}, {"E": 0}, {"ld": 1}, {"offsets": None}, {"ids": None},
                {"src": None}, {"pos": None}]:
        assert sort(**bad) == INVALID, bad
    assert sort(E=1025) == UNSUPPORTED and sort(T=1 << 22, topk=2) == UNSUPPORTED
    for name in ("ids", "offsets", "src", "pos"):
        assert sort(**{name: A + 2}) == MISALIGNED


def test_row_call_refusals():
    for call in (spread, combine, combine_grad):
        for bad in [{"T": -1}, {"topk": 0}, {"S": -1}, {"N": 0}, {"dtype": 3}, {"dtype": -1},
                    {"pos": None}]:
            assert call(**bad) == INVALID, (call.__name__, bad)
        assert call(T=1 << 30, topk=2) == UNSUPPORTED
        assert call(pos=A + 2) == MISALIGNED
    assert spread(ldx=15) == INVALID and spread(ldxs=15) == INVALID
    assert spread(x=None) == INVALID and spread(xs=None) == INVALID
    assert spread(x=A + 1) == MISALIGNED and spread(dtype=0, xs=A + 2) == MISALIGNED
    assert spread(T=0, x=None, pos=None) == 0 and spread(S=0, xs=None) == 0
    assert combine(ldys=15) == INVALID and combine(ldy=15) == INVALID
    assert combine(ys=None) == INVALID and combine(y=None) == INVALID
    assert combine(y=A + 1) == MISALIGNED and combine(weights=A + 2) == MISALIGNED
    assert combine(T=0, ys=None, pos=None, y=None) == 0
    assert combine_grad(dys=None, dw=None) == INVALID      # nothing asked for
    assert combine_grad(ys=None) == INVALID and combine_grad(dy=None) == INVALID
    assert combine_grad(lddy=15) == INVALID and combine_grad(ldys=15) == INVALID
    assert combine_grad(lddys=15) == INVALID
    assert combine_grad(dw=A + 2) == MISALIGNED and combine_grad(dys=A + 1) == MISALIGNED
    assert combine_grad(T=0, dy=None, ys=None, pos=None) == 0


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("call", [
    lambda: qg.qgemm_a16w4_bf16(bf(2, 64), u8(320), bf(2, 8)),                         # not on a GPU
    lambda: qg.qgemm_a16w4_bf16(bf(2, 64).float(), u8(320), bf(2, 8)),
    lambda: qg.qgemm_a16w4_bf16(bf(2, 64), u8(319), bf(2, 8)),                         # too short
    lambda: qg.qgemm_a16w4_bf16(bf(2, 64), u8(320), bf(3, 8)),
    lambda: qg.qgemm_a16w4_bf16(bf(64, 2).t(), u8(320), bf(2, 8)),                     # column-major
    lambda: qg.qgemm_a16w4_bf16(bf(2, 64), u8(320), bf(2, 8), weights="int4"),
    lambda: qg.qgemm_a16w4_bf16(bf(2, 64), u8(320), bf(2, 8), bias=torch.zeros(7)),
    lambda: qg.qgemm_a16w4_bf16_grad_x(bf(2, 8), u8(320), bf(3, 64)),
    lambda: qg.qgemm_a16w4_bf16_experts(bf(2, 64), i32(3), u8(1, 320), bf(2, 8)),      # E + 1 offsets
    lambda: qg.qgemm_a16w4_bf16_experts(bf(2, 64), i32(3), u8(640), bf(2, 8)),
    lambda: qg.qgemm_a16w4_bf16_experts(bf(2, 64), i32(3), u8(2, 320), bf(2, 8), src=i32(1)),
    lambda: qg.qgemm_a16w4_bf16_experts(bf(2, 64), i32(3), u8(2, 320), bf(2, 8),
                                        workspace=u8(1).expand(1 << 20)),
    lambda: qg.qgemm_a16w4_bf16_experts_grad_x(bf(2, 8), i32(2), u8(2, 320), bf(2, 64)),
    lambda: qg.qg_sort_by_expert(i32(4, 2), i32(9), i32(7), i32(4, 2)),
    lambda: qg.qg_sort_by_expert(i32(4, 2).long(), i32(9), i32(8), i32(4, 2)),
    lambda: qg.qg_spread_rows(bf(4, 16), i32(4, 2), bf(8, 17)),
    lambda: qg.qg_spread_rows(bf(4, 16), i32(3, 2), bf(8, 16)),
    lambda: qg.qg_spread_rows(bf(4, 16).long(), i32(4, 2), bf(8, 16)),
    lambda: qg.qg_combine_rows(bf(8, 16), i32(4, 2), bf(4, 16).float()),
    lambda: qg.qg_combine_rows(bf(8, 16), i32(4, 2), bf(4, 16), weights=torch.zeros(4, 3)),
    lambda: qg.qg_combine_rows_grad(bf(4, 16), None, i32(4, 2), None, None, torch.zeros(4, 2)),
    lambda: qg.qg_combine_rows_grad(bf(4, 16), bf(8, 16), i32(4, 2), None, bf(9, 16), None),
])
def test_bindings_refuse(call):
    with pytest.raises(ValueError):
        call()
