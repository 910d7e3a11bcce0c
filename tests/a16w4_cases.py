"""Inputs, references and tolerances of the weight-only int4 product tests.

bf16 values are handled as float32 arrays that hold bf16 values exactly.

Tolerance of one output y = sum_k x[k] w[k] + b, stored as bf16:
  - its last rounding: half a step, 2^-8 |y|;
  - the f32 sums: a group's dot product takes at most 32 additions in the
    tensor core (which may truncate: 2^-23 each, on partial sums of at most
    A_g = sum_{k in g} |x w|), the groups and K ranges at most K/32 + 16
    roundings of 2^-24, so at most (64 + K/32 + 16) * 2^-24 * A with
    A = sum_k |x w| + |b|;
  - where the kernel multiplies bf16 weights (many rows): every weight is
    rounded, off by at most 2^-8 |w|.  The errors of the K weights are
    independent of one another, so by Hoeffding's inequality their sum passes
    6.5 * 2^-8 * Q, Q = sqrt(sum_k (x w)^2), with a probability below 2e-9
    per output.  The sum of a weight's scale and zero parts is formed before
    that rounding;
  - where it multiplies codes (few rows) as c + 136 in sums that start at
    -136 X: the values of a group's sum stay below 280 sw sum |x|, and its 34
    additions are off by 2^-23 of that each, at most 0.0011 sw sum |x| in all.
    Over independent groups Hoeffding's 6.5 sigma is then, for |x| of one size,
    6.5 * 0.0011 * 32 * sqrt(K/32) sw |x| = 0.23 sqrt(K/32) sw |x|.  With codes
    spread evenly over [-8, 7], as here, the bf16 term above is
    6.5 * 2^-8 * 4.6 * sqrt(K) sw |x| = 0.66 sqrt(K/32) sw |x|: it stands for both.
"""
import numpy as np

import oracle


def bf16_round(a):
    """Nearest bf16 values (ties to even) of a float array, as float32."""
    b = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def weights(rng, N, K, fmt, E=None):
    """Codes, scales, zeros (or None); scales are bf16 values for "bf16"."""
    lead = () if E is None else (E,)
    qw = rng.integers(-8, 8, lead + (N, K)).astype(np.int8)
    sw = np.exp(rng.uniform(np.log(2e-3), np.log(2e-2), lead + (N, K // 32))).astype(np.float32)
    if fmt == "bf16":
        sw = bf16_round(sw)
    zw = None
    if fmt == "asym":
        zw = (sw * rng.integers(-3, 4, sw.shape)).astype(np.float32)
    return qw, sw, zw


def tolerance(x, w, ref, bias=None, rounded_weights=True):
    """Bound on |y - ref| for y = x @ w^T + bias (float64 arrays)."""
    K = w.shape[1]
    A = np.abs(x) @ np.abs(w).T + (0.0 if bias is None else np.abs(bias))
    inner = (64 + K / 32 + 16) * 2.0 ** -24 * A
    if rounded_weights:
        inner = inner + 6.5 * 2.0 ** -8 * np.sqrt((x * x) @ (w * w).T)
    return inner + 2.0 ** -8 * (np.abs(ref) + inner) + 1e-30


def assert_close(y, ref, tol, label=""):
    err = np.abs(y.astype(np.float64) - ref)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, err / tol, 0))), err.shape)
        raise AssertionError(f"{label}: {bad.sum()} of {bad.size} off; at {i}: {y[i]} vs {ref[i]}, "
                             f"tolerance {tol[i]}")


def pack(lib, torch, qw, sw, zw, fmt):
    """The packed matrix on the GPU, by the library's own packing."""
    q, s = torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda()
    if fmt == "asym":
        return lib.pack_w4_g32_asym(q, s, torch.from_numpy(zw).cuda())
    return lib.pack_w4_g32_bf16(q, s) if fmt == "bf16" else lib.pack_w4_g32(q, s)


def pack_experts(lib, torch, qw, sw, zw, fmt, gap=0):
    """[E][bytes]: the experts' packed matrices, `gap` bytes (a multiple of 16) apart."""
    parts = [pack(lib, torch, qw[e], sw[e], None if zw is None else zw[e], fmt)
             for e in range(qw.shape[0])]
    n = -(-parts[0].numel() // 16) * 16
    out = torch.full((len(parts), n + gap), 0xFF, dtype=torch.uint8, device="cuda")
    for e, p in enumerate(parts):
        out[e, :p.numel()] = p
    return out


def routing(rng, T, topk, E, drop=0.0, hot=None):
    """Expert ids [T][topk] (distinct per token), some tokens without any;
    `hot`: every token also picks expert `hot` first."""
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :topk].astype(np.int32)
    if hot is not None:
        ids[:, 0] = hot
    ids[rng.random(T) < drop] = -1
    return ids


def real(qw, sw, zw):
    return oracle.w4_values(qw, sw, zw)


def integer_rows(rng, M, K):
    """Rows of whole numbers in [-8, 8], bf16 values exactly."""
    return rng.integers(-8, 9, (M, K)).astype(np.float32)


def exact_codes_tolerance(x, qw, sw, zw, ref, bias=None):
    """Bound on |y - ref| where the codes are used exactly (few rows) and x are
    integer_rows.  A group's products (c + 136) x and its -136 X are whole
    numbers whose sums stay below 32 * 8 * (143 + 136) < 2^24, so the group's sum
    is exact in f32 in whatever order.  What is rounded, by 2^-24 of at most
    A = sum |sw c x| + sum |zw x| + |b| each time: the product with sw in its sum,
    the factor -1/136, its product with zw and that one's sum (four a group),
    the sum of eight warps and the bias.  Then half a step of the output."""
    A = np.abs(x) @ np.abs(real(qw, sw, None)).T + (0.0 if bias is None else np.abs(bias))
    if zw is not None:
        A = A + np.abs(x) @ np.repeat(np.abs(zw.astype(np.float64)), 32, axis=1).T
    inner = (4 * (qw.shape[1] // 32) + 9) * 2.0 ** -24 * A
    return inner + 2.0 ** -8 * (np.abs(ref) + inner) + 1e-30
