"""Cases of the weight-only int4 products, the per-expert products and the
expert ordering of tokens, with their plain forms.

Kinds of case (``case["op"]``):
  linear        y = x @ W^T + bias, x bf16, W int4 in groups of 32 along K
  linear_grad   dx = dy @ W
  experts       y[p] = x[src[p] / topk] @ W[e]^T + bias[e] for the rows of expert e
  experts_grad  dx[p] = dy[p] @ W[e]
  dispatch      expert ids -> stable order by expert, and the token rows in that order
  combine       y[t] = sum_j weights[t, j] * ys[pos[t, j]]
  combine_grad  the gradients of that sum with respect to ys and weights

``weights`` is the packing of the int4 codes: "f32" or "bf16" group scales, or
"asym" (f32 scales and f32 zeros).  A packed matrix is N rows of K/2 bytes,
where the little-endian 32-bit word j of a row holds code 8j+b (offset by 8)
in the low nibble and code 8j+4+b in the high nibble of byte b, followed by
the scales [N][K/32] and, for "asym", the zeros [N][K/32].  The packed
matrices of several experts follow one another.
"""
import math

import torch

own = False

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _linear(op, M, N, K, weights, bias=False):
    return {"op": op, "M": M, "N": N, "K": K, "weights": weights, "bias": bias}


def _experts(op, T, topk, E, N, K, weights, skew=0.5, drop=0.0, bias=False):
    return {"op": op, "T": T, "topk": topk, "E": E, "N": N, "K": K, "weights": weights,
            "skew": skew, "drop": drop, "bias": bias}


def _rows(op, T, topk, E, N, dtype, skew=0.5, drop=0.0):
    return {"op": op, "T": T, "topk": topk, "E": E, "N": N, "dtype": dtype, "skew": skew,
            "drop": drop}


def listed():
    return [
        # one generated token through a projection: the latency of a serving step
        dict(_linear("linear", 1, 14336, 4096, "f32"), name="linear_one_token"),
        # a step of a dozen sequences served together, the projection back
        dict(_linear("linear", 12, 4096, 14336, "bf16"), name="linear_few_tokens"),
        # a short ragged batch on a small matrix with odd sizes
        dict(_linear("linear", 77, 1000, 832, "asym", bias=True), name="linear_ragged"),
        # a long prompt
        dict(_linear("linear", 4096, 14336, 4096, "bf16"), name="linear_prompt"),
        # input gradient of a frozen projection: a training batch
        dict(_linear("linear_grad", 2048, 4096, 4096, "f32"), name="linear_grad_batch"),
        # one step of eight sequences through a layer of experts
        dict(_experts("experts", 8, 8, 64, 2048, 2048, "bf16"), name="experts_one_step"),
        # a prompt through a layer of experts
        dict(_experts("experts", 4096, 8, 64, 1536, 2048, "f32", bias=True),
             name="experts_prompt"),
        # input gradient of the experts, uneven routing, padding tokens left out
        dict(_experts("experts_grad", 1111, 4, 16, 2048, 1408, "asym", skew=1.0, drop=0.1),
             name="experts_grad_uneven"),
        # ordering the tokens of one serving step
        dict(_rows("dispatch", 16, 8, 128, 4096, "bf16"), name="dispatch_one_step"),
        # ordering a long prompt, with its rows
        dict(_rows("dispatch", 8192, 8, 128, 4096, "bf16"), name="dispatch_prompt"),
        # a long prompt back in token order, padding tokens left out
        dict(_rows("combine", 8192, 8, 128, 4096, "bf16", drop=0.1), name="combine_prompt"),
        # gradient of that sum in a training step kept in 32 bits
        dict(_rows("combine_grad", 4099, 6, 64, 2056, "f32", skew=1.0), name="combine_grad_f32"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "linear_grad", "experts", "experts",
                     "experts_grad", "dispatch", "combine", "combine_grad"])
    if op.startswith("linear"):
        N = _log_int(rng, 1000, 16384)
        if op == "linear_grad" or rng.random() < 0.5:
            N = max(64, N // 64 * 64)
        if op == "linear_grad":
            N = max(64, N // 8 * 8)
        K = _log_int(rng, 512, 16384, 64)
        M = _log_int(rng, 1, 4096)
        while M * N * K > 4096 * 14336 * 4096:
            M = max(1, M // 2)
        return _linear(op, M, N, K, rng.choice(["f32", "bf16", "asym"]), rng.random() < 0.5
                       and op == "linear")
    T = _log_int(rng, 1, 8192)
    topk = rng.choice([1, 2, 4, 6, 8])
    E = rng.choice([8, 16, 60, 64, 128, 160, 256])
    skew, drop = rng.choice([0.0, 0.5, 1.0]), rng.choice([0.0, 0.0, 0.1, 0.4])
    if op.startswith("experts"):
        E = min(E, 128)
        N = _log_int(rng, 512, 4096, 8)
        K = _log_int(rng, 512, 4096, 64)
        while E * N * K > 64 * 2048 * 4096:
            E = max(8, E // 2)
        while T > 1 and T * topk * N * K > 4096 * 8 * 2048 * 2048:
            T = max(1, T // 2)
        return _experts(op, T, topk, E, N, K, rng.choice(["f32", "bf16", "asym"]), skew, drop,
                        rng.random() < 0.5 and op == "experts")
    N = _log_int(rng, 512, 8192, rng.choice([1, 8, 64]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while T > 1 and T * topk * N * (4 if dtype == "f32" else 2) > 8192 * 8 * 4096 * 2:
        T = max(1, T // 2)
    return _rows(op, T, topk, E, N, dtype, skew, drop)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _weights(g, E, N, K, kind):
    """Codes in [-8, 7], scales and zeros of E matrices, as values."""
    codes = torch.randint(-8, 8, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    u = torch.rand((E, N, K // GROUP), generator=g, device="cuda")
    scales = torch.exp(math.log(2e-3) + u * math.log(10.0))
    if kind == "bf16":
        scales = scales.to(torch.bfloat16).float()
    zeros = None
    if kind == "asym":
        zeros = scales * torch.randint(-3, 4, scales.shape, generator=g, device="cuda")
    return codes, scales, zeros


def _pack(codes, scales, zeros, kind):
    E, N, K = codes.shape
    u = (codes + 8).to(torch.uint8).view(E, N, K // 8, 8)
    parts = [(u[..., :4] | (u[..., 4:] << 4)).reshape(E, -1)]
    stored = scales.to(torch.bfloat16) if kind == "bf16" else scales
    parts.append(stored.contiguous().view(torch.uint8).reshape(E, -1))
    if zeros is not None:
        parts.append(zeros.contiguous().view(torch.uint8).reshape(E, -1))
    out = torch.cat(parts, 1)
    pad = -out.shape[1] % 256  # every expert's matrix starts on 256 bytes
    return torch.nn.functional.pad(out, (0, pad)).contiguous()


def _routing(g, c):
    """Expert ids [T, topk] (-1: no expert) and routing weights [T, topk]."""
    T, topk, E = c["T"], c["topk"], c["E"]
    scores = torch.randn((T, E), generator=g, device="cuda")
    scores = scores + c["skew"] * torch.randn((1, E), generator=g, device="cuda")
    best, ids = torch.topk(scores, topk, dim=1)
    gone = torch.rand((T, 1), generator=g, device="cuda") < c["drop"]
    ids = torch.where(gone, -1, ids).to(torch.int32)
    return ids, torch.softmax(best, 1)


def _order(ids, E):
    """Stable order by expert: offsets [E+1], src [T*topk], pos [T, topk]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    edges = torch.arange(E + 1, device=ids.device)
    offsets = torch.searchsorted(key[order].contiguous(), edges).to(torch.int32)
    at = torch.arange(flat.numel(), device=ids.device)
    live = at < offsets[E]
    src = torch.where(live, order, -1).to(torch.int32)
    pos = torch.empty_like(src)
    pos[order] = torch.where(live, at, -1).to(torch.int32)
    return offsets, src, pos.view(ids.shape)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    op = c["op"]
    if op.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        s["packed"] = _pack(*_weights(g, 1, N, K, c["weights"]), c["weights"]).view(-1)
        if op == "linear":
            s["x"] = torch.randn((M, K), generator=g, device="cuda").bfloat16()
            s["bias"] = torch.randn(N, generator=g, device="cuda") if c["bias"] else None
            s["y"] = torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
        else:
            s["dy"] = torch.randn((M, N), generator=g, device="cuda").bfloat16()
            s["dx"] = torch.empty((M, K), device="cuda", dtype=torch.bfloat16)
        return s
    ids, weights = _routing(g, c)
    T, topk, E, N = c["T"], c["topk"], c["E"], c["N"]
    S = T * topk
    if op.startswith("experts"):
        K = c["K"]
        s["offsets"], s["src"], _ = _order(ids, E)
        s["packed"] = _pack(*_weights(g, E, N, K, c["weights"]), c["weights"])
        # most rows of one expert: the plain form pads to it
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        if op == "experts":
            s["x"] = torch.randn((T, K), generator=g, device="cuda").bfloat16()
            s["bias"] = torch.randn((E, N), generator=g, device="cuda") if c["bias"] else None
            s["y"] = torch.zeros((S, N), device="cuda", dtype=torch.bfloat16)
        else:
            s["dy"] = torch.randn((S, N), generator=g, device="cuda").bfloat16()
            s["dx"] = torch.zeros((S, K), device="cuda", dtype=torch.bfloat16)
        return s
    dt = DTYPES[c["dtype"]]
    if op == "dispatch":
        s["ids"] = ids
        s["x"] = torch.randn((T, N), generator=g, device="cuda").to(dt)
        s["offsets"] = torch.empty(E + 1, device="cuda", dtype=torch.int32)
        s["src"] = torch.full((S,), -1, device="cuda", dtype=torch.int32)
        s["pos"] = torch.empty((T, topk), device="cuda", dtype=torch.int32)
        s["xs"] = torch.zeros((S, N), device="cuda", dtype=dt)
        # scratch of the ordering, kept by a program from step to step
        s["scratch"] = torch.empty(4 * (1024 + 2 * (S // 128 + 8)) * (E + 1), device="cuda",
                                   dtype=torch.uint8)
        return s
    s["weights"] = weights.contiguous()
    _, _, s["pos"] = _order(ids, E)
    s["ys"] = torch.randn((S, N), generator=g, device="cuda").to(dt)
    if op == "combine":
        s["y"] = torch.empty((T, N), device="cuda", dtype=dt)
    else:
        s["dy"] = torch.randn((T, N), generator=g, device="cuda").to(dt)
        s["dys"] = torch.zeros((S, N), device="cuda", dtype=dt)
        s["dw"] = torch.empty((T, topk), device="cuda")
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _dequant(packed, E, N, K, kind):
    """The f32 matrices [E, N, K] of packed ones."""
    p = packed.view(E, -1)
    nib, G = N * K // 2, K // GROUP
    b = p[:, :nib].reshape(E, N, K // 8, 4)
    codes = torch.cat([b & 15, b >> 4], -1).view(E, N, G, GROUP).float() - 8.0
    wide = 2 if kind == "bf16" else 4
    raw = p[:, nib:nib + N * G * wide].contiguous()
    scales = raw.view(torch.bfloat16 if kind == "bf16" else torch.float32).view(E, N, G, 1).float()
    w = codes * scales
    if kind == "asym":
        at = nib + N * G * wide
        w = w + p[:, at:at + N * G * 4].contiguous().view(torch.float32).view(E, N, G, 1)
    return w.view(E, N, K)


def _plain_linear(s):
    c = s["case"]
    w = _dequant(s["packed"], 1, c["N"], c["K"], c["weights"])[0]
    if c["op"] == "linear_grad":
        return (s["dy"].float() @ w).bfloat16()
    y = s["x"].float() @ w.T
    return (y if s["bias"] is None else y + s["bias"]).bfloat16()


def _plain_experts(s):
    c = s["case"]
    E, N, K, most = c["E"], c["N"], c["K"], max(1, s["most"])
    off = s["offsets"].long()
    w = _dequant(s["packed"], E, N, K, c["weights"])
    S = c["T"] * c["topk"]
    at = off[:-1, None] + torch.arange(most, device="cuda")   # [E, most] sorted positions
    at = torch.clamp(at, max=S - 1)
    row = torch.arange(S, device="cuda")
    e = torch.clamp(torch.searchsorted(off, row, right=True) - 1, max=E - 1)
    col = torch.clamp(row - off[e], max=most - 1)
    live = (row < off[E])[:, None]
    if c["op"] == "experts_grad":
        out = torch.bmm(s["dy"].float()[at], w)[e, col]
        return torch.where(live, out.bfloat16(), s["dx"])
    token = torch.clamp(s["src"].long(), min=0)[at] // c["topk"]
    out = torch.bmm(s["x"].float()[token], w.transpose(1, 2))[e, col]
    if s["bias"] is not None:
        out = out + s["bias"][e]
    return torch.where(live, out.bfloat16(), s["y"])


def _plain_rows(s):
    c = s["case"]
    topk, dt = c["topk"], DTYPES[c["dtype"]]
    if c["op"] == "dispatch":
        offsets, src, pos = _order(s["ids"], c["E"])
        rows = s["x"][torch.clamp(src.long(), min=0) // topk]
        xs = torch.where((src >= 0)[:, None], rows, s["xs"])
        return {"offsets": offsets, "src": torch.where(src >= 0, src, s["src"]), "pos": pos,
                "xs": xs}
    pos = s["pos"].long()
    live = (pos >= 0)[..., None]
    rows = s["ys"][torch.clamp(pos, min=0)].float()
    rows = torch.where(live, rows, 0.0)                        # [T, topk, N]
    if c["op"] == "combine":
        return (rows * s["weights"][..., None]).sum(1).to(dt)
    dy = s["dy"].float()
    dw = (rows * dy[:, None, :]).sum(-1)
    d = (s["weights"][..., None] * dy[:, None, :]).to(dt).view(-1, c["N"])
    flat = pos.view(-1)
    kept = torch.zeros(flat.numel() + 1, c["N"], device="cuda", dtype=dt)
    kept[torch.where(flat >= 0, flat, flat.numel())] = d       # one place each; the last is nobody's
    used = torch.zeros(flat.numel() + 1, 1, device="cuda", dtype=torch.bool)
    used[torch.where(flat >= 0, flat, flat.numel())] = True
    return {"dys": torch.where(used[:-1], kept[:-1], s["dys"]), "dw": dw}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if not own:
        if op.startswith("linear"):
            return _plain_linear(s)
        return _plain_experts(s) if op.startswith("experts") else _plain_rows(s)
    import gemv_zero_point_b200 as qg
    c = s["case"]
    if op == "linear":
        qg.qgemm_a16w4_bf16(s["x"], s["packed"], s["y"], bias=s["bias"], weights=c["weights"])
        return s["y"]
    if op == "linear_grad":
        qg.qgemm_a16w4_bf16_grad_x(s["dy"], s["packed"], s["dx"], weights=c["weights"])
        return s["dx"]
    if op == "experts":
        qg.qgemm_a16w4_bf16_experts(s["x"], s["offsets"], s["packed"], s["y"], src=s["src"],
                                    topk=c["topk"], bias=s["bias"], weights=c["weights"])
        return s["y"]
    if op == "experts_grad":
        qg.qgemm_a16w4_bf16_experts_grad_x(s["dy"], s["offsets"], s["packed"], s["dx"],
                                           weights=c["weights"])
        return s["dx"]
    if op == "dispatch":
        qg.qg_sort_by_expert(s["ids"], s["offsets"], s["src"], s["pos"], workspace=s["scratch"])
        qg.qg_spread_rows(s["x"], s["pos"], s["xs"])
        return {"offsets": s["offsets"], "src": s["src"], "pos": s["pos"], "xs": s["xs"]}
    if op == "combine":
        qg.qg_combine_rows(s["ys"], s["pos"], s["y"], weights=s["weights"])
        return s["y"]
    qg.qg_combine_rows_grad(s["dy"], s["ys"], s["pos"], s["weights"], s["dys"], s["dw"])
    return {"dys": s["dys"], "dw": s["dw"]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    per_group = {"f32": 4, "bf16": 2, "asym": 8}
    if op.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K // 2 + N * (K // GROUP) * per_group[c["weights"]]
                + 2 * M * K + 2 * M * N + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    T, topk, E, N = c["T"], c["topk"], c["E"], c["N"]
    S = T * topk * (1.0 - c["drop"])
    if op.startswith("experts"):
        K = c["K"]
        # experts that an even routing of the tokens reaches
        used = E * (1.0 - (1.0 - topk / E) ** (T * (1.0 - c["drop"])))
        rows_in = T * (1.0 - c["drop"]) * K if op == "experts" else S * N
        rows_out = S * N if op == "experts" else S * K
        return {"bytes": used * (N * K / 2 + N * (K // GROUP) * per_group[c["weights"]]
                                 + (4 * N if c["bias"] else 0)) + 2 * rows_in + 2 * rows_out
                + 4 * (E + 1) + (4 * S if op == "experts" else 0), "flops": 2 * S * N * K}
    e = 4 if c["dtype"] == "f32" else 2
    if op == "dispatch":
        return {"bytes": 4 * T * topk * 3 + 4 * (E + 1) + e * N * (T * (1.0 - c["drop"]) + S),
                "flops": 0}
    if op == "combine":
        return {"bytes": 8 * T * topk + e * N * (S + T), "flops": 2 * S * N}
    return {"bytes": 12 * T * topk + e * N * (2 * S + T), "flops": 3 * S * N}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c, g, op = case, _gen(seed), case["op"]

    def real(codes, scales, zeros):
        w = codes.double() * scales.double().repeat_interleave(GROUP, -1)
        return w if zeros is None else w + zeros.double().repeat_interleave(GROUP, -1)

    if op.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        w = real(*_weights(g, 1, N, K, c["weights"]))[0]
        if op == "linear_grad":
            return torch.randn((M, N), generator=g, device="cuda").bfloat16().double() @ w
        y = torch.randn((M, K), generator=g, device="cuda").bfloat16().double() @ w.T
        return y + torch.randn(N, generator=g, device="cuda").double() if c["bias"] else y
    ids, weights = _routing(g, c)
    T, topk, E, N = c["T"], c["topk"], c["E"], c["N"]
    S = T * topk
    flat = ids.view(-1).long().cpu()
    if op.startswith("experts"):
        K = c["K"]
        parts = _weights(g, E, N, K, c["weights"])
        shape = (T, K) if op == "experts" else (S, N)
        rows = torch.randn(shape, generator=g, device="cuda").bfloat16().double()
        bias = torch.randn((E, N), generator=g, device="cuda").double() if c["bias"] else None
        out = torch.zeros((S, N if op == "experts" else K), device="cuda", dtype=torch.float64)
        at = 0
        for e in range(E):
            mine = (flat == e).nonzero().view(-1).cuda()
            n = mine.numel()
            if n:
                w = real(*[None if p is None else p[e] for p in parts])
                if op == "experts":
                    out[at:at + n] = rows[mine // topk] @ w.T + (0 if bias is None else bias[e])
                else:
                    out[at:at + n] = rows[at:at + n] @ w
            at += n
        return out
    dt = DTYPES[c["dtype"]]
    if op == "dispatch":
        x = torch.randn((T, N), generator=g, device="cuda").to(dt).double()
        out = torch.zeros((S, N), device="cuda", dtype=torch.float64)
        lists = [(flat == e).nonzero().view(-1) for e in range(E)]
        order = torch.cat(lists).cuda()
        out[:order.numel()] = x[order // topk]
        return {"offsets": None, "src": None, "pos": None, "xs": out}
    lists = torch.cat([(flat == e).nonzero().view(-1) for e in range(E)])
    place = torch.full((S,), -1, dtype=torch.long)
    place[lists] = torch.arange(lists.numel())
    place = place.view(T, topk).cuda()
    ys = torch.randn((S, N), generator=g, device="cuda").to(dt).double()
    w = weights.double()
    if op == "combine":
        y = torch.zeros((T, N), device="cuda", dtype=torch.float64)
        for j in range(topk):
            hit = place[:, j] >= 0
            y[hit] += w[hit, j, None] * ys[place[hit, j]]
        return y
    dy = torch.randn((T, N), generator=g, device="cuda").to(dt).double()
    dys = torch.zeros((S, N), device="cuda", dtype=torch.float64)
    dw = torch.zeros((T, topk), device="cuda", dtype=torch.float64)
    for j in range(topk):
        hit = place[:, j] >= 0
        dys[place[hit, j]] = w[hit, j, None] * dy[hit]
        dw[hit, j] = (dy[hit] * ys[place[hit, j]]).sum(-1)
    return {"dys": dys, "dw": dw}
