"""The operators of one mixture-of-experts layer around its expert products, as measurable cases:

  route     top-k routing of router logits with the balance loss and the per-expert counts, and its backward
  dispatch  expert-sorted order of the routed tokens: offsets, source row of each slot, slot of each choice
  quantize  E4M3 codes with one fp32 scale per 128 elements: rows (gathered), token columns per expert, weight blocks
  gemm      grouped product of such operands: forward, or the two backward products
  combine   weighted sum of each token's expert outputs, and its backward

``run`` computes a case in plain torch operations, or, where ``own`` is true,
by calls of the package's entry points.  ``exact`` restates the definitions
in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128          # elements that share a scale
TINY = 2.0 ** -100   # smallest block maximum that sets a scale by itself
LOSS_COEF = 0.01


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 16 sequences against 384 experts: latency only
        dict(name="route decode 16x384", op="route", tokens=16, experts=384, top_k=8, dtype="bf16", normalize=True,
             bias=True, masked=0.0, groups=False, train=False),
        # a training micro-batch: padded tokens, experts of half the groups ruled out per token, forward and backward
        dict(name="route train 16384x384", op="route", tokens=16384, experts=384, top_k=8, dtype="f32",
             normalize=True, bias=True, masked=0.05, groups=True, train=True),
        # the decoding step's 128 choices; and a training micro-batch with the padded tokens' choices left out
        dict(name="dispatch decode 16x8", op="dispatch", tokens=16, experts=384, top_k=8, masked=0.0),
        dict(name="dispatch train 16384x8", op="dispatch", tokens=16384, experts=384, top_k=8, masked=0.05),
        # activations of 4096 tokens gathered into 32768 expert-sorted slots, for the forward and for the weight gradient
        dict(name="quantize tokens 32768x7168", op="quantize", what="tokens", tokens=4096, top_k=8, experts=32,
             width=7168, skew=1.1, both=True),
        # the gate/up weights of 32 experts after an optimizer step, both orientations
        dict(name="quantize weights 32x4096x7168", op="quantize", what="weights", experts=32, n=4096, k=7168),
        # 8 decoding tokens, 64 routed rows over 32 experts: the weights are read for a row or two each
        dict(name="gemm decode 64 rows", op="gemm", way="fwd", rows=64, experts=32, n=4096, k=7168, skew=1.1),
        # odd sizes: ragged experts, widths that are no multiple of a tile or of a block
        dict(name="gemm ragged 3001 rows", op="gemm", way="fwd", rows=3001, experts=12, n=1424, k=2000, skew=1.5),
        # the gate/up product of the 32-expert training shard, and its gradients
        dict(name="gemm fwd 32768 rows", op="gemm", way="fwd", rows=32768, experts=32, n=4096, k=7168, skew=1.1),
        dict(name="gemm bwd 32768 rows", op="gemm", way="bwd", rows=32768, experts=32, n=4096, k=7168, skew=1.1),
        # the decoding step's outputs, and those of the training shard with their gradients
        dict(name="combine decode 16x7168", op="combine", tokens=16, top_k=8, width=7168, masked=0.0, train=False),
        dict(name="combine train 4096x7168", op="combine", tokens=4096, top_k=8, width=7168, masked=0.05, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "quantize", "gemm", "gemm", "combine"])
    masked = rng.choice([0.0, 0.05, 0.3])
    experts = _log(rng, 4, 512)
    top_k = rng.randint(1, min(8, experts // 2))
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=min(experts, 384), top_k=top_k,
                    dtype=rng.choice(["bf16", "f32"]), normalize=rng.random() < 0.5, bias=rng.random() < 0.5,
                    masked=masked, groups=rng.random() < 0.3, train=rng.random() < 0.6)
    if op == "dispatch":
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=min(experts, 384), top_k=top_k, masked=masked)
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 4096), top_k=rng.randint(1, 8), width=8 * _log(rng, 16, 896),
                    masked=masked, train=rng.random() < 0.6)
    if op == "quantize":
        if rng.random() < 0.5:
            return dict(op=op, what="weights", experts=_log(rng, 1, 32), n=16 * _log(rng, 8, 256),
                        k=16 * _log(rng, 8, 448))
        return dict(op=op, what="tokens", tokens=_log(rng, 1, 4096), top_k=rng.randint(1, 8),
                    experts=_log(rng, 1, 64), width=16 * _log(rng, 8, 448), skew=rng.choice([0.0, 1.1, 1.5]),
                    both=rng.random() < 0.5)
    way = rng.choice(["fwd", "fwd", "bwd"])
    return dict(op=op, way=way, rows=_log(rng, 1, 32768), experts=_log(rng, 1, 32), n=16 * _log(rng, 16, 256),
                k=16 * _log(rng, 16, 448), skew=rng.choice([0.0, 1.1, 1.5]))


def _counts(total, n, s):
    """Rows per expert, most popular first: P(rank r) ~ r^-s, largest remainders."""
    p = [(r + 1) ** -s for r in range(n)]
    raw = [total * v / sum(p) for v in p]
    c = [int(v) for v in raw]
    for i in sorted(range(n), key=lambda i: (c[i] - raw[i], i))[:total - sum(c)]:
        c[i] += 1
    return c


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        z = 2 if case["dtype"] == "bf16" else 4
        b, f = t * (e * z + 8 * k + 4) + 8 * e, 8 * t * e
        if case["train"]:
            b, f = b + t * (2 * e * z + 12 * k + 4) + 4 * e, f + 8 * t * e
        return {"bytes": b, "flops": f}
    if op == "dispatch":
        n = case["tokens"] * case["top_k"]
        return {"bytes": 12 * n + 4 * case["experts"], "flops": n}
    if op == "combine":
        t, k, w = case["tokens"], case["top_k"], case["width"]
        live = t * k - round(case["masked"] * t) * k
        b, f = 2 * live * w + 8 * t * k + 2 * t * w, 2 * live * w
        if case["train"]:
            b, f = b + 2 * t * w + 2 * live * w + 2 * t * k * w + 12 * t * k, f + 4 * live * w
        return {"bytes": b, "flops": f}
    if op == "quantize":
        if case["what"] == "weights":
            n = case["experts"] * case["n"] * case["k"]
            return {"bytes": 4 * n + n // 4096, "flops": 2 * n}
        m = case["tokens"] * case["top_k"] * case["width"]
        both = 2 if case["both"] else 1
        return {"bytes": 2 * case["tokens"] * case["width"] + both * (m + m // 32), "flops": 2 * both * m}
    m, n, k = case["rows"], case["n"], case["k"]
    live = sum(c > 0 for c in _counts(m, case["experts"], case["skew"]))
    if case["way"] == "fwd":
        return {"bytes": m * (k + k // 32) + live * n * k + 2 * m * n, "flops": 2 * m * n * k}
    return {"bytes": m * (2 * n + k) + m * (2 * n + k) // 32 + live * n * k + 2 * m * k + 2 * case["experts"] * n * k,
            "flops": 4 * m * n * k}


# --------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _offsets(rows, experts, skew, seed):
    """Host list of expert offsets: skewed counts, shuffled onto the experts."""
    c = _counts(rows, experts, skew)
    p = torch.randperm(experts, generator=torch.Generator().manual_seed(seed)).tolist()
    off = [0]
    for i in p:
        off.append(off[-1] + c[i])
    return off


def _rand_ids(tokens, experts, top_k, masked, g):
    """Distinct experts per token, some experts much more popular; -1 for the tokens that are padding."""
    pop = torch.rand(experts, generator=g, device=DEV) * 2
    ids = (torch.rand(tokens, experts, generator=g, device=DEV) + pop).topk(top_k, dim=1).indices.int()
    out = torch.randperm(tokens, generator=g, device=DEV)[:round(masked * tokens)]
    ids[out] = -1
    return ids


def _e4m3_blocks(shape, sigma, g):
    """Codes (uint8) of normal values along the last axis and fp32 scales [blocks][rows], as a row quantization gives."""
    rows, cols = shape
    nb = -(-cols // BLOCK)
    x = torch.zeros(rows, nb * BLOCK, device=DEV)
    x[:, :cols] = torch.randn(rows, cols, generator=g, device=DEV) * sigma
    x = x.view(rows, nb, BLOCK)
    a = x.abs().amax(2)
    codes = (x * (448.0 / a)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, nb * BLOCK)
    return codes[:, :cols].contiguous().view(torch.uint8), (a / 448.0).t().contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = torch.randn(t, e, generator=g, device=DEV) * 1.5
        if case["groups"]:  # a token may only go to the experts of half the groups
            n = max(2, min(8, e // (2 * k)))
            keep = torch.rand(t, n, generator=g, device=DEV).argsort(1) < -(-n // 2)
            x = x.masked_fill(~keep[:, torch.arange(e, device=DEV) * n // e], -math.inf)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.ones(t, dtype=torch.uint8, device=DEV)
            s["mask"][torch.randperm(t, generator=g, device=DEV)[:round(case["masked"] * t)]] = 0
            x[s["mask"] == 0] = math.nan  # what padding holds is never looked at
        s["logits"] = x.to(dt)
        s["bias"] = torch.randn(e, generator=g, device=DEV) * 0.1 if case["bias"] else None
        s["dweights"] = torch.randn(t, k, generator=g, device=DEV)
        s["dloss"] = torch.rand(1, generator=g, device=DEV) + 0.5
    elif op == "dispatch":
        s["ids"] = _rand_ids(case["tokens"], case["experts"], case["top_k"], case["masked"], g)
    elif op == "combine":
        t, k, w = case["tokens"], case["top_k"], case["width"]
        ids = _rand_ids(t, max(16, 2 * k), k, case["masked"], g)
        s["offsets"], _, s["slot"] = _dispatch(ids, max(16, 2 * k))
        s["ye"] = torch.randn(t * k, w, generator=g, device=DEV).bfloat16()
        s["ye"][(s["slot"] >= 0).sum():] = math.nan  # rows that no choice owns are never looked at
        s["weights"] = torch.rand(t, k, generator=g, device=DEV)
        s["dy"] = torch.randn(t, w, generator=g, device=DEV).bfloat16()
    elif op == "quantize" and case["what"] == "weights":
        s["w"] = (torch.randn(case["experts"] * case["n"], case["k"], generator=g, device=DEV) * 0.02).bfloat16()
    elif op == "quantize":
        t, k = case["tokens"], case["top_k"]
        s["off"] = _offsets(t * k, case["experts"], case["skew"], seed)
        s["offsets"] = torch.tensor(s["off"], dtype=torch.int32, device=DEV)
        s["row_index"] = (torch.randperm(t * k, generator=g, device=DEV) // k).int()
        x = torch.randn(t, case["width"], generator=g, device=DEV)
        x[:, torch.randperm(case["width"], generator=g, device=DEV)[:case["width"] // 100]] *= 50
        s["x"] = x.bfloat16()
    else:
        m, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        s["off"] = _offsets(m, e, case["skew"], seed)
        s["offsets"] = torch.tensor(s["off"], dtype=torch.int32, device=DEV)
        fwd = case["way"] == "fwd"
        # weights: codes [E*n][k] (forward) or transposed [E*k][n] (backward), scales [E][n blocks][k blocks]
        r, c = (n, k) if fwd else (k, n)
        s["w_codes"] = (torch.randn(e * r, c, generator=g, device=DEV) * 110).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s["w_scale"] = (1 + torch.rand(e, -(-n // BLOCK), -(-k // BLOCK), generator=g, device=DEV)) * 1e-4
        if fwd:
            s["a_codes"], s["a_scale"] = _e4m3_blocks((m, k), 1.0, g)
        else:
            s["dy_codes"], s["dy_scale"] = _e4m3_blocks((m, n), 1e-3, g)
            # token columns per expert: [width][P], an expert's segment on a 128-column boundary, padding zero
            p = BLOCK * (e + -(-m // BLOCK))
            real = torch.zeros(p, dtype=torch.bool, device=DEV)
            for i in range(e):
                at = BLOCK * (i + s["off"][i] // BLOCK)
                real[at:at + s["off"][i + 1] - s["off"][i]] = True
            for name, w, sigma in (("dyt", n, 1e-3), ("xt", k, 1.0)):
                codes, scale = _e4m3_blocks((w, p), sigma, g)
                codes[:, ~real] = 0
                scale *= real.view(-1, BLOCK).any(1)[:, None]
                s[name + "_codes"], s[name + "_scale"] = codes, scale
    return s


# ----------------------------------------------------------- the plain forms

def _route(s):
    e, k = s["experts"], s["top_k"]
    x = s["logits"].float()
    live = torch.ones(x.shape[0], dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"] != 0
    x = torch.where(live[:, None], x, -math.inf)
    key = x if s["bias"] is None else x + s["bias"]
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    ok = key.gather(1, order) > -math.inf
    live = ok.any(1)
    ids = torch.where(ok, order, -1).int()
    top = x.amax(1, keepdim=True)
    ex = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = ex.sum(1, keepdim=True)
    lse = torch.where(live, (torch.log(total) + top)[:, 0], -math.inf)
    p = ex / torch.where(total > 0, total, 1.0)
    w = torch.where(ok, p.gather(1, order), 0.0)
    if s["normalize"]:
        sel = w.sum(1, keepdim=True)
        w = w / torch.where(sel > 0, sel, 1.0)
    counts = (ids.flatten()[:, None] == torch.arange(e, device=x.device)).sum(0) if ids.numel() * e < 1 << 24 else \
        torch.zeros(e + 1, dtype=torch.int64, device=x.device).index_add_(
            0, torch.where(ok, order, e).flatten(), torch.ones_like(order).flatten())[:e]
    tokens = live.sum()
    nv = tokens.clamp(min=1)
    share = p.double().sum(0) / nv
    loss = (LOSS_COEF * e / k) * (counts * share).sum() / nv
    out = [ids, w, lse, torch.cat([counts, tokens[None]]).int(), loss.float().reshape(1)]
    if not s["train"]:
        return out
    dw = torch.where(ok, s["dweights"], 0.0)
    at = torch.where(ok, order, 0)
    if s["normalize"]:
        d = torch.zeros_like(x).scatter_add_(1, at, torch.where(ok, w * (dw - (w * dw).sum(1, keepdim=True)), 0.0))
        up = torch.zeros_like(x)
    else:
        d = torch.zeros_like(x)
        up = torch.zeros_like(x).scatter_add_(1, at, dw)
    up = up + ((s["dloss"] * LOSS_COEF * e / k) * counts / (nv.double() * nv)).float()
    d = d + p * (up - (p * up).sum(1, keepdim=True))
    return out + [torch.where(live[:, None], d, 0.0).to(s["logits"].dtype)]


def _dispatch(ids, experts):
    t, k = ids.shape
    flat = torch.where(ids < 0, experts, ids).flatten()
    grouped, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(grouped, torch.arange(experts + 1, device=ids.device, dtype=grouped.dtype)).int()
    ok = grouped < experts
    row_index = torch.where(ok, order // k, -1).int()
    slot = torch.empty(t * k, dtype=torch.int32, device=ids.device)
    slot[order] = torch.where(ok, torch.arange(t * k, device=ids.device), -1).int()
    return offsets, row_index, slot.view(t, k)


def _combine(s):
    slot, w, ye = s["slot"], s["weights"], s["ye"]
    ok = slot >= 0
    rows = torch.where(ok[:, :, None], ye[slot.clamp(min=0).long()].float(), 0.0)
    y = (torch.where(ok, w, 0.0)[:, :, None] * rows).sum(1)
    if not s["train"]:
        return [y.bfloat16()]
    dy = s["dy"].float()
    dw = (rows * dy[:, None, :]).sum(2)
    dye = torch.zeros(ye.shape[0] + 1, ye.shape[1], dtype=torch.bfloat16, device=ye.device)
    dye[torch.where(ok, slot, ye.shape[0]).long()] = (w[:, :, None] * dy[:, None, :]).bfloat16()
    dye[-1] = 0
    return [y.bfloat16(), dye[:-1], dw]


def _encode(x, a):
    """Codes and scales of blocks x with maxima a (broadcastable): RN(x * RN(448 / a)), RN(a / 448); zero blocks give 0."""
    c = a.clamp(min=TINY)
    return (x * (448.0 / c)).clamp(-448, 448).to(torch.float8_e4m3fn), torch.where(a > 0, c / 448.0, 0.0)


def _rows(x):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    codes, scale = _encode(x, x.abs().amax(2, keepdim=True))
    return codes.view(rows, -1)[:, :cols].contiguous(), scale[:, :, 0].t().contiguous()


def _columns(x, offsets):
    """Blocks of 128 down each group's rows, transposed: group i starts at column 128 * (i + offsets[i] // 128)."""
    rows, cols = x.shape
    e = offsets.numel() - 1
    p = BLOCK * (e + -(-rows // BLOCK))
    r = torch.arange(rows, device=x.device)
    grp = torch.searchsorted(offsets, r.int(), right=True) - 1
    start = offsets[grp].long()
    t = torch.zeros(p, cols, dtype=x.dtype, device=x.device)
    t[BLOCK * (grp + start // BLOCK) + r - start] = x
    t = t.float().view(p // BLOCK, BLOCK, cols)
    codes, scale = _encode(t, t.abs().amax(1, keepdim=True))
    return codes.view(p, cols).t().contiguous(), scale[:, 0].contiguous()


def _weights(w, e, n, k):
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    x = torch.nn.functional.pad(w.float().view(e, n, k), (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    x = x.view(e, nb, BLOCK, kb, BLOCK)
    codes, scale = _encode(x, x.abs().amax((2, 4), keepdim=True))
    codes = codes.view(e, nb * BLOCK, kb * BLOCK)[:, :n, :k].contiguous()
    return codes.view(e * n, k), codes.transpose(1, 2).contiguous().view(e * k, n), scale.view(e, nb, kb)


def _value(codes, scale):
    """fp32 values of codes [r][c] with scales [blocks][r]."""
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(BLOCK, 0)[:codes.shape[1]].t()


def _wvalue(codes, scale):
    """fp32 values of codes [r][c] with scales [r blocks][c blocks]."""
    f = scale.repeat_interleave(BLOCK, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).float() * f


def _gemm(s):
    off, n, k, m = s["off"], s["n"], s["k"], s["rows"]
    experts = [i for i in range(s["experts"]) if off[i + 1] > off[i]]
    if s["way"] == "fwd":
        y = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
        a = _value(s["a_codes"], s["a_scale"])
        for i in experts:
            y[off[i]:off[i + 1]] = a[off[i]:off[i + 1]] @ _wvalue(s["w_codes"][i * n:(i + 1) * n], s["w_scale"][i]).t()
        return [y]
    dx = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    dw = torch.zeros(s["experts"], n, k, dtype=torch.bfloat16, device=DEV)
    dy = _value(s["dy_codes"], s["dy_scale"])
    dyt, xt = _value(s["dyt_codes"], s["dyt_scale"]), _value(s["xt_codes"], s["xt_scale"])
    for i in experts:
        lo, hi = off[i], off[i + 1]
        dx[lo:hi] = dy[lo:hi] @ _wvalue(s["w_codes"][i * k:(i + 1) * k], s["w_scale"][i].t()).t()
        c = BLOCK * (i + lo // BLOCK)
        dw[i] = dyt[:, c:c + hi - lo] @ xt[:, c:c + hi - lo].t()
    return [dx, dw]


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "route":
        return _route(s)
    if op == "dispatch":
        return list(_dispatch(s["ids"], s["experts"]))
    if op == "combine":
        return _combine(s)
    if op == "gemm":
        return _gemm(s)
    if s["what"] == "weights":
        return list(_weights(s["w"], s["experts"], s["n"], s["k"]))
    x = s["x"][s["row_index"].long()]
    return list(_rows(x)) + (list(_columns(x, s["offsets"])) if s["both"] else [])


def _own(s):
    import block_scaled_precision_bsq_amd as bsq
    op = s["op"]
    f8 = torch.float8_e4m3fn
    if op == "route":
        how = dict(normalize=s["normalize"], loss_coef=LOSS_COEF)
        ids, w, lse, counts, loss = bsq.bsq_moe_route(s["logits"], s["top_k"], bias=s["bias"], mask=s["mask"], **how)
        out = [ids, w, lse, counts, loss]
        if s["train"]:
            out.append(bsq.bsq_moe_route_bwd(s["logits"], ids, w, lse, counts, s["dweights"], s["dloss"], **how))
        return out
    if op == "dispatch":
        return list(bsq.bsq_moe_dispatch(s["ids"], s["experts"]))
    if op == "combine":
        y = bsq.bsq_moe_combine(s["ye"], s["slot"], s["weights"])
        if not s["train"]:
            return [y]
        return [y, *bsq.bsq_moe_combine_bwd(s["dy"], s["ye"], s["slot"], s["weights"], s["offsets"])]
    if op == "quantize" and s["what"] == "weights":
        codes, codes_t, scale = bsq.bsq_quantize_fp8b128_weights(s["w"], s["experts"])
        return [codes.view(f8), codes_t.view(f8), scale]
    if op == "quantize":
        row, t = bsq.bsq_quantize_fp8b128(s["x"], row_index=s["row_index"], offsets=s["offsets"] if s["both"] else None)
        return [row[0].view(f8), row[1]] + ([t[0].view(f8), t[1]] if s["both"] else [])
    if s["way"] == "fwd":
        return [bsq.bsq_grouped_gemm_fp8b128_fwd((s["a_codes"], s["a_scale"]), (s["w_codes"], s["w_scale"]),
                                                 s["offsets"])]
    return list(bsq.bsq_grouped_gemm_fp8b128_bwd(
        s["offsets"], s["rows"], s["n"], s["k"], dy_q=(s["dy_codes"], s["dy_scale"]),
        wt_q=(s["w_codes"], s["w_scale"]), dyt_q=(s["dyt_codes"], s["dyt_scale"]),
        xt_q=(s["xt_codes"], s["xt_scale"])))


# ------------------------------------------------------- the same in 64 bits

def _e4m3_grid():
    """The finite non-negative E4M3 values by code, from their bit fields."""
    return torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=DEV)


def _nearest(v):
    """Nearest E4M3 value of v (|v| <= 448), ties to the even code."""
    grid = _e4m3_grid()
    a = v.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    return torch.copysign(grid[torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)], v)


def _blockwise(x, dim_rows, dim_cols):
    """Codes (values) and scales of dim_rows x dim_cols blocks of x [r][c] in 64 bits, a strip of rows at a time."""
    r, c = x.shape
    codes, scales = torch.empty(r, c, dtype=torch.float32, device=DEV), []
    strip = max(1, (1 << 25) // max(1, c) // dim_rows) * dim_rows
    for at in range(0, r, strip):
        v = x[at:at + strip].double()
        pad = torch.zeros(-(-v.shape[0] // dim_rows) * dim_rows, -(-c // dim_cols) * dim_cols, dtype=torch.float64,
                          device=DEV)
        pad[:v.shape[0], :c] = v
        b = pad.view(pad.shape[0] // dim_rows, dim_rows, pad.shape[1] // dim_cols, dim_cols)
        a = b.abs().amax((1, 3))
        inv = torch.where(a > 0, 448.0 / a, 0.0)
        codes[at:at + strip] = _nearest((b * inv[:, None, :, None]).clamp(-448, 448)).view(pad.shape)[:v.shape[0], :c]
        scales.append(a / 448.0)
    return codes, torch.cat(scales)


def _of_bytes(codes):
    grid = _e4m3_grid()
    b = codes.long()
    return torch.where(b >= 128, -grid[(b & 127).clamp(max=126)], grid[(b & 127).clamp(max=126)])


def exact(case, seed):
    if case["op"] == "dispatch":  # whole numbers only
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        k, e = s["top_k"], s["experts"]
        x = s["logits"].double()
        if s["mask"] is not None:
            x[s["mask"] == 0] = -math.inf
        key = (s["logits"].float() + (0 if s["bias"] is None else s["bias"])).double()
        key[torch.isnan(key) | (x == -math.inf)] = -math.inf
        # the k first of the order (key descending, index ascending), one at a time
        chosen = torch.zeros_like(x, dtype=torch.bool)
        picks = []
        for _ in range(k):
            best = key.masked_fill(chosen, -math.inf)
            top = best.amax(1, keepdim=True)
            first = (best == top).int().argmax(1, keepdim=True)
            picks.append(torch.where(top > -math.inf, first, -1))
            chosen.scatter_(1, first, chosen.gather(1, first) | (top > -math.inf))
        ids = torch.cat(picks, 1)
        live = chosen.any(1)
        p = torch.where(live[:, None], torch.softmax(x, 1), 0.0)
        lse = torch.where(live, torch.logsumexp(x, 1), -math.inf)
        of = chosen * p
        den = of.sum(1, keepdim=True) if s["normalize"] else torch.ones_like(of[:, :1])
        share = torch.where(chosen, p / den, 0.0)
        w = torch.where(ids >= 0, share.gather(1, ids.clamp(min=0)), 0.0)
        f = chosen.double().sum(0)
        nv = max(1, int(live.sum()))
        coef = LOSS_COEF * e / (k * nv)
        out = [None, w, lse, None, (coef * (f * p.sum(0) / nv).sum()).reshape(1)]
        if s["train"]:
            dw = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, s["dweights"].double(), 0.0))
            up = s["dloss"].double() * coef * f / nv
            d = p * (up - (p @ up)[:, None])
            inner = (share * dw).sum(1, keepdim=True)
            d = d + (share * (dw - inner) if s["normalize"] else share * dw - p * inner)
            out.append(torch.where(live[:, None], d, 0.0))
        return out
    if op == "combine":
        t, k, width = s["tokens"], s["top_k"], s["width"]
        y = torch.zeros(t, width, dtype=torch.float64, device=DEV)
        dye = torch.zeros(t * k, width, dtype=torch.float64, device=DEV)
        dw = torch.zeros(t, k, dtype=torch.float64, device=DEV)
        dy = s["dy"].double()
        for j in range(k):
            on = (s["slot"][:, j] >= 0).nonzero()[:, 0]
            at = s["slot"][on, j].long()
            rows, w = s["ye"][at].double(), s["weights"][on, j].double()[:, None]
            y[on] += w * rows
            dye[at] = w * dy[on]
            dw[on, j] = (rows * dy[on]).sum(1)
        return [y, dye, dw] if s["train"] else [y]
    if op == "quantize" and case["what"] == "weights":
        e, n, k = s["experts"], s["n"], s["k"]
        codes, scales = zip(*(_blockwise(s["w"][i * n:(i + 1) * n], BLOCK, BLOCK) for i in range(e)))
        return [torch.cat(codes), torch.cat([c.t() for c in codes]), torch.stack(scales)]
    if op == "quantize":
        x = s["x"][s["row_index"].long()]
        codes, scale = _blockwise(x, 1, BLOCK)
        out = [codes, scale.t()]
        if s["both"]:
            e, off = s["experts"], s["off"]
            p = BLOCK * (e + -(-x.shape[0] // BLOCK))
            tc = torch.zeros(p, x.shape[1], device=DEV)
            ts = torch.zeros(p // BLOCK, x.shape[1], dtype=torch.float64, device=DEV)
            for i in range(e):
                if off[i + 1] > off[i]:
                    c, sc = _blockwise(x[off[i]:off[i + 1]], BLOCK, 1)
                    b = i + off[i] // BLOCK
                    tc[BLOCK * b:BLOCK * b + c.shape[0]] = c
                    ts[b:b + sc.shape[0]] = sc
            out += [tc.t(), ts]
        return out
    m, n, k, off = s["rows"], s["n"], s["k"], s["off"]

    def value(codes, scale):  # scale: [r or 1 of each block row][c blocks], by index
        return _of_bytes(codes) * scale.double()[:, torch.arange(codes.shape[1], device=DEV) // BLOCK]

    def by_row(scale, r):
        return scale[torch.arange(r, device=DEV) // BLOCK]

    live = [i for i in range(s["experts"]) if off[i + 1] > off[i]]
    if case["way"] == "fwd":
        y = torch.empty(m, n, dtype=torch.float64, device=DEV)
        for i in live:
            w = value(s["w_codes"][i * n:(i + 1) * n], by_row(s["w_scale"][i], n))
            y[off[i]:off[i + 1]] = torch.matmul(value(s["a_codes"][off[i]:off[i + 1]],
                                                      s["a_scale"][:, off[i]:off[i + 1]].t()), w.t())
        return [y]
    dx = torch.empty(m, k, dtype=torch.float64, device=DEV)
    dw = torch.zeros(s["experts"], n, k, dtype=torch.float64, device=DEV)
    for i in live:
        lo, hi = off[i], off[i + 1]
        w = value(s["w_codes"][i * k:(i + 1) * k], by_row(s["w_scale"][i].t(), k))
        dx[lo:hi] = torch.matmul(value(s["dy_codes"][lo:hi], s["dy_scale"][:, lo:hi].t()), w.t())
        b, nb = i + lo // BLOCK, -(-(hi - lo) // BLOCK)
        sl = slice(BLOCK * b, BLOCK * (b + nb))
        dw[i] = torch.matmul(value(s["dyt_codes"][:, sl], s["dyt_scale"][b:b + nb].t()),
                             value(s["xt_codes"][:, sl], s["xt_scale"][b:b + nb].t()).t())
    return [dx, dw]
