"""Plain NumPy implementations of routing, dispatch, combine and the FP8B128
format, in 64 bits, written from their definitions.  Test infrastructure, like
the rest of this package."""
from __future__ import annotations

import numpy as np

BLOCK = 128
F32_MAX = float(np.finfo(np.float32).max)


def _canon(logits):
    x = np.asarray(logits, np.float64).copy()
    x[np.isnan(x)] = -np.inf
    return np.minimum(x, F32_MAX)


def route(logits, top_k, bias=None, mask=None, normalize=True, scale=1.0, coef=0.0):
    """(ids, weights, lse, counts [E + 1], loss) of float logits [T][E]."""
    l = _canon(logits)
    T, E = l.shape
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        key = (l.astype(np.float32) + (np.float32(0) if bias is None else np.asarray(bias, np.float32))).astype(np.float32)
    key[np.isnan(key)] = -np.inf
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    lse = np.full(T, -np.inf)
    counts = np.zeros(E + 1, np.int32)
    psum = np.zeros(E)
    for t in range(T):
        order = sorted((e for e in range(E) if key[t, e] > -np.inf), key=lambda e: (-float(key[t, e]), e))[:top_k]
        if not order:
            continue
        m = l[t].max()
        ex = np.exp(l[t] - m)
        lse[t] = m + np.log(ex.sum())
        p = ex / ex.sum()
        ids[t, :len(order)] = order
        if normalize:
            s = np.exp(l[t, order] - l[t, order].max())
            weights[t, :len(order)] = scale * s / s.sum()
        else:
            weights[t, :len(order)] = scale * p[order]
        counts[order] += 1
        counts[E] += 1
        psum += p
    v = max(1, int(counts[E]))
    loss = coef * E / (top_k * v) * float((counts[:E] * psum).sum()) / v
    return ids, weights, lse, counts, loss


def route_bwd(logits, ids, counts, dweights, dloss, normalize=True, scale=1.0, coef=0.0, mask=None):
    """dlogits [T][E] for the given choices."""
    l = _canon(logits)
    T, E = l.shape
    K = ids.shape[1]
    v = max(1, int(counts[E]))
    u0 = dloss * coef * E / (K * v) * counts[:E].astype(np.float64) / v
    d = np.zeros((T, E))
    for t in range(T):
        sel = ids[t][ids[t] >= 0]
        if sel.size == 0 or (mask is not None and mask[t] == 0):
            continue
        ex = np.exp(l[t] - l[t].max())
        p = ex / ex.sum()
        dw = scale * np.asarray(dweights[t][:sel.size], np.float64)
        u = u0.copy()
        if normalize:
            q = np.exp(l[t, sel] - l[t, sel].max())
            q /= q.sum()
            d[t, sel] += q * (dw - (q * dw).sum())
        else:
            u[sel] += dw
        d[t] += p * (u - (p * u).sum())
    return d


def dispatch(ids, num_experts):
    """(offsets, row_index, slot) by a plain scan."""
    T, K = ids.shape
    flat = ids.reshape(-1)
    lists = [[] for _ in range(num_experts + 1)]
    for i, e in enumerate(flat):
        lists[e if 0 <= e < num_experts else num_experts].append(i)
    offsets = np.zeros(num_experts + 1, np.int32)
    row_index = np.full(T * K, -1, np.int32)
    slot = np.full(T * K, -1, np.int32)
    at = 0
    for e in range(num_experts):
        for i in lists[e]:
            row_index[at], slot[i] = i // K, at
            at += 1
        offsets[e + 1] = at
    return offsets, row_index, slot.reshape(T, K)


def combine(ye, slot, weights=None):
    T, K = slot.shape
    y = np.zeros((T, ye.shape[1]))
    for t in range(T):
        for j in range(K):
            if 0 <= slot[t, j] < ye.shape[0]:
                y[t] += (1.0 if weights is None else float(weights[t, j])) * ye[slot[t, j]].astype(np.float64)
    return y


def combine_bwd(dy, ye, slot, weights=None):
    T, K = slot.shape
    dye = np.zeros(ye.shape)
    dw = np.zeros((T, K))
    for t in range(T):
        for j in range(K):
            s = slot[t, j]
            if 0 <= s < ye.shape[0]:
                dye[s] = (1.0 if weights is None else float(weights[t, j])) * dy[t].astype(np.float64)
                dw[t, j] = (dy[t].astype(np.float64) * ye[s].astype(np.float64)).sum()
    return dye, dw


def _grid():
    return np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def e4m3_encode(v):
    """Nearest E4M3 codes of |v|, ties to even, saturating at 448; sign kept."""
    g = _grid()
    a = np.minimum(np.abs(v).astype(np.float64), 448.0)
    hi = np.clip(np.searchsorted(g, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - g[lo], g[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return c | (np.signbit(v).astype(np.uint8) << 7)


def e4m3_decode(c):
    g = np.append(_grid(), np.nan)
    return np.where(c & 0x80, -1.0, 1.0) * g[c & 0x7F]


def _block(x):
    """Codes and scale of one block of float32 values (the binary32 steps of the definition)."""
    a = np.float32(np.abs(x).max()) if x.size else np.float32(0)
    c = max(a, np.float32(2.0 ** -100))
    inv = np.float32(448.0) / c
    return e4m3_encode((x.astype(np.float32) * inv).astype(np.float32)), (c / np.float32(448.0) if a > 0 else np.float32(0))


def b128_rows(x):
    """x float32 [R][C] -> codes [R][C], scale [ceil(C/128)][R]."""
    R, C = x.shape
    nb = -(-C // BLOCK)
    codes, scale = np.zeros((R, C), np.uint8), np.zeros((nb, R), np.float32)
    for r in range(R):
        for b in range(nb):
            s = slice(b * BLOCK, min(C, (b + 1) * BLOCK))
            codes[r, s], scale[b, r] = _block(x[r, s])
    return codes, scale


def b128_columns(x, offsets):
    """x float32 [R][C] -> t_codes [C][P], t_scale [P/128][C]."""
    R, C = x.shape
    G = len(offsets) - 1
    P = BLOCK * (G + -(-R // BLOCK))
    codes, scale = np.zeros((C, P), np.uint8), np.zeros((P // BLOCK, C), np.float32)
    for g in range(G):
        for at in range(offsets[g], offsets[g + 1], BLOCK):
            end = min(at + BLOCK, offsets[g + 1])
            b = g + offsets[g] // BLOCK + (at - offsets[g]) // BLOCK
            for c in range(C):
                codes[c, b * BLOCK:b * BLOCK + end - at], scale[b, c] = _block(x[at:end, c])
    return codes, scale


def b128_weights(w, num_experts):
    """w float32 [E*n][k] -> codes [E*n][k], codes_t [E*k][n], scale [E][nb][kb]."""
    n, k = w.shape[0] // num_experts, w.shape[1]
    x = w.reshape(num_experts, n, k)
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    codes, scale = np.zeros(x.shape, np.uint8), np.zeros((num_experts, nb, kb), np.float32)
    for e in range(num_experts):
        for i in range(nb):
            for j in range(kb):
                s = (e, slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                codes[s], scale[e, i, j] = _block(x[s])
    return codes.reshape(-1, k), np.ascontiguousarray(codes.transpose(0, 2, 1)).reshape(-1, n), scale


def b128_value(codes, scale):
    """Values of row-form codes [R][C], scale [blocks][R]."""
    return e4m3_decode(codes) * np.repeat(scale.astype(np.float64), BLOCK, 0)[:codes.shape[1]].T


def b128_weight_value(codes, scale):
    """Values of one expert's codes [r][c] with scale [r blocks][c blocks]."""
    s = np.repeat(np.repeat(scale.astype(np.float64), BLOCK, 0), BLOCK, 1)
    return e4m3_decode(codes) * s[:codes.shape[0], :codes.shape[1]]


def b128_gemm_fwd(a_q, w_q, offsets, n):
    """(y, sum of |products|) [M][n]; rows past offsets[-1] are zero."""
    a = b128_value(*a_q)
    y = np.zeros((a.shape[0], n))
    mag = np.zeros_like(y)
    for e in range(len(offsets) - 1):
        s = slice(offsets[e], offsets[e + 1])
        w = b128_weight_value(w_q[0][e * n:(e + 1) * n], w_q[1][e])
        y[s] = a[s] @ w.T
        mag[s] = np.abs(a[s]) @ np.abs(w).T
    return y, mag


def b128_gemm_dgrad(dy_q, wt_codes, w_scale, offsets, k):
    a = b128_value(*dy_q)
    y = np.zeros((a.shape[0], k))
    mag = np.zeros_like(y)
    for e in range(len(offsets) - 1):
        s = slice(offsets[e], offsets[e + 1])
        w = b128_weight_value(wt_codes[e * k:(e + 1) * k], w_scale[e].T)
        y[s] = a[s] @ w.T
        mag[s] = np.abs(a[s]) @ np.abs(w).T
    return y, mag


def b128_gemm_wgrad(dyt_q, xt_q, offsets):
    dy, x = b128_value(*dyt_q), b128_value(*xt_q)
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[0], x.shape[0]))
    mag = np.zeros_like(dw)
    for e in range(E):
        c0 = BLOCK * (e + offsets[e] // BLOCK)
        s = slice(c0, c0 + offsets[e + 1] - offsets[e])
        dw[e] = dy[:, s] @ x[:, s].T
        mag[e] = np.abs(dy[:, s]) @ np.abs(x[:, s]).T
    return dw, mag
