"""Routing of so many tokens that a wave takes several of them, with padding between,
and dispatch of so many choices that a wave reads some of them again: every row
against 64-bit references on the GPU (the bounds that test_gpu_moe.py states)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

REL = 2.0 ** -16


def reference(l, K, bias, mask, normalize, scale, coef, dw, dl):
    """ids, weights, lse, counts, loss and the logits' gradient."""
    T, E = l.shape
    x = torch.where(torch.isnan(l), -math.inf, l.float())
    x = torch.where(mask[:, None], x, -math.inf)
    key, order = torch.sort(x + bias, dim=1, descending=True, stable=True)
    ok = key[:, :K] > -math.inf
    ids = torch.where(ok, order[:, :K], -1)
    live = ok.any(1)
    x = x.double()
    p = torch.where(live[:, None], torch.softmax(x, 1), 0.0)
    at = order[:, :K]
    share = torch.where(ok, p.gather(1, at), 0.0)
    q = share / share.sum(1, keepdim=True).clamp(min=1e-300)
    w = scale * (q if normalize else share)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device).index_add_(
        0, torch.where(ok, at, E).flatten(), torch.ones(T * K, dtype=torch.int64, device=l.device))
    counts[E] = V = int(live.sum())
    f = counts[:E].double()
    loss = coef * E / (K * V) * float((f * p.sum(0)).sum()) / V
    u = (dl * coef * E / (K * V * V) * f).expand(T, E).contiguous()
    g = torch.zeros(T, E, dtype=torch.float64, device=l.device)
    dw = scale * torch.where(ok, dw.double(), 0.0)
    if normalize:
        g.scatter_add_(1, at, torch.where(ok, q * (dw - (q * dw).sum(1, keepdim=True)), 0.0))
    else:
        u = u.scatter_add(1, at, dw)
    g += p * (u - (p * u).sum(1, keepdim=True))
    return ids, w, torch.where(live, torch.logsumexp(x, 1), -math.inf), counts, loss, g


def within(got, ref, bound):
    assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() - bound).max())


@pytest.mark.parametrize("T,E,K", [(4097, 64, 4), (9001, 130, 6), (20000, 384, 8), (12345, 1000, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize,masked", [(True, 0.05), (False, 0.05), (True, 0.5), (False, 0.5)])
def test_route(bsq_gpu, T, E, K, dtype, normalize, masked):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = torch.randn(T, E, generator=g, device="cuda") * 2
    groups = torch.rand(T, 8, generator=g, device="cuda") < 0.5
    l = l.masked_fill(groups[:, torch.arange(E, device="cuda") * 8 // E], -math.inf)  # (some tokens keep fewer than K, or none)
    mask = torch.rand(T, generator=g, device="cuda") >= masked
    mask[-40:-20] = False
    l[~mask] = math.nan
    l = l.to(dtype)
    bias = torch.randn(E, generator=g, device="cuda") * 0.3
    dw, dl = torch.randn(T, K, generator=g, device="cuda"), 1.25
    how = dict(normalize=normalize, scale=1.5, loss_coef=0.01)
    ids, w, lse, counts, loss = bsq_gpu.bsq_moe_route(l, K, bias=bias, mask=mask, **how)
    d = bsq_gpu.bsq_moe_route_bwd(l, ids, w, lse, counts, dw, torch.full((1,), dl, device="cuda"), **how)
    ri, rw, rl, rc, rloss, rd = reference(l, K, bias, mask, normalize, 1.5, 0.01, dw, dl)
    assert torch.equal(ids, ri.int()) and torch.equal(counts, rc.int())
    within(w, rw, REL * rw + 2.0 ** -126)
    live = rl > -math.inf
    assert torch.equal(lse > -math.inf, live)
    within(lse[live], rl[live], REL + 2.0 ** -23 * rl[live].abs())
    assert abs(float(loss) - rloss) <= REL * rloss
    mag = (1.5 * dw.abs().double() * (ri >= 0)).sum(1, keepdim=True) + 0.01 * dl * E / K
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert d.dtype == dtype
    within(d, rd, step * rd.abs() + 2.0 ** -15 * mag)
    # one gradient at a time: none of the other's in it
    only = bsq_gpu.bsq_moe_route_bwd(l, ids, w, lse, counts, None, torch.full((1,), dl, device="cuda"), **how)
    rd = reference(l, K, bias, mask, normalize, 1.5, 0.01, dw * 0, dl)[5]
    # p (u - sum p u), both u at most its largest
    within(only, rd, step * rd.abs() + 2.0 ** -15 * 0.01 * dl * E / K * int(rc[:E].max()) / int(rc[E]) ** 2 + 2.0 ** -126)
    only = bsq_gpu.bsq_moe_route_bwd(l, ids, w, lse, counts, dw, None, **how)
    rd = reference(l, K, bias, mask, normalize, 1.5, 0.0, dw, dl)[5]
    within(only, rd, step * rd.abs() + 2.0 ** -15 * mag)


@pytest.mark.parametrize("T,K,E", [(65537, 8, 384), (131072, 4, 64), (131073, 4, 1000), (400000, 8, 256)])
@pytest.mark.parametrize("lo,over", [(0, 0), (-3, 5), (-300, 0)])
def test_dispatch(bsq_gpu, T, K, E, lo, over):
    """More than 524288 choices: a wave's range is longer than what it holds in registers."""
    g = torch.Generator(device="cuda").manual_seed(T + lo)
    ids = torch.randint(lo, E + over, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[T // 3:T // 3 + 5000] = -1                # padding in one piece
    ids[T // 2:T // 2 + 9000, 0] = E // 2         # and one expert for many tokens in a row
    offsets, row_index, slot = bsq_gpu.bsq_moe_dispatch(ids, E)
    bucket = torch.where((ids < 0) | (ids >= E), E, ids).flatten()
    grouped, order = torch.sort(bucket, stable=True)
    ends = torch.bincount(bucket, minlength=E + 1)[:E].cumsum(0).int()
    assert torch.equal(offsets, torch.cat([ends.new_zeros(1), ends]))
    ok = grouped < E
    assert torch.equal(row_index, torch.where(ok, order // K, -1).int())
    ref = torch.empty_like(bucket)
    ref[order] = torch.where(ok, torch.arange(T * K, device="cuda"), -1).int()
    assert torch.equal(slot.flatten(), ref)
