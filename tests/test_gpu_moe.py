"""Routing, dispatch and combine on the GPU against the 64-bit oracle.

Whole numbers are compared exactly.  Floating bounds, before any run: a
binary32 softmax term carries the rounding of its argument (|l - m| 2^-24, at
most 2^-17 for the |l - m| <= 100 drawn here), a few ulps of exp and the sum
of E terms: 2^-16 relative.  A balance loss is a sum of positive terms: the
same.  A logit gradient is a difference of such terms: 2^-15 of the sum of
their magnitudes, and half a step of the output type (bf16 2^-8)."""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

REL = 2.0 ** -16


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def within(got, ref, bound):
    """|got - ref| <= bound everywhere, with a short message where not."""
    d = np.abs(np.asarray(got, np.float64) - ref) - bound
    if d.size == 0:
        return
    i = np.unravel_index(np.argmax(d), d.shape)
    assert d.max() <= 0, f"at {i}: {np.asarray(got)[i]} for {ref[i]}, {d[i]} past the bound"


def logits_for(rng, T, E, dtype, spread=2.0):
    l = torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32)).to(dtype)
    return l


def check_route(bsq, l, K, bias=None, mask=None, normalize=True, scale=1.0, coef=0.01, seed=0):
    T, E = l.shape
    l64 = l.double().numpy()
    ref = moe.route(l64, K, bias=bias, mask=mask, normalize=normalize, scale=scale, coef=coef)
    ld = l.cuda()
    b = None if bias is None else dev(bias)
    m = None if mask is None else dev(mask)
    kw = dict(normalize=normalize, scale=scale, loss_coef=coef)
    ids, w, lse, counts, loss = bsq.bsq_moe_route(ld, K, bias=b, mask=m, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), ref[0])
    assert np.array_equal(counts.cpu().numpy(), ref[3])
    within(w.cpu().numpy(), ref[1], REL * np.abs(ref[1]) + 2.0 ** -126)
    got = lse.cpu().numpy().astype(np.float64)
    live = ref[2] > -np.inf
    assert np.array_equal(got > -np.inf, live)
    within(got[live], ref[2][live], REL + 2.0 ** -23 * np.abs(ref[2][live]))
    assert abs(float(loss) - ref[4]) <= REL * abs(ref[4]) + 2.0 ** -126  # binary32 holds nothing below
    rng = np.random.default_rng(seed + 99)
    dw, dl = rng.standard_normal((T, K)).astype(np.float32), np.float32(1.25)
    d = bsq.bsq_moe_route_bwd(ld, ids, w, lse, counts, dev(dw), dev(np.array([dl])), **kw)
    torch.cuda.synchronize()
    rd = moe.route_bwd(l64, ref[0], ref[3], dw, float(dl), normalize=normalize, scale=scale, coef=coef, mask=mask)
    mag = (np.abs(scale * dw) * (ref[0] >= 0)).sum(1, keepdims=True) + abs(coef * float(dl)) * E / K
    step = 2.0 ** -8 if l.dtype == torch.bfloat16 else 2.0 ** -24
    assert d.dtype == l.dtype
    within(d.double().cpu().numpy(), rd, step * np.abs(rd) + 2.0 ** -15 * mag)
    return ids, w, lse, counts, loss, d


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,K", [(1, 4, 2), (3, 64, 8), (64, 65, 4), (65, 128, 8), (200, 129, 6), (130, 256, 8),
                                   (97, 384, 8), (70, 385, 3), (40, 512, 16), (33, 1000, 64), (66, 1024, 1), (5, 1, 1)])
def test_route(bsq_gpu, T, E, K, dtype):
    rng = np.random.default_rng(T * 7 + E)
    l = logits_for(rng, T, E, dtype)
    bias = (rng.standard_normal(E) * 0.3).astype(np.float32)
    check_route(bsq_gpu, l, K, normalize=True, seed=T)
    check_route(bsq_gpu, l, K, bias=bias, normalize=False, scale=2.5, seed=T)


@pytest.mark.parametrize("T", [50, 300])
def test_route_masks_and_edges(bsq_gpu, T):
    """Padding that holds NaN, experts ruled out, rows with nothing left, the
    type's lowest value, infinities, ties across lanes."""
    rng = np.random.default_rng(T)
    E, K = 96, 6
    for dtype in (torch.bfloat16, torch.float32):
        l = logits_for(rng, T, E, dtype)
        l[rng.random((T, E)) < 0.5] = -np.inf
        l[1] = -np.inf
        l[2] = -np.inf
        l[2, [5, 77]] = 1.0
        l[3] = torch.finfo(dtype).min
        l[4] = 0.25                                   # every key equal
        l[5] = torch.finfo(dtype).min
        l[5, 90] = 3.0
        l[6, 10] = np.inf
        l[7, 11] = np.nan
        mask = (rng.random(T) < 0.8).astype(np.uint8)
        mask[1:8] = 1
        l[mask == 0] = np.nan
        for normalize in (True, False):
            out = check_route(bsq_gpu, l, K, mask=mask, normalize=normalize)
            assert out[0][4].tolist() == list(range(K)) and out[0][1].tolist() == [-1] * K
            assert out[0][2].tolist() == [5, 77] + [-1] * (K - 2)
        zero = np.zeros(T, np.uint8)
        out = check_route(bsq_gpu, l, K, mask=zero)
        assert float(out[4]) == 0.0 and (out[5] == 0).all()


def test_route_bias_lifts_negligible_experts(bsq_gpu):
    """Chosen experts whose share of the softmax underflows still get a normalized weight."""
    l = torch.zeros(9, 64)
    l[:, 0] = 300.0
    bias = np.zeros(64, np.float32)
    bias[[20, 40]] = 1000.0
    ids, w, *_ = check_route(bsq_gpu, l, 2, bias=bias, normalize=True)
    assert ids[0].tolist() == [20, 40] and w[0].tolist() == [0.5, 0.5]
    bias[3] = -np.inf
    bias[0] = -np.inf
    ids, *_ = check_route(bsq_gpu, l, 64, bias=bias, normalize=True)
    assert ids[0, 62:].tolist() == [-1, -1]


def test_route_strides_streams_and_repeats(bsq_gpu):
    rng = np.random.default_rng(11)
    big = logits_for(rng, 500, 103, torch.float32).cuda()
    for view in (big[:, 1:98], big[::2, :96], big[:, 2:66]):
        ref = bsq_gpu.bsq_moe_route(view.contiguous(), 4, loss_coef=0.1)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = bsq_gpu.bsq_moe_route(view, 4, loss_coef=0.1, stream=s)
        d = bsq_gpu.bsq_moe_route_bwd(view, *got[:4], got[1], got[4], loss_coef=0.1, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        assert torch.equal(d, bsq_gpu.bsq_moe_route_bwd(view.contiguous(), *ref[:4], ref[1], ref[4], loss_coef=0.1))
        assert all(torch.equal(a, b) for a, b in zip(ref, bsq_gpu.bsq_moe_route(view, 4, loss_coef=0.1)))


def test_route_no_tokens(bsq_gpu):
    l = torch.empty(0, 32, device="cuda")
    ids, w, lse, counts, loss = bsq_gpu.bsq_moe_route(l, 4, loss_coef=0.1)
    assert ids.shape == (0, 4) and counts.tolist() == [0] * 33 and float(loss) == 0.0
    assert bsq_gpu.bsq_moe_route_bwd(l, ids, w, lse, counts).shape == (0, 32)


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 384), (16, 8, 384), (100, 4, 7), (512, 8, 64), (513, 8, 64),
                                   (3000, 8, 384), (5000, 3, 1000), (40000, 8, 1024), (0, 2, 5)])
def test_dispatch(bsq_gpu, T, K, E):
    rng = np.random.default_rng(T + E)
    for lo, hi in ((0, E), (-1, E + 2), (0, max(1, E // 16)), (-5, 0)):
        ids = rng.integers(lo, hi, (T, K)).astype(np.int32) if hi > lo else np.full((T, K), -1, np.int32)
        got = bsq_gpu.bsq_moe_dispatch(dev(ids), E)
        torch.cuda.synchronize()
        for g, r in zip(got, moe.dispatch(ids, E)):
            assert np.array_equal(g.cpu().numpy(), r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,W", [(1, 1, 8), (5, 8, 64), (40, 3, 1032), (33, 9, 2048), (17, 17, 2056), (3, 8, 7168)])
def test_combine(bsq_gpu, T, K, W, dtype):
    """Sums of K terms and of W terms in binary32: (K + 2) and (W / 64 + 16) roundings of the sum of magnitudes."""
    rng = np.random.default_rng(T + W)
    ids = rng.integers(-1, 6, (T, K)).astype(np.int32)
    off, _, slot = moe.dispatch(ids, 6)
    M = T * K
    pad = 8
    ye = torch.from_numpy(rng.standard_normal((M, W + pad)).astype(np.float32)).to(dtype)
    ye[off[-1]:] = np.nan                      # rows no choice owns are never used
    dy = torch.from_numpy(rng.standard_normal((T, W)).astype(np.float32)).to(dtype)
    w = rng.random((T, K)).astype(np.float32)
    yv, dv = ye.cuda()[:, :W], dy.cuda()
    y64 = np.nan_to_num(ye[:, :W].double().numpy())
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for weights in (w, None):
        wd = None if weights is None else dev(weights)
        y = bsq_gpu.bsq_moe_combine(yv, dev(slot), wd)
        dye, dw = bsq_gpu.bsq_moe_combine_bwd(dv, yv, dev(slot), wd, offsets=dev(off))
        torch.cuda.synchronize()
        ref, mag = moe.combine(y64, slot, weights), moe.combine(np.abs(y64), slot, weights)
        within(y.double().cpu().numpy(), ref, step * np.abs(ref) * 1.01 + (K + 2) * 2.0 ** -24 * mag)
        rye, rdw = moe.combine_bwd(dy.double().numpy(), y64, slot, weights)
        within(dye.double().cpu().numpy(), rye, step * np.abs(rye) * 1.01 + 2.0 ** -126)
        _, mdw = moe.combine_bwd(np.abs(dy.double().numpy()), np.abs(y64), slot, weights)
        within(dw.cpu().numpy(), rdw, (W / 64 + 16) * 2.0 ** -24 * mdw)
    # slots outside the rows count as none
    bad = slot.copy()
    bad[0, 0] = M + 5
    assert torch.equal(bsq_gpu.bsq_moe_combine(yv, dev(bad)),
                       bsq_gpu.bsq_moe_combine(yv, dev(np.where(bad >= M, -1, bad).astype(np.int32))))


def test_combine_without_rows_or_ye(bsq_gpu):
    slot = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    y = bsq_gpu.bsq_moe_combine(torch.empty(0, 16, device="cuda"), slot)
    assert (y == 0).all()
    slot[1, 0] = 3
    dy = torch.ones(4, 16, device="cuda")
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    dye, dw = bsq_gpu.bsq_moe_combine_bwd(dy, None, slot, offsets=off, m_total=8, need_dweights=False)
    assert dw is None and (dye[1:3] == 0).all() and (dye[4:] == 0).all()


@pytest.mark.parametrize("E,K", [(384, 8), (1024, 20), (256, 6), (130, 5)])
def test_route_choices_that_share_a_lane(bsq_gpu, E, K):
    """The first choices at positions 2 l and 2 l + 1 of every 128, in any order, tied
    among each other, with others before and after them, and zeros of both signs."""
    rng = np.random.default_rng(E + K)
    T = 80
    l = logits_for(rng, T, E, torch.float32, spread=1.0)
    for t in range(T):
        lane = int(rng.integers(0, 64))
        at = np.array([128 * c + 2 * lane + i for c in range(-(-E // 128)) for i in (0, 1)])
        at = torch.from_numpy(at[at < E])
        if t % 4 == 0:
            l[t, at] = 10.0 + torch.from_numpy(rng.permutation(len(at)).astype(np.float32))
        elif t % 4 == 1:
            l[t, at] = 10.0                                             # all tied, in one lane
            l[t, torch.from_numpy(rng.integers(0, E, 3))] = 10.0        # and elsewhere
        elif t % 4 == 2:
            l[t] = torch.from_numpy(rng.choice([0.0, -0.0, -1.0], E).astype(np.float32))
        else:
            l[t] = torch.from_numpy(np.round(rng.standard_normal(E) * 2).astype(np.float32))
    bias = np.where(rng.random(E) < 0.5, np.float32(-0.0), np.float32(0.0))
    check_route(bsq_gpu, l, K, bias=None, normalize=True, seed=1)
    check_route(bsq_gpu, l, K, bias=bias, normalize=False, seed=2)
    check_route(bsq_gpu, l.bfloat16(), K, bias=np.round(rng.standard_normal(E)).astype(np.float32), seed=3)
