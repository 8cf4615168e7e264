"""Logits far from 0: finite masks of a vocabulary, and rows whose every logit is large."""
import pytest
import torch

import head_device as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
LOWEST = torch.finfo(torch.bfloat16).min
MOST = torch.finfo(torch.float32).max
# tokens, vocabulary: logits in tiles of 64, 128 (on the caller's x, and on a copy) and 256 columns
WIDTHS = [(20, 1500), (100, 33000), (300, 9001), (1000, 12500)]


def f32(t):
    """In binary32, as numbers of 64 bits (what lies beyond it is infinite)."""
    return t.float().double()


@pytest.mark.parametrize("T,V", WIDTHS)
@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("value", [-1e9, -1e10, -1e12, -1e20, -1e30, LOWEST])
def test_masked_vocabulary(bsq_gpu, T, V, distill, value):
    """x ends in a one, against a finite mask value in the rows of w that are not to be sampled: single columns, and
    whole groups of 16, 64, 256 and 4096 (as far as there are). Some targets are masked too."""
    b = bsq_gpu
    H = 72
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=gen, device="cuda") * 0.2).bfloat16()
    x[:, -1] = 1.0
    out = torch.rand(V, generator=gen, device="cuda") < 0.2
    for n, at in ((16, 32), (64, 128), (256, 512), (4096, 8192)):
        out[at:at + n] = True
    w[:, -1] = torch.where(out, value, 0.0)
    free = torch.where(~out)[0]
    lab = free[torch.randint(0, len(free), (T,), generator=gen, device="cuda")].int()
    lab[5::7] = -1
    lab[3::7] = torch.where(out)[0][torch.randint(0, int(out.sum()), (len(lab[3::7]),), generator=gen, device="cuda")].int()
    ids = torch.stack([lab, torch.where(lab >= 0, free[:T].int(), -1)], 1)
    tl = torch.randn(T, 2, generator=gen, device="cuda")
    ones = torch.ones(T, device="cuda")
    for scale in (1.0, 0.5, 0.8, 1.25):
        i, q = ref.teacher_targets(ids, tl, V) if distill else ref.label_targets(lab, V)
        loss, lse, at, z = ref.forward(x, w, i, q, scale)
        if distill:  # (of logits that are outputs, and so numbers of 32 bits)
            loss = torch.where(q > 0, q * (torch.log(q.clamp(min=1e-300)) - f32(at) + lse[:, None]), 0.0).sum(1)
            got = b.bsq_linear_distill(x, w, ids, tl, scale=scale)
        else:
            got = b.bsq_linear_ce(x, w, lab, scale=scale)
        on = lab >= 0
        lse = torch.where(on, lse, 0.0)
        # a free logit is a chain of H / 32 matrix instructions, each summing 32 products: (H / 32 + 32) roundings of the
        # sum of magnitudes at most; lse has those of the largest, of an exponential's argument and of the merge
        dz = scale * (H / 32 + 32) * U * (x[:, :-1].abs().float() @ w[:, :-1].abs().float().t()).amax(1).double()
        tail = (64 + V / 1024) * U + 4 * U * lse.abs()
        assert torch.isneginf(got[1][~on]).all() and (got[0][~on] == 0).all()
        assert ((got[1].double() - lse).abs() <= dz + tail)[on].all()
        # (a masked target's logit is the mask's, but for its own rounding; q sum to 1, with 16 roundings)
        far = at.abs().amax(1)
        want, g = f32(loss), got[0].double()
        tol = 2 * dz + tail + 32 * U * (1 + far + lse.abs())
        inf = torch.isinf(want)
        assert (torch.isinf(g) == inf)[on].all() and ((g - want).abs() <= tol)[on & ~inf].all()
        if distill:
            d, zi = got[2].double(), f32(at)
            same = torch.where(torch.isinf(zi), d == zi, (d - zi).abs() <= dz[:, None] + 2 * U * zi.abs())
            assert (same | ~on[:, None]).all()
            dx, dw = b.bsq_linear_distill_bwd(x, w, ids, tl, got[1], dloss=ones, scale=scale, dw_dtype=b.BSQ_F32)
        else:
            dx, dw = b.bsq_linear_ce_bwd(x, w, lab, got[1], dloss=ones, scale=scale, dw_dtype=b.BSQ_F32)
        gz, size = ref.logit_gradient(z, i, q, ones, 0 * ones, scale)
        live = torch.where(on[:, None], x, 0).double()
        # (lse's error and the logit's are those of p, relatively; 128 roundings for q, the exponentials and g's three parts,
        # and the sum's: one for each of T / 32 matrix instructions, 32 within them)
        tol = size.t() @ ((2 * dz + tail + (160 + T / 32) * U)[:, None] * live.abs())
        assert ((dw.double() - gz.t() @ live).abs() <= tol).all()
        assert (dx[~on] == 0).all()
        want = (gz @ w.double())[on, :-1]
        assert (dx.double()[on, :-1] - want).norm() <= 2.0 ** -7 * want.norm()  # bf16 outputs, g in bf16 or a pair


@pytest.mark.parametrize("T,V", WIDTHS)
@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("value", [1e5, 1e7, 1e9, 1e10, 1e20, 1e30, -LOWEST])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_rows(bsq_gpu, T, V, distill, value, sign):
    """Every logit of the row is far from 0, and exact (one product): the largest ones tie."""
    b = bsq_gpu
    H = 8
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 1] = 1.0
    x[::3, 1] = 0.5
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    top = torch.tensor(sign * value, device="cuda").bfloat16()
    if sign < 0:
        top = (top.float() * 0.875).bfloat16()
    low = (top.float() * (0.875 if sign > 0 else 1 / 0.875)).bfloat16()
    ties = torch.zeros(V, dtype=torch.bool, device="cuda")
    ties[torch.randint(0, V, (37,), generator=gen, device="cuda")] = True
    ties[V - 1] = ties[64:80] = True
    w[:, 1] = torch.where(ties, top, low)
    lab = torch.where(ties)[0][torch.randint(0, int(ties.sum()), (T,), generator=gen, device="cuda")].int()
    lab[1::5] = torch.where(~ties)[0][:len(lab[1::5])].int()
    tl = torch.zeros(T, 1, device="cuda")
    for scale in (1.0, 0.5, 0.8, 1.25):
        z = scale * x[:, 1:2].double() * w[None, :, 1].double()
        lse = torch.logsumexp(z, 1)
        at = z.gather(1, lab.long()[:, None])[:, 0]
        loss = lse - at
        # lse of numbers this size in 64 bits has an error of its own: the count of ties says it exactly
        tie = z.amax(1) == at
        loss = torch.where(tie, torch.log((z == at[:, None]).sum(1).double()), loss)
        if distill:
            if z.abs().max() > MOST:
                continue  # its logits are outputs, and beyond their type
            got = b.bsq_linear_distill(x, w, lab[:, None].contiguous(), tl, scale=scale)
            assert ((got[2][:, 0].double() - at).abs() <= U * at.abs()).all()
        else:
            got = b.bsq_linear_ce(x, w, lab, scale=scale)
        n = f32(lse)
        inf = torch.isinf(n)
        assert (torch.isinf(got[1]) == inf).all() and ((got[1].double() - n).abs() <= 4 * U * n.abs())[~inf].all()
        n = f32(loss)
        inf = torch.isinf(n)
        # equal terms' number to a few roundings, and a rounding or two of the distance from the largest; an output logit has
        # a rounding of its own, which shows beside the largest where that is not large
        tol = 128 * U * (1 + n.abs())
        if distill:
            tol = tol + 2 * U * torch.where(tie, at.abs().clamp(max=65536.0), at.abs())
        assert (torch.isinf(got[0]) == inf).all() and ((got[0].double() - n).abs() <= tol)[~inf].all()


@pytest.mark.parametrize("T,V", WIDTHS)
@pytest.mark.parametrize("value", [1e5, 1e9, 1e10, 1e20, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_rows_backward(bsq_gpu, T, V, value, sign):
    """One logit far above the others, all of them far from 0: its p is 1, the others' 0."""
    b = bsq_gpu
    H = 64
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(T), torch.arange(T) % 8] = 1.0
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    top = torch.tensor(sign * value, device="cuda").bfloat16().float()
    w[:, :8] = (top * (0.5 if sign > 0 else 2.0)).bfloat16()
    best = torch.randperm(V, generator=gen, device="cuda")[:8]
    w[best, torch.arange(8)] = top.bfloat16()
    best = best[torch.arange(T, device="cuda") % 8]
    lab = torch.where(torch.arange(T, device="cuda") % 3 == 0, best, (best + 5) % V).int()
    dloss = torch.rand(T, generator=gen, device="cuda") + 0.5
    rows = torch.arange(T, device="cuda")
    for scale in (1.0, 0.5, 0.8, 1.25):
        lse = b.bsq_linear_ce(x, w, lab, scale=scale)[1]
        g = torch.zeros(T, V, dtype=torch.float64, device="cuda")
        g[rows, best] += scale * dloss.double()
        g[rows, lab.long()] -= scale * dloss.double()
        dx, dw = b.bsq_linear_ce_bwd(x, w, lab, lse, dloss=dloss, scale=scale, dx_dtype=b.BSQ_F32, dw_dtype=b.BSQ_F32)
        # p is exactly 1 or 0, and g two products: a rounding each, and one for each of the sums' (T / 8 equal signs at most)
        want = g.t() @ x.double()
        assert ((dw.double() - want).abs() <= (8 + T / 32) * U * (g.abs().t() @ x.double())).all()
        want = g @ w.double()
        assert ((dx.double() - want).abs() <= 16 * U * (g.abs() @ w.double().abs())).all()


@pytest.mark.parametrize("T", [20, 300])
def test_p_is_at_most_one(bsq_gpu, T):
    """Equal largest logits, so large that their number does not show in lse: each has a p from 0 to 1."""
    b = bsq_gpu
    V, H = 1000, 8
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    lab = torch.zeros(T, dtype=torch.int32, device="cuda")
    for value in (1e6, -1e6, 1e9, -1e9, 1e20, -1e20):
        for scale in (1.0, 0.7):
            w[:, 0] = value
            lse = b.bsq_linear_ce(x, w, lab, scale=scale)[1]
            # with dlse alone, dw of column 0 is scale p, summed over the tokens
            p = b.bsq_linear_ce_bwd(x, w, lab, lse, dlse=torch.ones(T, device="cuda"), scale=scale, flags=b.BSQ_WGRAD,
                                    dw_dtype=b.BSQ_F32)[1][:, 0] / (scale * T)
            assert (p >= 0).all() and (p <= 1 + (T / 32 + 40) * U).all()


@pytest.mark.parametrize("T,V", WIDTHS)
@pytest.mark.parametrize("power", [27, 28, 29, 30, 31, 33])
@pytest.mark.parametrize("sign", [1, -1])
def test_neighbouring_far_logits(bsq_gpu, T, V, power, sign):
    """Logits of 2^27 to 2^33 that differ in their last bits, whose exponents a whole number of 24 bits still holds or no longer
    does: two products a logit, whose sum binary32 holds."""
    b = bsq_gpu
    gen = torch.Generator(device="cuda").manual_seed(power + V)
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    x[:, :2] = 1.0
    w = torch.zeros(V, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = sign * 2.0 ** power * (1 + T % 3 / 128)
    w[:, 1] = torch.randint(0, 250, (V,), generator=gen, device="cuda") * 2.0 ** (power - 23)
    z = w[:, 0].double() + w[:, 1].double()
    assert torch.equal(z, f32(z))
    lab = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
    for scale in (1.0, 0.5, 0.7, 0.8, 1.25):
        s = torch.tensor(scale, dtype=torch.float32).double().item()  # (as the call gets it)
        top = torch.logsumexp(s * (z - z.max()), 0)
        want = top - s * (z - z.max())[lab.long()]
        # the merge's roundings, and a few of the label's distance from the largest
        tol = (64 + V / 1024) * U + 8 * U * want
        ce, lse = b.bsq_linear_ce(x, w, lab, scale=scale)
        assert ((ce.double() - want).abs() <= tol).all()
        assert ((lse.double() - (s * z.max() + top)).abs() <= 4 * U * (s * z.max()).abs()).all()
        kl, same, at = b.bsq_linear_distill(x, w, lab[:, None].contiguous(), torch.zeros(T, 1, device="cuda"), scale=scale)
        assert ((kl.double() - want).abs() <= tol).all() and torch.equal(same, lse)
        assert torch.equal(at[:, 0], (s * z[lab.long()]).float())
