"""Cross entropy and top-logit distillation at the output head in each form of their kernels, against the formula in 64
bits on the device."""
import pytest
import torch

import head_device as ref
from head_forms import BATCH, FORMS, PIECES, STREAMED, THREE_PARTS

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


class Data:
    def __init__(self, T, V, H, K=0, scale=0.8, masked=0.15):
        self.T, self.V, self.H, self.K, self.scale = T, V, H, K, scale
        gen = torch.Generator(device="cuda").manual_seed(T + V + K)

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.x = normal(T, H).bfloat16()
        self.w = (normal(V, H) * (2 / H ** 0.5)).bfloat16()
        off = torch.rand(T, generator=gen, device="cuda") < masked
        self.dloss, self.dlse = torch.rand(T, generator=gen, device="cuda") + 0.5, 0.3 * normal(T)
        if K:
            self.ids = torch.randint(0, V, (T, K), generator=gen, device="cuda").int()
            self.ids[:, -1] = self.ids[:, 0]
            self.ids[0, 0] = V - 1
            self.ids[torch.arange(K, device="cuda") >= 1 + torch.randint(0, K, (T, 1), generator=gen, device="cuda")] = -1
            self.ids[off] = V
            self.tl = normal(T, K) * 3
            self.i, self.q = ref.teacher_targets(self.ids, self.tl, V, scale=0.7)
        else:
            self.lab = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
            self.lab[0], self.lab[-1] = V - 1, 0
            self.lab[off] = -100
            self.i, self.q = ref.label_targets(self.lab, V)
        self.x[off] = float("nan")
        self.on = ~off

    def rows(self, rows):
        d = Data.__new__(Data)
        d.__dict__.update(self.__dict__)
        d.x = self.x[rows]
        for name in ("ids", "tl") if self.K else ("lab",):
            setattr(d, name, getattr(self, name)[rows])
        return d

    def forward(self, b):
        if self.K:
            return b.bsq_linear_distill(self.x, self.w, self.ids, self.tl, scale=self.scale, teacher_scale=0.7)
        return b.bsq_linear_ce(self.x, self.w, self.lab, scale=self.scale)

    def backward(self, b, lse, dx32, dw32, flags=3, dloss=True):
        kw = dict(dloss=self.dloss if dloss else None, dlse=self.dlse, scale=self.scale, flags=flags,
                  dx_dtype=b.BSQ_F32 if dx32 else b.BSQ_BF16, dw_dtype=b.BSQ_F32 if dw32 else b.BSQ_BF16)
        if self.K:
            return b.bsq_linear_distill_bwd(self.x, self.w, self.ids, self.tl, lse, teacher_scale=0.7, **kw)
        return b.bsq_linear_ce_bwd(self.x, self.w, self.lab, lse, **kw)

    def check(self, b, types):
        """Both passes; the gradients in each pair of types (f32 or not)."""
        loss, lse, at, z = ref.forward(self.x, self.w, self.i, self.q, self.scale)
        got = self.forward(b)
        on = self.on
        x = torch.where(on[:, None], self.x, 0)
        # a logit: a chain of H / 32 matrix instructions, each summing 32 products: (H / 32 + 32) roundings at most of the sum of
        # magnitudes; lse: the largest of those, an exponential's argument's, the merge's
        dz = self.scale * (self.H / 32 + 32) * U * (x.float().abs() @ self.w.float().abs().t()).amax(1).double()
        n = torch.where(on, lse, 0.0)
        tail = (64 + self.V / 1024) * U + 4 * U * n.abs()
        assert torch.isneginf(got[1][~on]).all() and (got[0][~on] == 0).all()
        assert ((got[1].double() - n).abs() <= dz + tail)[on].all()
        # (q's errors, of teacher logits up to 16: 64 roundings of a loss's terms)
        tol = self.q.sum(1) * (2 * dz + tail) + 64 * U * (self.q * ((self.q.clamp(min=1e-300)).log().abs() + at.abs() + n.abs()[:, None] + 1)).sum(1)
        assert ((got[0].double() - loss).abs() <= tol)[on].all()
        if self.K:
            some = (self.ids >= 0) & (self.ids < self.V)
            assert (got[2][~some] == 0).all()
            assert ((got[2].double() - at).abs() <= dz[:, None] + 2 * U * at.abs())[some].all()
        g, size = ref.logit_gradient(z, self.i, self.q, self.dloss, self.dlse, self.scale)
        del z
        x, w = x.double(), self.w.double()
        want = g @ w, g.t() @ x
        # errors of g: those of a logit and of lse (p's, relatively), 128 roundings for q and the exponential; then each
        # product's: one for each of its chain's matrix instructions, 32 within one, and one for each of 64 partial sums
        near = size * (2 * dz + tail + 128 * U)[:, None]
        base = near @ w.abs() + (self.V / 32 + 96) * U * (g.abs() @ w.abs()), \
            near.t() @ x.abs() + (self.T / 32 + 96) * U * (g.abs().t() @ x.abs())
        rounded = g.abs() @ w.abs(), g.abs().t() @ x.abs()
        squares = ((g ** 2) @ (w ** 2)).sum(), ((g ** 2).t() @ (x ** 2)).sum()
        for kinds in types:
            d = self.backward(b, got[1], *kinds)
            for flag, one, full, base_, rounded_, square, kind in zip((1, 2), d, want, base, rounded, squares, kinds):
                alone = self.backward(b, got[1], *kinds, flags=flag)
                eps_g = 2.0 ** -24 if kind else 2.0 ** -16 if self.T <= 256 else 2.0 ** -8
                eps = 2.0 ** -24 if kind else 2.0 ** -8
                for out in (one, alone[flag - 1]):  # (one gradient alone may be split otherwise)
                    far = out.double() - full
                    assert (far.abs() <= 1.01 * (base_ + eps_g * rounded_ + eps * full.abs())).all()
                    if not kind:  # roundings are independent, and at most half a step: 1 / sqrt(3) of it on average at most
                        assert far.norm() <= 1.2 * ((eps_g ** 2 * square + eps ** 2 * (full ** 2).sum()) / 3).sqrt()
                assert alone[2 - flag] is None
            assert (d[0][~on] == 0).all()


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("K", [0, 9])
def test_forms(bsq_gpu, name, K):
    Data(*FORMS[name][:3], K).check(bsq_gpu, [(0, 0), (1, 1), (0, 1), (1, 0)])


@pytest.mark.parametrize("name", STREAMED)
@pytest.mark.parametrize("K", [0, 5])
def test_streamed(bsq_gpu, name, K):
    Data(*STREAMED[name][:3], K).check(bsq_gpu, [(0, 0), (1, 1)])


@pytest.mark.parametrize("K", [0, 9])
def test_pieces(bsq_gpu, K):
    Data(*PIECES[:3], K).check(bsq_gpu, [(1, 1), (0, 0)])


@pytest.mark.parametrize("K", [0, 7])
def test_bits_across_tile_widths(bsq_gpu, K):
    """loss and lse (and logits) of a token in batches whose tiles are 64, 128 and 256 columns wide."""
    T, V, blocks = BATCH
    d = Data(T, V, 136, K)
    full = d.forward(bsq_gpu)
    for n in blocks:
        for first in {0, T - n}:
            rows = torch.arange(first, first + n, device="cuda")
            for got, want in zip(d.rows(rows).forward(bsq_gpu), full):
                assert torch.equal(got, want[rows])


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("K", [0, 3])
def test_three_parts(bsq_gpu, name, K):
    """f32 gradients take all of g: dx shows single values of g, as w holds one number a column, and dw sums over tokens.
    With dlse alone, g = scale dlse p, whose error is lse's rounding (2^-21: lse is below 16), z - lse's (2^-21), its product
    with log2 e's (2^-21 ln 2), and a few of 2^-24: 1.5e-6 at most, and so is its norm's; of g in two parts the rest is 2.4e-6
    by itself."""
    T, V, H = FORMS[name][:3]
    d = Data(T, V, H, K, scale=1.0)
    gen = torch.Generator(device="cuda").manual_seed(T)
    rows = torch.randperm(V, generator=gen, device="cuda")[:H]
    d.w.zero_()
    d.w[rows, torch.arange(H, device="cuda")] = (torch.rand(H, generator=gen, device="cuda") / 2 + 0.5).bfloat16()
    z = ref.forward(d.x, d.w, d.i, d.q)[3]
    g, _ = ref.logit_gradient(z, d.i, d.q, 0 * d.dloss, d.dlse)
    x = torch.where(d.on[:, None], d.x, 0).double()
    lse = d.forward(bsq_gpu)[1]
    for kinds in ((1, 1), (0, 1), (1, 0)):
        got = d.backward(bsq_gpu, lse, *kinds, dloss=False)
        for out, want, kind in zip(got, (g @ d.w.double(), g.t() @ x), kinds):
            if kind:
                assert (out.double() - want).norm() <= THREE_PARTS * want.norm()


@pytest.mark.parametrize("T,V,H", [(20, 900, 72), (100, 4001, 328), (1100, 1000, 72)])
def test_graph_of_lists(bsq_gpu, T, V, H):
    """Distillation's two passes captured together and replayed on other lists, with eager calls between; two graphs share
    a workspace."""
    b = bsq_gpu
    cases = [Data(T, V, H, 6) for _ in range(2)]
    cases[1].ids, cases[1].tl = cases[1].ids.flip(0).contiguous(), cases[1].tl.flip(0).contiguous()
    cases[1].x = cases[1].x.flip(0).contiguous()
    x, w, ids, tl, dloss = (t.clone() for t in (cases[0].x, cases[0].w, cases[0].ids, cases[0].tl, cases[0].dloss))
    room = max(b.bsq_linear_loss_workspace_size(T, H, V, 6, flags) for flags in (0, 3))
    ws = torch.empty(room, dtype=torch.uint8, device="cuda")

    def step():
        out = b.bsq_linear_distill(x, w, ids, tl, workspace=ws)
        return (*out, *b.bsq_linear_distill_bwd(x, w, ids, tl, out[1], dloss=dloss, workspace=ws))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for i in (0, 1, 0, 1, 1):
        c = cases[i]
        for to, of in ((x, c.x), (ids, c.ids), (tl, c.tl)):
            to.copy_(of)
        dloss.mul_(1.5)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for g, out in graphs:
            for t in out:
                t.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, e) for a, e in zip(out, want))
