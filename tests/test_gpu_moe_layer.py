"""The example layer, forward, backward and decoding, against the layer's
formula in 64 bits without quantization, on the layer's own choice of experts.

Bounds, before any run: an E4M3 code is off by up to 2^-4 of its value, evenly
spread over a step whose size relative to the value runs from 2^-3 to 2^-4: an
rms of about 0.026.  Errors of a product's two operands are independent of each
other and of the signs in its sums, so a product adds sqrt(2) * 0.026 of its
Frobenius norm, and a result that n quantized operands lie on the way of is off
by about 0.026 sqrt(n) (the bf16 roundings between, 2^-9, do not count).  Twice
that is allowed."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def close(got, ref, n):
    got = got.double().cpu().reshape(ref.shape)
    err = float((got - ref).norm() / ref.norm())
    assert err <= 2 * 0.026 * n ** 0.5, (err, n)


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inner", [(200, 8, 2, 256, 128), (333, 12, 4, 272, 144), (1, 4, 2, 128, 128)])
def test_layer(bsq_gpu, tokens, experts, top_k, hidden, inner):
    from moe_layer import MoELayer
    layer = MoELayer(experts, hidden, inner, top_k, loss_coef=0.05)
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g).bfloat16()
    dy = torch.randn(tokens, hidden, generator=g).bfloat16()
    mask = torch.ones(tokens, dtype=torch.uint8)
    mask[3:7] = 0
    y, loss = layer.forward(x.cuda(), mask=mask.cuda())
    ids = layer.saved[2].cpu().long()
    assert (ids[mask == 0] == -1).all() and (ids[mask == 1] >= 0).all()
    dx, drouter, dgu, ddn = layer.backward(dy.cuda(), torch.full((1,), 1.5, device="cuda"))

    X = x.double().requires_grad_()
    R = layer.router.double().cpu().requires_grad_()
    GU = layer.gate_up.double().cpu().view(experts, 2 * inner, hidden).requires_grad_()
    D = layer.down.double().cpu().view(experts, hidden, inner).requires_grad_()
    p = torch.softmax(X @ R.t(), 1)
    live = mask.bool()
    chosen = torch.zeros(tokens, experts, dtype=torch.bool)
    chosen[live] = torch.zeros_like(chosen[live]).scatter_(1, ids[live], True)
    w = torch.where(chosen, p, 0.0)
    w = w / torch.where(live, w.sum(1), 1.0)[:, None]
    ref = torch.zeros(tokens, hidden, dtype=torch.float64)
    for e in range(experts):
        on = chosen[:, e].nonzero()[:, 0]
        z = X[on] @ GU[e].t()
        ref = ref.index_add(0, on, w[on, e:e + 1] * ((torch.nn.functional.silu(z[:, :inner]) * z[:, inner:]) @ D[e].t()))
    V = live.sum()
    balance = 0.05 * experts / top_k * (chosen.double().sum(0) * torch.where(live[:, None], p, 0.0).sum(0)).sum() / V ** 2
    ((ref * dy.double()).sum() + 1.5 * balance).backward()
    assert abs(float(loss) - float(balance.detach())) <= 2.0 ** -12 * float(balance.detach())  # (the logits are f32 products here)
    close(y, ref.detach(), 5)             # x, gate_up twice (gate and up), h, down
    close(ddn, D.grad, 5)                 # dye; x, gate_up twice, h
    close(dgu, GU.grad, 7)                # dye, down; gate, up; dgu, x
    close(dx, X.grad, 8)                  # the same, gate_up, and the router's part
    close(drouter, R.grad, 8)
    assert (y[mask == 0] == 0).all() and (dx[mask == 0] == 0).all()


def test_decoding_matches_the_batch(bsq_gpu):
    """A token's output through the form for few rows: the same codes and scales, sums in another order."""
    from moe_layer import MoELayer
    layer = MoELayer(16, 512, 256, 4)
    x = torch.randn(600, 512, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    full, _ = layer.forward(x, train=False)
    for n in (1, 8):
        y, _ = layer.forward(x[:n], train=False)
        # gu may round to another bf16, h to another code: a few elements differ by their step
        err = (y.float() - full[:n].float()).norm() / full[:n].float().norm()
        assert float(err) <= 0.026


def test_step_in_a_graph(bsq_gpu):
    """Forward and backward captured, replayed on new inputs, against the eager step."""
    from moe_layer import MoELayer
    layer = MoELayer(8, 256, 128, 2)
    g = torch.Generator().manual_seed(9)
    one = torch.ones(1, device="cuda")
    x = torch.randn(96, 256, generator=g).bfloat16().cuda()
    dy = torch.randn(96, 256, generator=g).bfloat16().cuda()

    def step():
        y, loss = layer.forward(x)
        return (y, loss) + layer.backward(dy, one)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        x.copy_(torch.randn(96, 256, generator=g).bfloat16())
        dy.copy_(torch.randn(96, 256, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
