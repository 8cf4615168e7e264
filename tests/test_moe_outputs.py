"""The outputs of routing and dispatch are tensors of their own, also where one allocation holds several."""
import pytest
import torch


def own(tensors):
    """An in-place change of one tensor is none of another."""
    for t in tensors:
        others = [(o, o._version) for o in tensors if o is not t]
        before = [o.clone() for o, _ in others]
        t.zero_()
        assert all(o._version == v and torch.equal(o, b) for (o, v), b in zip(others, before))


def test_carve():
    import block_scaled_precision_bsq_amd as bsq
    for scratch in (0, 512):
        out = bsq._carve(None, torch.int32, "cpu", (5, 3, 7), scratch)[:3]
        assert [t.numel() for t in out] == [5, 3, 7]
        for i, t in enumerate(out):
            t.fill_(i + 1)
        own(out)
    # an output saved for a backward pass, another one changed in place before it
    a, b = bsq._carve(None, torch.float32, "cpu", (4, 4))
    a.fill_(3.0)
    x = torch.ones(4, requires_grad=True)
    y = (x * a).sum()
    b.add_(1)
    y.backward()
    assert torch.equal(x.grad, a)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [16, 5000])
def test_outputs(bsq_gpu, tokens):
    l = torch.randn(tokens, 384, generator=torch.Generator().manual_seed(1)).cuda()
    ids, w, lse, counts, loss = bsq_gpu.bsq_moe_route(l, 8, loss_coef=0.1)
    # what is kept for a log does not keep the tokens' outputs or a large workspace
    assert counts.untyped_storage().nbytes() <= 1 << 14 and loss.untyped_storage().nbytes() <= 1 << 14
    offsets, row_index, slot = bsq_gpu.bsq_moe_dispatch(ids, 384)
    x = torch.ones(tokens, 8, device="cuda", requires_grad=True)
    y = (x * w).sum()
    counts.zero_()
    y.backward()
    assert torch.equal(x.grad, w)
    own([ids, w, lse, counts, loss])
    own([offsets, row_index, slot])
