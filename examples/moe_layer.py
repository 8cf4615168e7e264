"""A mixture-of-experts layer on the library's routing, dispatch, FP8B128 and
combine entry points: a training step (forward and backward) and a decoding
step.

    python examples/moe_layer.py [--tokens T] [--experts E] [--top-k K] [--hidden H] [--inner I]

The router's product and SwiGLU are plain torch operations; everything between
them runs in the library.  The layer keeps its weights' FP8B128 codes beside the
bf16 weights and makes them anew after an update (``requantize``).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_bsq_amd as bsq  # noqa: E402


class MoELayer:
    """y = sum over a token's experts of weight * (silu(x G^T) * (x U^T)) D^T, with a
    balance loss on the router.  Weights: router f32 [E, H]; gate_up bf16
    [E * 2I, H] (an expert's gate rows, then its up rows); down bf16 [E * H, I]."""

    def __init__(self, experts, hidden, inner, top_k, loss_coef=0.01, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(rows, cols):
            return torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5

        self.E, self.H, self.I, self.K, self.coef = experts, hidden, inner, top_k, loss_coef
        self.router = normal(experts, hidden)
        self.gate_up = normal(experts * 2 * inner, hidden).bfloat16()
        self.down = normal(experts * hidden, inner).bfloat16()
        self.bias = torch.zeros(experts, device=device)  # selection bias, moved by the caller if at all
        self.requantize()

    def requantize(self):
        """Codes of both orientations after a change of the weights."""
        self.gu_q, self.gu_t, self.gu_s = bsq.bsq_quantize_fp8b128_weights(self.gate_up, self.E)
        self.dn_q, self.dn_t, self.dn_s = bsq.bsq_quantize_fp8b128_weights(self.down, self.E)

    def forward(self, x, mask=None, train=True):
        """(y, loss); a training call also leaves what backward needs.  x bf16
        [tokens, H]; mask [tokens] is 0 for padding."""
        logits = x.float() @ self.router.t()
        ids, w, lse, counts, loss = bsq.bsq_moe_route(logits, self.K, bias=self.bias, mask=mask, loss_coef=self.coef)
        offsets, row_index, slot = bsq.bsq_moe_dispatch(ids, self.E)
        columns = offsets if train else None
        xr, xt = bsq.bsq_quantize_fp8b128(x, row_index=row_index, offsets=columns)
        gu = bsq.bsq_grouped_gemm_fp8b128_fwd(xr, (self.gu_q, self.gu_s), offsets)
        gate, up = gu.float().split(self.I, 1)
        h = (torch.nn.functional.silu(gate) * up).bfloat16()
        hr, ht = bsq.bsq_quantize_fp8b128(h, offsets=columns)
        ye = bsq.bsq_grouped_gemm_fp8b128_fwd(hr, (self.dn_q, self.dn_s), offsets)
        y = bsq.bsq_moe_combine(ye, slot, w)
        if train:
            self.saved = x, logits, ids, w, lse, counts, offsets, slot, xt, gu, ht, ye
        return y, loss

    def backward(self, dy, dloss=None):
        """Gradients (dx f32, router f32, gate_up bf16 [E, 2I, H], down bf16 [E, H, I])
        of the last training call for those of y and of the loss."""
        x, logits, ids, w, lse, counts, offsets, slot, xt, gu, ht, ye = self.saved
        M = ye.shape[0]
        dye, dw = bsq.bsq_moe_combine_bwd(dy, ye, slot, w, offsets)
        dyr, dyt = bsq.bsq_quantize_fp8b128(dye, offsets=offsets)
        dh, ddown = bsq.bsq_grouped_gemm_fp8b128_bwd(offsets, M, self.H, self.I, dy_q=dyr, wt_q=(self.dn_t, self.dn_s),
                                                     dyt_q=dyt, xt_q=ht)
        gate, up = gu.float().split(self.I, 1)
        s, dh = torch.sigmoid(gate), dh.float()
        dgu = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1).bfloat16()
        dgr, dgt = bsq.bsq_quantize_fp8b128(dgu, offsets=offsets)
        dxe, dgate_up = bsq.bsq_grouped_gemm_fp8b128_bwd(offsets, M, 2 * self.I, self.H, dy_q=dgr,
                                                         wt_q=(self.gu_t, self.gu_s), dyt_q=dgt, xt_q=xt)
        dlogits = bsq.bsq_moe_route_bwd(logits, ids, w, lse, counts, dw, dloss, loss_coef=self.coef)
        dx = bsq.bsq_moe_combine(dxe, slot).float() + dlogits @ self.router  # (a gather's gradient: the sum of its rows)
        return dx, dlogits.t() @ x.float(), dgate_up, ddown


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 2048), ("experts", 32), ("top-k", 8), ("hidden", 2048), ("inner", 1024)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    layer = MoELayer(a.experts, a.hidden, a.inner, a.top_k)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.hidden, generator=g, device="cuda")
    one = torch.ones(1, device="cuda")
    for step in range(4):
        y, balance = layer.forward(x)
        diff = y.float() - target
        print(f"step {step}: squared error {float(diff.square().mean()):.5f}, balance loss {float(balance):.5f}")
        _, drouter, dgu, ddn = layer.backward((2 * diff / a.hidden).bfloat16(), one)
        lr = 0.5 / a.tokens * a.hidden
        layer.router -= 0.01 * lr * drouter
        layer.gate_up -= (lr * dgu.float()).view_as(layer.gate_up).bfloat16()
        layer.down -= (lr * ddn.float()).view_as(layer.down).bfloat16()
        layer.requantize()
    y, _ = layer.forward(x[:16], train=False)
    full, _ = layer.forward(x, train=False)
    err = (y.float() - full[:16].float()).norm() / full[:16].float().norm()
    print(f"decoding step of 16 tokens: relative difference to the full batch {float(err):.1e}")


if __name__ == "__main__":
    main()
