"""FP8B128 quantization and the layer around it without a row: nothing to do is no error."""
import ctypes
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

FAKE = ctypes.c_void_p(0x100000)


def test_rows_on_the_host():
    """Tensors without elements have null addresses."""
    import block_scaled_precision_bsq_amd as bsq
    f = bsq._lib.bsq_quantize_fp8b128

    def call(x=None, src=0, C=64, ld=64, idx=None, R=0, off=None, G=0, c=None, s=None, tc=None, ts=None):
        return f(x, src, C, ld, idx, R, off, G, c, s, tc, ts, None)

    assert call() == bsq.BSQ_OK                                    # no rows
    assert call(x=FAKE, src=5) == bsq.BSQ_OK                       # an index without entries
    assert call(x=FAKE, src=5, C=0, ld=0, R=5) == bsq.BSQ_OK       # no columns
    assert call(C=0, ld=0, off=FAKE, G=2) == bsq.BSQ_OK
    assert call(x=FAKE, src=5, R=5) == bsq.BSQ_ERR_INVALID_ARG     # rows, and nothing wanted
    assert call(x=FAKE, src=5, R=4, c=FAKE, s=FAKE) == bsq.BSQ_ERR_INVALID_ARG
    assert call(c=FAKE) == call(tc=FAKE) == bsq.BSQ_ERR_INVALID_ARG
    assert call(tc=FAKE, ts=FAKE) == bsq.BSQ_ERR_INVALID_ARG       # columns need offsets


@pytest.mark.gpu
def test_quantize(bsq_gpu):
    x = torch.ones(5, 32, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    for src, idx in ((x[:0], None), (x[:0], none), (x, none)):
        row, t = bsq_gpu.bsq_quantize_fp8b128(src, row_index=idx)
        assert row[0].shape == (0, 32) and row[1].shape == (1, 0) and t is None
        out = (torch.full((32, 384), 7, dtype=torch.uint8, device="cuda"), torch.full((3, 32), 7.0, device="cuda"))
        row, t = bsq_gpu.bsq_quantize_fp8b128(src, row_index=idx, offsets=off, t=out)
        assert row[0].shape == (0, 32) and not t[0].any() and not t[1].any()
    row, _ = bsq_gpu.bsq_quantize_fp8b128(x[:, :0])
    assert row[0].shape == (5, 0) and row[1].shape == (0, 5)


@pytest.mark.gpu
def test_layer(bsq_gpu):
    from moe_layer import MoELayer
    layer = MoELayer(4, 128, 64, 2, loss_coef=0.1)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    y, loss = layer.forward(x, train=False)
    assert y.shape == (0, 128) and float(loss) == 0.0
    y, loss = layer.forward(x)
    dx, drouter, dgu, ddn = layer.backward(torch.empty_like(y), torch.ones(1, device="cuda"))
    assert dx.shape == (0, 128) and not drouter.any() and not dgu.any() and not ddn.any()
