"""An infinity or a NaN in a block of the FP8B128 quantizers: the block's scale is NaN,
so nothing of it passes for a number in a product; every other block is as without it."""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

VALUES = [float("nan"), -float("nan"), float("inf"), -float("inf")]
ROWS, COLS = 200, 272
OFF = np.array([0, 130, 200], np.int32)
AT = [(0, 0), (7, 127), (129, 130), (131, 271), (199, 200)]


def inputs(value):
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((ROWS, COLS)).astype(np.float32)).bfloat16()
    bad = x.clone()
    for at in AT:
        bad[at] = value
    return x, bad


def check(got, ref, hit, per_code):
    """`hit`: the scales of blocks with a bad element; per_code: for every code whether its block is one."""
    codes, scale = got[0].cpu().numpy(), got[1].cpu().numpy()
    assert np.isnan(scale[hit]).all()
    assert np.array_equal(scale[~hit], ref[1][~hit])
    assert np.array_equal(codes[~per_code], ref[0][~per_code])


@pytest.mark.parametrize("value", VALUES)
def test_rows_and_columns(bsq_gpu, value):
    x, bad = inputs(value)
    off = torch.from_numpy(OFF).cuda()
    rows, cols = moe.b128_rows(x.float().numpy()), moe.b128_columns(x.float().numpy(), OFF)
    rhit, chit = np.zeros(rows[1].shape, bool), np.zeros(cols[1].shape, bool)
    for r, c in AT:
        rhit[c // 128, r] = True
        g = int(r >= OFF[1])
        chit[g + OFF[g] // 128 + (r - OFF[g]) // 128, c] = True
    rcode = np.repeat(rhit.T, 128, 1)[:, :COLS]
    ccode = np.repeat(chit.T, 128, 1)
    b = bad.cuda()
    check(bsq_gpu.bsq_quantize_fp8b128(b)[0], rows, rhit, rcode)
    both = bsq_gpu.bsq_quantize_fp8b128(b, offsets=off)
    check(both[0], rows, rhit, rcode)
    check(both[1], cols, chit, ccode)
    idx = torch.arange(ROWS, dtype=torch.int32, device="cuda")
    check(bsq_gpu.bsq_quantize_fp8b128(b, row_index=idx)[0], rows, rhit, rcode)
    check(bsq_gpu.bsq_quantize_fp8b128(b, row_index=idx, offsets=off, rows_form=False)[1], cols, chit, ccode)


@pytest.mark.parametrize("value", VALUES)
def test_weights_and_product(bsq_gpu, value):
    """A row of the product is NaN where its block is, in every column whose weights share the block."""
    E, n, k = 2, 144, 272
    w = torch.from_numpy(np.random.default_rng(4).standard_normal((E * n, k)).astype(np.float32)).bfloat16()
    ref = moe.b128_weights(w.float().numpy(), E)
    bad = w.clone()
    bad[5, 140] = value
    codes, codes_t, scale = bsq_gpu.bsq_quantize_fp8b128_weights(bad.cuda(), E)
    hit = np.zeros(ref[2].shape, bool)
    hit[0, 0, 1] = True
    block = np.zeros((E, n, k), bool)
    block[0, :128, 128:256] = True
    check((codes, scale), (ref[0], ref[2]), hit, block.reshape(E * n, k))
    check((codes_t, scale), (ref[1], ref[2]), hit, np.ascontiguousarray(block.transpose(0, 2, 1)).reshape(E * k, n))
    x = torch.randn(9, k, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    row, _ = bsq_gpu.bsq_quantize_fp8b128(x)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row, (codes, scale), torch.tensor([0, 6, 9], dtype=torch.int32, device="cuda"))
    nan = torch.isnan(y).cpu()
    assert nan[:6, :128].all() and not nan[:6, 128:].any() and not nan[6:].any()
