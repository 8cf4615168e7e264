"""The 16 x 64 tiles of the FP8B128 grouped GEMMs, which calls of at most two
rows an expert take: the bounds of test_gpu_gemm_b128.py (the four partial sums
of a block order add two roundings to it), at one row, 16 and 17 rows of one
expert, empty experts, one to nine blocks and partial column tiles."""
import numpy as np
import pytest
import torch

from oracle import moe
from test_gpu_gemm_b128 import close, codes, dev, offsets, scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[1], [2, 0], [0, 0, 1], [17] + [0] * 9, [16, 1] + [0, 1] * 8, [0] * 69 + [40, 1]])
@pytest.mark.parametrize("width,red", [(16, 16), (80, 128), (64, 144), (208, 528), (144, 1040), (1040, 1168)])
@pytest.mark.parametrize("tail", [0, 1])
def test_fwd_and_dgrad(bsq_gpu, counts, width, red, tail):
    rng = np.random.default_rng(width + red + len(counts))
    off = offsets(counts)
    E, M = len(counts), int(off[-1]) + tail
    wb, rb = -(-width // 128), -(-red // 128)
    w, ws = codes(rng, (E * width, red)), scales(rng, (E, wb, rb))
    a, asc = codes(rng, (M, red)), scales(rng, (rb, M))
    ad, wd, offd = (dev(a), dev(asc)), (dev(w), dev(ws)), dev(off)
    buf = torch.full((M + 2, width), 7.0, device="cuda")
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(ad, wd, offd, y_dtype=bsq_gpu.BSQ_F32, y=buf[1:1 + M])
    close(y, *moe.b128_gemm_fwd((a, asc), (w, ws), off, width))
    assert (y[off[-1]:] == 0).all() and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(ad, wd, offd), y.bfloat16())
    wst = np.ascontiguousarray(ws.transpose(0, 2, 1))
    kw = dict(dy_q=ad, wt_q=(wd[0], dev(wst)), flags=bsq_gpu.BSQ_DGRAD)
    dx, _ = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, red, width, dx_dtype=bsq_gpu.BSQ_F32, **kw)
    close(dx, *moe.b128_gemm_dgrad((a, asc), w, wst, off, width))


def test_invalid_offsets(bsq_gpu):
    rng = np.random.default_rng(1)
    E, M, n, k = 8, 9, 80, 272
    w, ws = dev(codes(rng, (E * n, k))), dev(scales(rng, (E, 1, 3)))
    a, asc = dev(codes(rng, (M, k))), dev(scales(rng, (3, M)))
    work = torch.empty(bsq_gpu.bsq_grouped_gemm_fp8b128_workspace_size(E), dtype=torch.uint8, device="cuda")
    y = torch.full((M, n), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, 1, 2, 3, 2, 5, 6, 7, 9], [0, 1, 2, 3, 4, 5, 6, 7, 10], [1, 1, 2, 3, 4, 5, 6, 7, 9]):
        bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(np.array(bad, np.int32)), y=y, workspace=work)
        assert bsq_gpu.bsq_debug_status(work) == 1 and (y == 7).all()
