"""The 256 x 256 and 256 x 128 tiles of the FP8B128 grouped GEMMs, which calls of many tiles
and rows take: the same bounds as test_gpu_gemm_b128.py states, at the edges of a tile
(1, 128, 129, 256, 257 rows; partial columns), of the pipeline (one to five
blocks of 128) and of an expert's rows."""
import numpy as np
import pytest
import torch

from oracle import moe
from test_gpu_gemm_b128 import close, codes, columns, dev, offsets, scales

pytestmark = pytest.mark.gpu

# experts of 0, 1, 128, 129, 256, 257 rows and more
COUNTS = [1, 0, 128, 129, 256, 257, 384, 511]
SHAPES = [(3984, 16), (4096, 128), (4112, 144), (3984, 272), (4064, 400), (4000, 528)]  # width, reduction


# fewer rows: 256 x 128 tiles
MID = [130, 257, 0, 600, 1]
CASES = [(COUNTS, t, w, r) for w, r in SHAPES for t in (0, 300)] + [(MID, t, w, r) for w, r in SHAPES for t in (0, 9)]


@pytest.mark.parametrize("counts,tail,width,red", CASES)
def test_fwd_and_dgrad(bsq_gpu, counts, tail, width, red):
    rng = np.random.default_rng(width + red)
    off = offsets(counts)
    E, M = len(counts), int(off[-1]) + tail
    wb, rb = -(-width // 128), -(-red // 128)
    w, ws = codes(rng, (E * width, red)), scales(rng, (E, wb, rb))
    a, asc = codes(rng, (M, red)), scales(rng, (rb, M))
    ad, wd, offd = (dev(a), dev(asc)), (dev(w), dev(ws)), dev(off)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(ad, wd, offd, y_dtype=bsq_gpu.BSQ_F32)
    close(y, *moe.b128_gemm_fwd((a, asc), (w, ws), off, width))
    assert (y[off[-1]:] == 0).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(ad, wd, offd), y.bfloat16())
    # dgrad with the same operands: dY rows of `red`, dX of `width`; scales by [red block][width block]
    wst = np.ascontiguousarray(ws.transpose(0, 2, 1))
    kw = dict(dy_q=ad, wt_q=(wd[0], dev(wst)), flags=bsq_gpu.BSQ_DGRAD)
    dx, _ = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, red, width, dx_dtype=bsq_gpu.BSQ_F32, **kw)
    close(dx, *moe.b128_gemm_dgrad((a, asc), w, wst, off, width))
    assert (dx[off[-1]:] == 0).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, red, width, **kw)[0], dx.bfloat16())


@pytest.mark.parametrize("n,k", [(528, 784), (400, 1040), (1040, 272)])
@pytest.mark.parametrize("tail", [0, 300])
def test_wgrad(bsq_gpu, n, k, tail):
    counts = [1, 0, 128, 129, 256, 257, 3, 17, 0, 400, 640, 31] + [5] * 48
    rng = np.random.default_rng(n + k)
    off = offsets(counts)
    M = int(off[-1]) + tail
    dyt, xt = columns(rng, n, off, M), columns(rng, k, off, M)
    kw = dict(dyt_q=tuple(map(dev, dyt)), xt_q=tuple(map(dev, xt)), flags=bsq_gpu.BSQ_WGRAD)
    dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(dev(off), M, n, k, dw_dtype=bsq_gpu.BSQ_F32, **kw)[1]
    close(dw, *moe.b128_gemm_wgrad(dyt, xt, off))
    for e, c in enumerate(counts):
        assert c > 0 or (dw[e] == 0).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(dev(off), M, n, k, **kw)[1], dw.bfloat16())


@pytest.mark.parametrize("counts", [COUNTS, MID])
def test_guards_and_invalid_offsets(bsq_gpu, counts):
    """Nothing outside the outputs is written, also where offsets are invalid; repeated calls give the same bits."""
    rng = np.random.default_rng(3)
    off = offsets(counts)
    E, M, n, k = len(counts), int(off[-1]), 3984, 272
    w, ws = dev(codes(rng, (E * n, k))), dev(scales(rng, (E, -(-n // 128), 3)))
    a, asc = dev(codes(rng, (M, k))), dev(scales(rng, (3, M)))
    buf = torch.full(((M + 4) * n,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[2 * n:2 * n + M * n].view(M, n)
    work = torch.empty(bsq_gpu.bsq_grouped_gemm_fp8b128_workspace_size(E), dtype=torch.uint8, device="cuda")
    for bad in (off[:-1].tolist() + [int(off[-1]) + 1], [1] + off[1:].tolist(), [0, 5, 2] + off[3:].tolist()):
        bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(np.array(bad, np.int32)), y=y, workspace=work)
        assert bsq_gpu.bsq_debug_status(work) == 1 and (buf == 7).all()
    bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(off), y=y, workspace=work)
    assert bsq_gpu.bsq_debug_status(work) == 0
    assert (buf[:2 * n] == 7).all() and (buf[2 * n + M * n:] == 7).all()
    again = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(off))
    assert torch.equal(again, y)


def test_streamed_weights(bsq_gpu):
    """Few rows against more weights than the caches hold: a row's output is the bits
    that the same call gives with one expert's weights in place (a product of its own)."""
    E, n, k, M = 72, 2048, 2048, 300
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randint(0, 120, (E * n, k), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.rand(E, 16, 16, device="cuda", generator=g)
    a = torch.randint(0, 120, (M, k), dtype=torch.uint8, device="cuda", generator=g)
    asc = torch.rand(16, M, device="cuda", generator=g)
    counts = [4] * 70 + [0, 20]
    off = offsets(counts)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(off))
    for e in (0, 33, 69, 71):
        s = slice(int(off[e]), int(off[e + 1]))
        one = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a[s].contiguous(), asc[:, s].contiguous()),
                                                   (w[e * n:(e + 1) * n], ws[e:e + 1]), dev(offsets([s.stop - s.start])))
        assert torch.equal(y[s], one)
