"""Few output tiles with a long reduction, which the FP8B128 grouped GEMMs split into
parts and join: the bounds that test_gpu_gemm_b128.py states (a join adds parts
in binary32, one rounding a part, fewer than the blocks that the bound counts)."""
import numpy as np
import pytest
import torch

from oracle import moe
from test_gpu_gemm_b128 import close, codes, columns, dev, offsets, scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[9], [5, 0, 130, 1], [257, 3], [0, 40]])
@pytest.mark.parametrize("width,red", [(16, 2560), (144, 2688), (272, 5136), (128, 9040)])
@pytest.mark.parametrize("tail", [0, 70])
def test_fwd_and_dgrad(bsq_gpu, counts, width, red, tail):
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
    wst = np.ascontiguousarray(ws.transpose(0, 2, 1))
    kw = dict(dy_q=ad, wt_q=(wd[0], dev(wst)), flags=bsq_gpu.BSQ_DGRAD)
    dx, _ = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, red, width, dx_dtype=bsq_gpu.BSQ_F32, **kw)
    close(dx, *moe.b128_gemm_dgrad((a, asc), w, wst, off, width))
    assert (dx[off[-1]:] == 0).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, red, width, **kw)[0], dx.bfloat16())


@pytest.mark.parametrize("counts,n,k", [([2700], 144, 272), ([2600], 16, 16), ([4000, 0, 1, 900], 272, 144), ([0, 5000], 128, 128)])
@pytest.mark.parametrize("tail", [0, 300])
def test_wgrad(bsq_gpu, counts, n, k, tail):
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


def test_guards_invalid_offsets_and_graph(bsq_gpu):
    """Nothing outside the outputs and the workspace is written, also where offsets are
    invalid; a captured call gives the eager call's bits on new inputs."""
    rng = np.random.default_rng(5)
    off = offsets([100, 0, 33])
    E, M, n, k = 3, 133, 144, 2832
    kb = -(-k // 128)
    w, ws = dev(codes(rng, (E * n, k))), dev(scales(rng, (E, 2, kb)))
    a, asc = dev(codes(rng, (M, k))), dev(scales(rng, (kb, M)))
    buf = torch.full(((M + 4) * n,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[2 * n:2 * n + M * n].view(M, n)
    need = bsq_gpu.bsq_grouped_gemm_fp8b128_workspace_size(E)
    room = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
    work = room[:need]
    for bad in ([0, 100, 100, 134], [1, 100, 100, 133], [0, 101, 100, 133]):
        bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(np.array(bad, np.int32)), y=y, workspace=work)
        assert bsq_gpu.bsq_debug_status(work) == 1 and (buf == 7).all()
    offd = dev(off)
    bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), offd, y=y, workspace=work)
    assert bsq_gpu.bsq_debug_status(work) == 0
    assert (buf[:2 * n] == 7).all() and (buf[2 * n + M * n:] == 7).all() and (room[need:] == 9).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), offd)
    for _ in range(3):
        a.copy_(dev(codes(rng, (M, k))))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), offd))
        torch.cuda.synchronize()
