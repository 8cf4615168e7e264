"""FP8B128 quantizers and products in a row: against the 64-bit products of the
oracle's own codes and scales (the bounds that test_gpu_gemm_b128.py states), and,
per expert, against the bf16 operands' product without quantization: an E4M3 code is
off by an rms of about 0.026 of its value, two operands by sqrt(2) of it; twice
that of the Frobenius norm is allowed."""
import numpy as np
import pytest
import torch

from oracle import moe
from test_gpu_gemm_b128 import close, offsets

pytestmark = pytest.mark.gpu


def near(got, ref):
    assert np.linalg.norm(got - ref) <= 2 * 0.026 * 2 ** 0.5 * np.linalg.norm(ref)


@pytest.mark.parametrize("counts,n,k", [([90, 33, 0, 141], 144, 272), ([1, 0, 2], 272, 400), ([129, 300], 400, 144)])
def test_against_the_oracles_codes(bsq_gpu, counts, n, k):
    rng = np.random.default_rng(n + k)
    off = offsets(counts)
    E, M = len(counts), int(off[-1])

    def bf16(shape, sigma):
        return torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).bfloat16()

    x, w, dy = bf16((M, k), 1.0), bf16((E * n, k), 0.05), bf16((M, n), 1e-3)
    offd = torch.from_numpy(off).cuda()
    f32 = bsq_gpu.BSQ_F32
    row, t = bsq_gpu.bsq_quantize_fp8b128(x.cuda(), offsets=offd)
    drow, dt = bsq_gpu.bsq_quantize_fp8b128(dy.cuda(), offsets=offd)
    wc, wt, ws = bsq_gpu.bsq_quantize_fp8b128_weights(w.cuda(), E)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row, (wc, ws), offd, y_dtype=f32)
    dx, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, n, k, dy_q=drow, wt_q=(wt, ws), dyt_q=dt, xt_q=t, dx_dtype=f32,
                                                  dw_dtype=f32)
    X, W, G = x.float().numpy(), w.float().numpy(), dy.float().numpy()
    oc, ot, os = moe.b128_weights(W, E)
    close(y, *moe.b128_gemm_fwd(moe.b128_rows(X), (oc, os), off, n))
    close(dx, *moe.b128_gemm_dgrad(moe.b128_rows(G), ot, os, off, k))
    close(dw, *moe.b128_gemm_wgrad(moe.b128_columns(G, off), moe.b128_columns(X, off), off))
    X, W, G = X.astype(np.float64), W.astype(np.float64), G.astype(np.float64)
    y, dx, dw = (v.double().cpu().numpy() for v in (y, dx, dw))
    for e in range(E):
        s, we = slice(off[e], off[e + 1]), W[e * n:(e + 1) * n]
        near(y[s], X[s] @ we.T)
        near(dx[s], G[s] @ we)
        near(dw[e], G[s].T @ X[s])
