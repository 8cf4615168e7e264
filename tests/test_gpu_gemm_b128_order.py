"""One order of every sum: what a row of the FP8B128 products gets (and, in the
weight gradient, an expert) is the same bits whatever else the call holds, so in
every form that the sizes choose: few or many rows, experts, columns and blocks."""
import numpy as np
import pytest
import torch

from test_gpu_gemm_b128 import codes, columns, dev, offsets, scales

pytestmark = pytest.mark.gpu


def same(got, ref):
    assert torch.equal(got.view(torch.int32), ref.view(torch.int32))


# rows of the other experts: none, one, a few, many for one of them, many for all
LOADS = [[0, 0], [1, 0], [9, 4], [130, 0], [0, 700], [300, 900], [2600, 2500]]


@pytest.mark.parametrize("width", [16, 304, 1424, 4112])
@pytest.mark.parametrize("red", [272, 5712])
def test_rows(bsq_gpu, width, red):
    rng = np.random.default_rng(width + red)
    E, mine, wb, rb = 3, 5, -(-width // 128), -(-red // 128)
    w, ws = dev(codes(rng, (E * width, red))), dev(scales(rng, (E, wb, rb)))
    wst = ws.transpose(1, 2).contiguous()
    most = mine + max(map(sum, LOADS))
    a, asc = dev(codes(rng, (most, red))), dev(scales(rng, (rb, most)))
    # the expert alone, and with others: its rows are the first ones
    ref = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a[:mine], asc[:, :mine].contiguous()), (w[:width], ws[:1]),
                                               dev(offsets([mine])), y_dtype=bsq_gpu.BSQ_F32)
    for load in LOADS:
        M = mine + sum(load)
        aq, off = (a[:M], asc[:, :M].contiguous()), dev(offsets([mine] + load))
        same(bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(aq, (w, ws), off, y_dtype=bsq_gpu.BSQ_F32)[:mine], ref)
        dx, _ = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off, M, red, width, dy_q=aq, wt_q=(w, wst), flags=bsq_gpu.BSQ_DGRAD,
                                                     dx_dtype=bsq_gpu.BSQ_F32)
        same(dx[:mine], ref)
    # more experts, none of them with more than a few rows
    E = 64 if width < 4112 else 8
    w, ws = w[:width].repeat(E, 1), ws[:1].repeat(E, 1, 1)
    for rows in (1, 3, 5):
        n = rows * E
        y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a[:rows].repeat(E, 1), asc[:, :rows].repeat(1, E)), (w, ws),
                                                 dev(offsets([rows] * E)), y_dtype=bsq_gpu.BSQ_F32)
        same(y, ref[:rows].repeat(E, 1)[:n])


def test_rows_of_streamed_weights(bsq_gpu):
    """Weights past the last-level cache are loaded by another policy."""
    rng = np.random.default_rng(2)
    E, n, k, rows = 33, 2048, 4224, 7
    w, ws = dev(codes(rng, (n, k))), dev(scales(rng, (1, n // 128, k // 128)))
    a, asc = dev(codes(rng, (rows, k))), dev(scales(rng, (k // 128, rows)))
    ref = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), dev(offsets([rows])), y_dtype=bsq_gpu.BSQ_F32)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a.repeat(E, 1), asc.repeat(1, E)), (w.repeat(E, 1), ws.repeat(E, 1, 1)),
                                             dev(offsets([rows] * E)), y_dtype=bsq_gpu.BSQ_F32)
    same(y, ref.repeat(E, 1))


@pytest.mark.parametrize("n,k", [(16, 48), (272, 304), (1424, 2000)])
@pytest.mark.parametrize("tokens", [100, 3900])
def test_weight_gradient(bsq_gpu, n, k, tokens):
    rng = np.random.default_rng(n + tokens)
    alone = [columns(rng, d, offsets([tokens]), tokens) for d in (n, k)]

    def call(before, after):
        off = offsets(before + [tokens] + after)
        e, M = len(before), int(off[-1])
        P = 128 * (len(off) - 1 + -(-M // 128))
        b, nb = e + off[e] // 128, -(-tokens // 128)
        q = []
        for c, s in alone:  # the other experts' tokens are zeros
            wide, ws = np.zeros((c.shape[0], P), np.uint8), np.zeros((P // 128, c.shape[0]), np.float32)
            wide[:, 128 * b:128 * (b + nb)] = c[:, :128 * nb]
            ws[b:b + nb] = s[:nb]
            q.append((dev(wide), dev(ws)))
        return bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(dev(off), M, n, k, dyt_q=q[0], xt_q=q[1], flags=bsq_gpu.BSQ_WGRAD,
                                                    dw_dtype=bsq_gpu.BSQ_F32)[1][e]

    ref = call([], [])
    for before, after in (([1], []), ([0], [130]), ([5000], [3]), ([], [9000]), ([0] * 9, [40] * 6), ([20] * 40, [700])):
        same(call(before, after), ref)
