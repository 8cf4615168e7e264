"""Grouped GEMMs on FP8B128 operands against the 64-bit products of the same
codes and scales.

Bound, before any run: the matrix core sums a block's products in a window
aligned to the largest (within 2^-12.2 of the sum of their magnitudes, the
worst case the MXFP8 tests pin); the scales' product, the block's multiply and
the binary32 sum over the blocks add at most (blocks + 3) roundings of 2^-24.
So |y - r| <= 2^-11 sum|products|, and rms |y - r| <= 2^-15 of it (the typical
2^-16 the same tests record).  A bf16 output is the f32 output rounded."""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def codes(rng, shape):
    """Codes of normal values (no NaN pattern), some zero."""
    return moe.e4m3_encode(rng.standard_normal(shape) * 60.0)


def scales(rng, shape):
    return (2.0 ** rng.uniform(-12, -4, shape)).astype(np.float32)


def close(got, ref, mag):
    d = np.abs(got.double().cpu().numpy() - ref)
    assert (d <= 2.0 ** -11 * mag).all(), (d - 2.0 ** -11 * mag).max()
    assert np.sqrt((d ** 2).mean()) <= 2.0 ** -15 * np.sqrt((mag ** 2).mean()) or d.size == 0


def columns(rng, width, off, M):
    """Token-column operand: random codes and scales where a group has tokens, zero elsewhere."""
    E = len(off) - 1
    P = 128 * (E + -(-M // 128))
    c, s = np.zeros((width, P), np.uint8), np.zeros((P // 128, width), np.float32)
    for e in range(E):
        m = off[e + 1] - off[e]
        b = e + off[e] // 128
        c[:, 128 * b:128 * b + m] = codes(rng, (width, m))
        s[b:b + -(-m // 128)] = scales(rng, (-(-m // 128), width))
    return c, s


CASES = [  # counts, n, k
    ([1], 16, 16),
    ([5, 0, 3], 48, 144),
    ([130, 0, 0, 1, 257], 272, 400),
    ([64], 128, 128),
    ([300, 40], 256, 1040),
    ([0, 0], 32, 64),
    ([17] * 70, 144, 256),
    ([700, 3, 520], 528, 272),
    ([1, 2, 1, 0, 4, 1, 1, 6], 1040, 2064),
]


@pytest.mark.parametrize("counts,n,k", CASES)
@pytest.mark.parametrize("tail", [0, 37])
def test_fwd_and_dgrad(bsq_gpu, counts, n, k, tail):
    """`tail` rows past the last expert become zero."""
    rng = np.random.default_rng(len(counts) * 1000 + n + k)
    off = offsets(counts)
    E, M = len(counts), int(off[-1]) + tail
    if M == 0:
        return
    offd = dev(off)
    w, ws = codes(rng, (E * n, k)), scales(rng, (E, -(-n // 128), -(-k // 128)))
    a, asc = codes(rng, (M, k)), scales(rng, (-(-k // 128), M))
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((dev(a), dev(asc)), (dev(w), dev(ws)), offd, y_dtype=bsq_gpu.BSQ_F32)
    close(y, *moe.b128_gemm_fwd((a, asc), (w, ws), off, n))
    assert (y[off[-1]:] == 0).all()
    yb = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((dev(a), dev(asc)), (dev(w), dev(ws)), offd)
    assert torch.equal(yb, y.bfloat16())
    wt = np.ascontiguousarray(w.reshape(E, n, k).transpose(0, 2, 1)).reshape(E * k, n)
    g, gs = codes(rng, (M, n)), scales(rng, (-(-n // 128), M))
    kw = dict(dy_q=(dev(g), dev(gs)), wt_q=(dev(wt), dev(ws)), flags=bsq_gpu.BSQ_DGRAD)
    dx, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, n, k, dx_dtype=bsq_gpu.BSQ_F32, **kw)
    assert dw is None
    close(dx, *moe.b128_gemm_dgrad((g, gs), wt, ws, off, k))
    assert (dx[off[-1]:] == 0).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, n, k, **kw)[0], dx.bfloat16())


@pytest.mark.parametrize("counts,n,k", CASES)
@pytest.mark.parametrize("tail", [0, 37])
def test_wgrad(bsq_gpu, counts, n, k, tail):
    rng = np.random.default_rng(len(counts) * 1000 + n + k + 1)
    off = offsets(counts)
    M = int(off[-1]) + tail
    dyt, xt = columns(rng, n, off, M), columns(rng, k, off, M)
    kw = dict(dyt_q=tuple(map(dev, dyt)), xt_q=tuple(map(dev, xt)), flags=bsq_gpu.BSQ_WGRAD)
    dx, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(dev(off), M, n, k, dw_dtype=bsq_gpu.BSQ_F32, **kw)
    assert dx is None
    close(dw, *moe.b128_gemm_wgrad(dyt, xt, off))
    for e, c in enumerate(counts):
        assert c > 0 or (dw[e] == 0).all()
    assert torch.equal(bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(dev(off), M, n, k, **kw)[1], dw.bfloat16())


def test_exact_products(bsq_gpu):
    """Power-of-two codes and scales: every partial sum is a binary32 number, so the products are exact."""
    rng = np.random.default_rng(5)
    off = offsets([70, 0, 200])
    E, M, n, k = 3, 270, 160, 272
    vals = np.array([0, 1, 2, 4, -1, -2])
    a, w = moe.e4m3_encode(rng.choice(vals, (M, k))), moe.e4m3_encode(rng.choice(vals, (E * n, k)))
    p2 = lambda s: (2.0 ** rng.integers(-2, 3, s)).astype(np.float32)
    asc, ws = p2((3, M)), p2((E, 2, 3))
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((dev(a), dev(asc)), (dev(w), dev(ws)), dev(off), y_dtype=bsq_gpu.BSQ_F32)
    assert np.array_equal(y.cpu().numpy(), moe.b128_gemm_fwd((a, asc), (w, ws), off, n)[0])
    P = 128 * (E + 3)
    xt, dyt = columns(rng, k, off, M), columns(rng, n, off, M)
    ops = []
    for c, s in (dyt, xt):
        c = np.where(c != 0, moe.e4m3_encode(rng.choice(vals, c.shape)), 0).astype(np.uint8)
        ops.append((c, np.where(s != 0, p2(s.shape), 0).astype(np.float32)))
    assert ops[0][0].shape == (n, P)
    _, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(dev(off), M, n, k, dyt_q=tuple(map(dev, ops[0])),
                                                 xt_q=tuple(map(dev, ops[1])), flags=bsq_gpu.BSQ_WGRAD,
                                                 dw_dtype=bsq_gpu.BSQ_F32)
    assert np.array_equal(dw.cpu().numpy(), moe.b128_gemm_wgrad(ops[0], ops[1], off)[0])


def test_rows_do_not_depend_on_their_batch(bsq_gpu):
    """A row's output is the same bits whatever else is routed, as long as the
    same kernel form runs, and repeated calls agree."""
    rng = np.random.default_rng(6)
    E, n, k = 4, 272, 528
    w, ws = dev(codes(rng, (E * n, k))), dev(scales(rng, (E, 3, 5)))
    a, asc = codes(rng, (600, k)), scales(rng, (5, 600))
    y1 = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((dev(a), dev(asc)), (w, ws), dev(offsets([100, 200, 0, 300])))
    y2 = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((dev(a), dev(asc)), (w, ws), dev(offsets([100, 100, 100, 300])))
    assert torch.equal(y1[:200], y2[:200]) and torch.equal(y1[300:], y2[300:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y3 = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((dev(a), dev(asc)), (w, ws), dev(offsets([100, 200, 0, 300])), stream=s)
    s.synchronize()
    assert torch.equal(y1, y3)


def test_invalid_offsets_do_no_work(bsq_gpu):
    rng = np.random.default_rng(7)
    E, n, k, M = 3, 64, 128, 90
    w, ws = dev(codes(rng, (E * n, k))), dev(scales(rng, (E, 1, 1)))
    a, asc = dev(codes(rng, (M, k))), dev(scales(rng, (1, M)))
    P = 128 * (E + 1)
    t = [(dev(codes(rng, (d, P))), dev(scales(rng, (P // 128, d)))) for d in (n, k)]
    work = torch.empty(bsq_gpu.bsq_grouped_gemm_fp8b128_workspace_size(E), dtype=torch.uint8, device="cuda")
    for bad in ([0, 50, 40, 90], [1, 30, 60, 90], [0, 30, 60, 91], [0, -5, 60, 90]):
        off = dev(np.array(bad, np.int32))
        y = torch.full((M, n), 7.0, dtype=torch.bfloat16, device="cuda")
        bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), off, y=y, workspace=work)
        assert bsq_gpu.bsq_debug_status(work) == 1 and (y == 7).all()
        dw = torch.full((E, n, k), 7.0, dtype=torch.bfloat16, device="cuda")
        bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off, M, n, k, dyt_q=t[0], xt_q=t[1], flags=bsq_gpu.BSQ_WGRAD, dw=dw,
                                             workspace=work)
        assert bsq_gpu.bsq_debug_status(work) == 1 and (dw == 7).all()
    off = dev(np.array([0, 30, 60, 90], np.int32))
    bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), off, y=y, workspace=work)
    assert bsq_gpu.bsq_debug_status(work) == 0


def test_quantized_end_to_end(bsq_gpu):
    """The quantizers' outputs through the products: within the format's error of the bf16 operands' product."""
    rng = np.random.default_rng(8)
    off = offsets([90, 33, 0, 141])
    E, M, n, k = 4, 264, 144, 272
    x = torch.from_numpy(rng.standard_normal((M, k)).astype(np.float32)).bfloat16()
    w = torch.from_numpy((rng.standard_normal((E * n, k)) * 0.05).astype(np.float32)).bfloat16()
    dy = torch.from_numpy(rng.standard_normal((M, n)).astype(np.float32)).bfloat16()
    offd = dev(off)
    row, t = bsq_gpu.bsq_quantize_fp8b128(x.cuda(), offsets=offd)
    drow, dt = bsq_gpu.bsq_quantize_fp8b128(dy.cuda(), offsets=offd)
    wc, wt, ws = bsq_gpu.bsq_quantize_fp8b128_weights(w.cuda(), E)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row, (wc, ws), offd, y_dtype=bsq_gpu.BSQ_F32).double().cpu()
    dx, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(offd, M, n, k, dy_q=drow, wt_q=(wt, ws), dyt_q=dt, xt_q=t,
                                                  dx_dtype=bsq_gpu.BSQ_F32, dw_dtype=bsq_gpu.BSQ_F32)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        W, X, G = w[e * n:(e + 1) * n].double(), x[s].double(), dy[s].double()
        # two roundings of E4M3 (2^-4 each at most) per product, and half a subnormal step of a
        # block whose largest element is under 5 standard deviations: 2^-3 + 2^-8 of sum|products| and of the blocks
        for got, ref, mag in ((y[s], X @ W.T, X.abs() @ W.abs().T), (dx[s].double().cpu(), G @ W, G.abs() @ W.abs()),
                              (dw[e].double().cpu(), G.T @ X, G.abs().T @ X.abs())):
            assert ((got - ref).abs() <= (2.0 ** -3 + 2.0 ** -7) * mag + 1e-30).all()
