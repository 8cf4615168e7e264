"""The 128 x 128 tiles of the FP8B128 grouped GEMMs (in even shares of the XCDs and in
groups of row tiles) and the weight loads past the last-level cache, at sizes that
take them, every row of every expert: the bounds that test_gpu_gemm_b128.py states,
against 64-bit products on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rand_codes(g, rows, cols):
    return (torch.randn(rows, cols, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn).view(torch.uint8)


def rand_scales(g, *shape):
    return 2.0 ** (torch.rand(*shape, generator=g, device="cuda") * 8 - 12)


def value(codes, scale):
    """64-bit values of codes [r][c] with scale [c blocks][r]."""
    return codes.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(128, 0)[:codes.shape[1]].t()


def product(a, asc, w, ws, counts):
    """(64-bit result, sum of magnitudes); rows past the last expert are zero."""
    E, C = len(counts), w.shape[0] // len(counts)
    y = torch.zeros(a.shape[0], C, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    at = 0
    for e, m in enumerate(counts):
        s = slice(at, at + m)
        x = value(a[s], asc[:, s])
        v = value(w[e * C:(e + 1) * C], ws[e].t().repeat_interleave(128, 1)[:, :C])
        y[s], mag[s] = x @ v.t(), x.abs() @ v.abs().t()
        at += m
    return y, mag


def close(got, ref, mag):
    d = (got.double() - ref).abs()
    assert bool((d <= 2.0 ** -11 * mag).all())
    assert float(d.square().mean().sqrt()) <= 2.0 ** -15 * float(mag.square().mean().sqrt())


def spread(E, least, most, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(least, most + 1, (E,), generator=g).tolist()
    c[E // 2] = 0
    return c


CASES = {
    "all at once": (spread(2, 1, 1500, 1)[:1] + [900], 1552, 400),
    "all at once, more experts than lanes": (spread(70, 25, 60, 2), 1008, 4112),
    "several rounds": (spread(20, 38, 62, 3), 4240, 4112),
    "several rounds, more experts than lanes": (spread(70, 25, 60, 4), 1168, 4112),
    "streamed weights": (spread(72, 0, 9, 5), 2048, 2048),
    "streamed weights, 128 rows of one expert": ([3] * 70 + [130, 1], 2064, 2048),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("tail", [0, 45])
def test_fwd_and_dgrad(bsq_gpu, name, tail):
    counts, width, red = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(width + red)
    E, M, wb, rb = len(counts), sum(counts) + tail, -(-width // 128), -(-red // 128)
    w, ws = rand_codes(g, E * width, red), rand_scales(g, E, wb, rb)
    a, asc = rand_codes(g, M, red), rand_scales(g, rb, M)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    ref, mag = product(a, asc, w, ws, counts)
    y = torch.full((M, width), 7.0, device="cuda")
    bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), off, y_dtype=bsq_gpu.BSQ_F32, y=y)
    close(y, ref, mag)
    assert not y[M - tail:].any()
    yb = torch.full((M, width), 7.0, dtype=torch.bfloat16, device="cuda")
    bsq_gpu.bsq_grouped_gemm_fp8b128_fwd((a, asc), (w, ws), off, y=yb)
    assert torch.equal(yb, y.bfloat16())
    # the same product as a gradient of the input: rows of `red`, results of `width`
    kw = dict(dy_q=(a, asc), wt_q=(w, ws.transpose(1, 2).contiguous()), flags=bsq_gpu.BSQ_DGRAD)
    for dt, out in ((bsq_gpu.BSQ_F32, y), (bsq_gpu.BSQ_BF16, yb)):
        dx = torch.full_like(out, 7.0)
        bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off, M, red, width, dx_dtype=dt, dx=dx, **kw)
        assert torch.equal(dx, out)
