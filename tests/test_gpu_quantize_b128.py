"""FP8B128 quantizers on the GPU: bytes and scales equal the oracle's."""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu


def bf16_input(rng, rows, cols):
    """Normals with per-row magnitudes from subnormal to near the type's largest, zero blocks and zero rows."""
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    if rows > 4:
        x[1] *= 2.0 ** -120
        x[2] *= 2.0 ** 100
        x[3] = 0
        x[4, : min(cols, 128)] = 0
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def check(got, ref):
    for g, r in zip(got, ref):
        assert np.array_equal(g.cpu().numpy(), r)


def offsets_for(rng, rows, groups):
    cut = np.sort(rng.integers(0, rows + 1, groups - 1))
    return np.concatenate([[0], cut, [rows]]).astype(np.int32)


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (17, 144), (130, 256), (40, 1040), (5, 2064)])
def test_rows(bsq_gpu, rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = bf16_input(rng, rows, cols)
    wide = torch.zeros(rows, cols + 24, dtype=torch.bfloat16)
    wide[:, 8:8 + cols] = x
    ref = moe.b128_rows(x.float().numpy())
    check(bsq_gpu.bsq_quantize_fp8b128(x.cuda())[0], ref)
    check(bsq_gpu.bsq_quantize_fp8b128(wide.cuda()[:, 8:8 + cols])[0], ref)
    idx = rng.integers(-2, rows + 2, 2 * rows + 1).astype(np.int32)
    src = np.where(((idx >= 0) & (idx < rows))[:, None], x.float().numpy()[idx.clip(0, rows - 1)], 0)
    check(bsq_gpu.bsq_quantize_fp8b128(x.cuda(), row_index=torch.from_numpy(idx).cuda())[0], moe.b128_rows(src))


@pytest.mark.parametrize("rows,cols,groups", [(1, 16, 1), (129, 144, 3), (300, 128, 70), (500, 272, 2), (128, 48, 1),
                                              (0, 32, 2)])
def test_columns_and_both(bsq_gpu, rows, cols, groups):
    rng = np.random.default_rng(rows + cols + groups)
    x = bf16_input(rng, rows, cols)
    off = offsets_for(rng, rows, groups)
    offd = torch.from_numpy(off).cuda()
    xf = x.float().numpy()
    row, t = bsq_gpu.bsq_quantize_fp8b128(x.cuda(), offsets=offd, rows_form=False)
    assert row is None
    check(t, moe.b128_columns(xf, off))
    if rows == 0:
        return
    row, t = bsq_gpu.bsq_quantize_fp8b128(x.cuda(), offsets=offd)
    check(row, moe.b128_rows(xf))
    check(t, moe.b128_columns(xf, off))
    # gathered, with slots that no choice owns past the last group
    idx = rng.integers(0, rows, rows + 9).astype(np.int32)
    idx[rows:] = -1
    src = np.where((idx >= 0)[:, None], xf[idx.clip(0)], 0)
    row, t = bsq_gpu.bsq_quantize_fp8b128(x.cuda(), row_index=torch.from_numpy(idx).cuda(), offsets=offd)
    check(row, moe.b128_rows(src))
    check(t, moe.b128_columns(src, off))


@pytest.mark.parametrize("E,n,k", [(1, 16, 16), (3, 128, 128), (2, 144, 272), (1, 272, 144), (2, 400, 48)])
def test_weights(bsq_gpu, E, n, k):
    rng = np.random.default_rng(E + n + k)
    w = bf16_input(rng, E * n, k)
    ref = moe.b128_weights(w.float().numpy(), E)
    check(bsq_gpu.bsq_quantize_fp8b128_weights(w.cuda(), E), ref)
    codes, ct, scale = bsq_gpu.bsq_quantize_fp8b128_weights(w.cuda(), E, transposed=False)
    assert ct is None
    check((codes, scale), (ref[0], ref[2]))


def test_bad_offsets_stay_in_bounds(bsq_gpu):
    """Decreasing offsets give unspecified bytes; the buffers' neighbours stay untouched."""
    x = torch.ones(100, 32, dtype=torch.bfloat16, device="cuda")
    for off in ([0, 90, 20, 100], [50, 100, 100, 100], [0, 40, 60, 80]):
        offd = torch.tensor(off, dtype=torch.int32, device="cuda")
        P = bsq_gpu.bsq_colwise_padded_cols(3, 100)
        buf = torch.full((32 * P + 4096,), 7, dtype=torch.uint8, device="cuda")
        tc = buf[2048:2048 + 32 * P].view(32, P)
        ts = torch.empty(P // 128, 32, device="cuda")
        bsq_gpu.bsq_quantize_fp8b128(x, offsets=offd, t=(tc, ts))
        torch.cuda.synchronize()
        assert (buf[:2048] == 7).all() and (buf[2048 + 32 * P:] == 7).all()


def test_every_maximum(bsq_gpu):
    """Each finite bf16 magnitude as a block's maximum, to the type's ends: scales
    and codes are the correctly rounded quotients' in all three forms."""
    rng = np.random.default_rng(17)
    bits = np.arange(1, 0x7F80, dtype=np.uint16)
    top = torch.from_numpy((bits | (rng.integers(0, 2, bits.size) << 15).astype(np.uint16)).view(np.int16)).view(torch.bfloat16)
    x = (top.double()[:, None] * torch.from_numpy(rng.uniform(-1, 1, (bits.size, 128)))).bfloat16()
    x[torch.arange(bits.size), torch.from_numpy(rng.integers(0, 128, bits.size))] = top
    check(bsq_gpu.bsq_quantize_fp8b128(x.cuda())[0], moe.b128_rows(x.float().numpy()))
    xt = x.t().contiguous()[:, :32512]  # the same blocks down 128 rows
    off = np.array([0, 128], np.int32)
    check(bsq_gpu.bsq_quantize_fp8b128(xt.cuda(), offsets=torch.from_numpy(off).cuda(), rows_form=False)[1],
          moe.b128_columns(xt.float().numpy(), off))
    # and over a 128 x 128 block each (of every 64th)
    w = torch.zeros(128 * 510, 128, dtype=torch.bfloat16)
    w[::128] = x[::64][:510]
    check(bsq_gpu.bsq_quantize_fp8b128_weights(w.cuda(), 510), moe.b128_weights(w.float().numpy(), 510))
