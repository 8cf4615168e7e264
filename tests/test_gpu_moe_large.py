"""Tensors of more than 2^31 elements.  What a row, a token or an expert gets does
not depend on the others beside it, so the last ones of a large call must be those
of a small call, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

WIDTH = 7168
ROWS = 2 ** 31 // WIDTH + 400  # more than 2^31 elements and no multiple of a tile
LAST = 200


def randn(rows, cols, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for part in x.split(1 << 16):
        part.normal_(generator=g)
    return x


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(got, ref):
    assert torch.equal(got, ref.to(got.dtype).view(got.shape))


def test_route(bsq_gpu):
    """The loss: a wave adds the probabilities of T / 4096 tokens, a workgroup those of
    16 waves, each of a softmax within 32 roundings (logits within 8 of each other)."""
    E, K = 384, 8
    T = 2 ** 31 // E + 77
    l = randn(T, E, torch.float32)
    ids, w, lse, counts, loss = bsq_gpu.bsq_moe_route(l, K, loss_coef=1.0)
    few = bsq_gpu.bsq_moe_route(l[-LAST:].clone(), K)
    for got, ref in zip((ids, w, lse), few):
        same(got[-LAST:], ref)
    same(counts[:E], torch.bincount(ids.view(-1), minlength=E))
    assert int(counts[E]) == T
    p = sum(part.double().softmax(1).sum(0) for part in l.split(1 << 17))
    ref = float(E / K * (counts[:E].double() * p).sum() / T ** 2)
    assert abs(float(loss) - ref) <= ref * (T / 4096 + 16 + 32) * 2 ** -24
    del p
    dw = randn(T, K, torch.float32)
    got = bsq_gpu.bsq_moe_route_bwd(l, ids, w, lse, counts, dweights=dw)
    ref = bsq_gpu.bsq_moe_route_bwd(l[-LAST:].clone(), *few[:4], dweights=dw[-LAST:].clone())
    same(got[-LAST:], ref)


def test_combine(bsq_gpu):
    x = randn(ROWS, WIDTH)
    slot = torch.arange(ROWS - 1, -1, -1, dtype=torch.int32, device="cuda").view(ROWS, 1)
    same(bsq_gpu.bsq_moe_combine(x, slot), x.flip(0))
    w = randn(ROWS, 1, torch.float32)
    dx, dw = bsq_gpu.bsq_moe_combine_bwd(x, x, slot, weights=w, offsets=ints(0, ROWS))
    # the last tokens own the first rows
    few = torch.cat((x[:LAST], x[-LAST:]))
    own = slot[-LAST:].clone()
    part, dwl = bsq_gpu.bsq_moe_combine_bwd(few[LAST:].clone(), few, own, weights=w[-LAST:].clone())
    same(dx[:LAST], part[:LAST])
    same(dw[-LAST:], dwl)
    # and the first tokens the last rows
    part, dwl = bsq_gpu.bsq_moe_combine_bwd(few[:LAST].clone(), few, own + LAST, weights=w[:LAST].clone())
    same(dx[-LAST:], part[LAST:])
    same(dw[:LAST], dwl)


def test_tokens(bsq_gpu):
    """Quantizer and products of many tokens, the last of two experts with few of them."""
    x = randn(ROWS, WIDTH)
    off, off_few = ints(0, ROWS - LAST, ROWS), ints(0, 0, LAST)
    row, t = bsq_gpu.bsq_quantize_fp8b128(x, offsets=off)
    row_few, t_few = bsq_gpu.bsq_quantize_fp8b128(x[-LAST:].clone(), offsets=off_few)
    rows_alone = bsq_gpu.bsq_quantize_fp8b128(x)[0]
    for r in (row, rows_alone):
        same(r[0][-LAST:], row_few[0])
        same(r[1][:, -LAST:], row_few[1])
    del rows_alone
    b, nb = 1 + (ROWS - LAST) // 128, (LAST + 127) // 128
    same(t[0][:, 128 * b:128 * (b + nb)], t_few[0][:, 128:128 * (1 + nb)])
    same(t[1][b:b + nb], t_few[1][1:1 + nb])
    index = torch.arange(ROWS - 1, ROWS - 1 - LAST, -1, dtype=torch.int32, device="cuda")
    gathered = bsq_gpu.bsq_quantize_fp8b128(x, row_index=index)[0]
    same(gathered[0], row_few[0].flip(0))
    del x
    codes, codes_t, scale = bsq_gpu.bsq_quantize_fp8b128_weights(randn(2 * WIDTH, WIDTH), 2)
    y = bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row, (codes, scale), off)
    same(y[-LAST:], bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row_few, (codes, scale), off_few))
    del y
    kw = dict(wt_q=(codes_t, scale), dw_dtype=bsq_gpu.BSQ_F32)
    dx, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off, ROWS, WIDTH, WIDTH, dy_q=row, dyt_q=t, xt_q=t, **kw)
    dx_few, dw_few = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off_few, LAST, WIDTH, WIDTH, dy_q=row_few, dyt_q=t_few,
                                                          xt_q=t_few, **kw)
    same(dx[-LAST:], dx_few)
    same(dw[1], dw_few[1])


def test_weights(bsq_gpu):
    E = 2 ** 31 // WIDTH ** 2 + 2
    w = randn(E * WIDTH, WIDTH)
    codes, codes_t, scale = bsq_gpu.bsq_quantize_fp8b128_weights(w, E)
    few = bsq_gpu.bsq_quantize_fp8b128_weights(w[-2 * WIDTH:].clone(), 2)
    del w
    for got, ref in ((codes, few[0]), (codes_t, few[1]), (scale.view(E, -1), few[2].view(2, -1))):
        same(got[-ref.shape[0]:], ref)
    # the last expert's rows in each form of the product
    for rows in (3, LAST):
        row, t = bsq_gpu.bsq_quantize_fp8b128(randn(rows, WIDTH), offsets=ints(*[0] * E, rows))
        off, off_few = ints(*[0] * E, rows), ints(0, 0, rows)
        same(bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row, (codes, scale), off),
             bsq_gpu.bsq_grouped_gemm_fp8b128_fwd(row, (few[0], few[2]), off_few))
        dx, dw = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off, rows, WIDTH, WIDTH, dy_q=row, wt_q=(codes_t, scale), dyt_q=t,
                                                      xt_q=t)
        _, t = bsq_gpu.bsq_quantize_fp8b128(randn(rows, WIDTH), offsets=off_few)
        dx_few, dw_few = bsq_gpu.bsq_grouped_gemm_fp8b128_bwd(off_few, rows, WIDTH, WIDTH, dy_q=row,
                                                              wt_q=(few[1], few[2]), dyt_q=t, xt_q=t)
        same(dx, dx_few)
        same(dw[-1], dw_few[1])
        assert not dw[:-1].any()
        del dw
