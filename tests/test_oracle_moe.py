"""Pins of the 64-bit routing, dispatch, combine and FP8B128 implementations
the GPU tests compare with: closed forms, differences and torch."""
import numpy as np
import pytest
import torch

from oracle import moe


def test_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 5.0], [4.0, 4.0, 8.0]]))
    ids, w, lse, counts, loss = moe.route(l, 2, normalize=False, coef=1.0)
    assert ids.tolist() == [[2, 1], [2, 0]]              # ties go to the lowest index
    assert np.allclose(w, [[5 / 8, 2 / 8], [1 / 2, 1 / 4]], rtol=1e-14)
    assert np.allclose(lse, np.log([8.0, 16.0]), rtol=1e-14)
    assert counts.tolist() == [1, 1, 2, 2]
    P = np.array([1 / 8 + 1 / 4, 2 / 8 + 1 / 4, 5 / 8 + 1 / 2]) / 2
    assert np.isclose(loss, 3 / (2 * 2) * (np.array([1, 1, 2]) * P).sum(), rtol=1e-14)
    assert np.allclose(moe.route(l, 2, normalize=True, scale=3.0)[1], [[15 / 7, 6 / 7], [2, 1]], rtol=1e-14)
    ids, w, *_ = moe.route(l, 2, bias=np.array([9.0, 0, 0]), normalize=False)
    assert ids.tolist() == [[0, 2], [0, 2]] and np.isclose(w[0, 0], 1 / 8)  # the bias selects only


def test_route_edges():
    l = np.full((3, 4), -np.inf)
    l[1, 2] = 7.0
    l[2] = [np.nan, 3.0, np.inf, -np.inf]
    ids, w, lse, counts, _ = moe.route(l, 3)
    assert ids.tolist() == [[-1] * 3, [2, -1, -1], [2, 1, -1]]
    assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0] and w[2, 0] == 1.0
    assert lse[0] == -np.inf and counts.tolist() == [0, 1, 2, 0, 2]
    assert moe.route(l, 3, mask=[1, 0, 0])[3].tolist() == [0] * 5


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_against_differences(normalize):
    rng = np.random.default_rng(3)
    T, E, K, coef, scale = 5, 7, 3, 0.7, 1.5
    l = rng.standard_normal((T, E)) * 2
    l[1, 2] = -np.inf
    dw, dl = rng.standard_normal((T, K)), 1.3
    ids, _, _, counts, _ = moe.route(l, K, normalize=normalize, scale=scale, coef=coef)

    def value(x):
        i, w, _, c, loss = moe.route(x, K, normalize=normalize, scale=scale, coef=coef)
        assert (i == ids).all() and (c == counts).all()
        return (w * dw).sum() + dl * loss

    d = moe.route_bwd(l, ids, counts, dw, dl, normalize=normalize, scale=scale, coef=coef)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(l[t, e]):
                assert d[t, e] == 0
                continue
            p, m = l.copy(), l.copy()
            p[t, e] += h
            m[t, e] -= h
            assert abs((value(p) - value(m)) / (2 * h) - d[t, e]) < 1e-7


def test_dispatch_against_stable_sort():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 7, (50, 3)).astype(np.int32)
    off, row, slot = moe.dispatch(ids, 6)
    flat = np.where((ids < 0) | (ids >= 6), 6, ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    m = int((flat < 6).sum())
    assert off.tolist() == [int((flat < e).sum()) for e in range(7)] and off[-1] == m
    assert (row[:m] == order[:m] // 3).all() and (row[m:] == -1).all()
    assert (slot.reshape(-1)[order[:m]] == np.arange(m)).all() and (slot.reshape(-1)[order[m:]] == -1).all()


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 4, (6, 2)).astype(np.int32)
    off, _, slot = moe.dispatch(ids, 4)
    ye, w, dy = rng.standard_normal((12, 3)), rng.random((6, 2)), rng.standard_normal((6, 3))
    dye, dw = moe.combine_bwd(dy, ye, slot, w)
    f = lambda a, b: (moe.combine(a, slot, b) * dy).sum()
    for a, d in ((ye, dye), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 0.5
            hi = f(ye, w)
            a[i] = old - 0.5
            lo = f(ye, w)
            a[i] = old
            assert abs(hi - lo - d[i]) < 1e-12   # linear in each entry
    assert (dye[off[-1]:] == 0).all()


def test_e4m3_against_torch():
    c = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(c.copy()).view(torch.float8_e4m3fn).double().numpy()
    ok = ~np.isnan(v)
    assert (moe.e4m3_decode(c)[ok] == v[ok]).all() and np.isnan(moe.e4m3_decode(c)[~ok]).all()
    assert (moe.e4m3_encode(v[ok]) == c[ok]).all()
    x = np.random.default_rng(6).standard_normal(20000).astype(np.float32) * np.float32(100)
    x[:2000] *= np.float32(1e-4)
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (moe.e4m3_encode(x) == ref).all()


def test_b128_forms():
    rng = np.random.default_rng(7)
    x = torch.from_numpy(rng.standard_normal((200, 272)).astype(np.float32)).bfloat16().float().numpy()
    x[3, 128:256] = 0
    codes, scale = moe.b128_rows(x)
    assert scale.shape == (3, 200) and scale[1, 3] == 0 and (codes[3, 128:256] == 0).all()
    assert scale[0, 0] == np.float32(np.abs(x[0, :128]).max()) / np.float32(448)
    # the largest element of a block is code 0x7E (448), others within half a step of E4M3
    assert ((codes[:, :128] & 0x7F).max(1) == 0x7E).all()
    amax = np.repeat(scale, 128, 0)[:272].T * 448
    assert (np.abs(moe.b128_value(codes, scale) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, amax * 2.0 ** -18) * 1.001).all()
    off = np.array([0, 130, 130, 190], np.int32)
    tc, ts = moe.b128_columns(x, off)
    assert tc.shape == (272, 128 * 5) and ts.shape == (5, 272)
    seg, sc = moe.b128_rows(np.ascontiguousarray(x[:130].T))
    assert (tc[:, :130] == seg).all() and (ts[:2] == sc).all() and (tc[:, 130:256] == 0).all()
    seg, sc = moe.b128_rows(np.ascontiguousarray(x[130:190].T))   # group 2 starts at block 2 + 130 // 128
    assert (tc[:, 384:444] == seg).all() and (ts[3] == sc[0]).all()
    assert (tc[:, 444:] == 0).all() and (ts[2] == 0).all() and (ts[4] == 0).all()
    c, ct, s = moe.b128_weights(x[:192], 1)
    assert s.shape == (1, 2, 3) and (ct == c.T).all()
    assert s[0, 1, 2] == np.float32(np.abs(x[128:192, 256:]).max()) / np.float32(448)


def test_b128_products_against_plain_matmul():
    """Operands the format holds exactly (integers, block maxima 448): the products are exact."""
    rng = np.random.default_rng(8)
    grid = np.array([0, 1, 2, 4, 8, 16, 448.0])
    a, w = rng.choice(grid, (40, 256)), rng.choice(grid, (2 * 48, 256))
    a[:, ::128], w[:, ::128] = 448, 448
    off = np.array([0, 25, 40], np.int32)
    wq, wt, ws = moe.b128_weights(w.astype(np.float32), 2)
    aq = moe.b128_rows(a.astype(np.float32))
    y, _ = moe.b128_gemm_fwd(aq, (wq, ws), off, 48)
    assert (y[:25] == a[:25] @ w[:48].T).all() and (y[25:] == a[25:] @ w[48:].T).all()
    g = rng.choice(grid, (40, 48))
    g[:, 0] = 448
    dx, _ = moe.b128_gemm_dgrad(moe.b128_rows(g.astype(np.float32)), wt, ws, off, 256)
    assert (dx[:25] == g[:25] @ w[:48]).all() and (dx[25:] == g[25:] @ w[48:]).all()
    a[[0, 25]], g[[0, 25]] = 448, 448
    dw, _ = moe.b128_gemm_wgrad(moe.b128_columns(g.astype(np.float32), off), moe.b128_columns(a.astype(np.float32), off), off)
    assert (dw[0] == g[:25].T @ a[:25]).all() and (dw[1] == g[25:].T @ a[25:]).all()
