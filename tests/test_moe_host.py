"""Refusals of the routing, dispatch, combine and FP8B128 entry points, on the
host: the pointers are never dereferenced."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100001)
BIG = 1 << 40


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_amd as b
    return b


def test_route(bsq):
    f = bsq._lib.bsq_moe_route
    need = bsq.bsq_moe_route_workspace_size(100, 64)
    assert need > 0 and need % 256 == 0
    assert bsq.bsq_moe_route_workspace_size(100, 1025) == 0 and bsq.bsq_moe_route_workspace_size(-1, 4) == 0

    def call(logits=FAKE, dt=0, T=100, E=64, ld=64, K=8, ids=FAKE, counts=FAKE, ws=FAKE, wb=need):
        return f(logits, dt, T, E, ld, K, None, None, 1, 1.0, 0.0, ids, FAKE, FAKE, counts, FAKE, ws, wb, None)

    assert call(logits=None) == call(ids=None) == call(counts=None) == call(ws=None) == bsq.BSQ_ERR_INVALID_ARG
    assert call(K=0) == call(K=65) == call(T=-1) == call(E=0) == call(ld=63) == call(dt=2) == bsq.BSQ_ERR_INVALID_ARG
    assert call(E=1025, ld=1025) == call(E=128, ld=128, K=65) == call(T=1 << 31) == bsq.BSQ_ERR_UNSUPPORTED
    assert call(logits=ODD) == call(ws=ctypes.c_void_p(0x100010)) == bsq.BSQ_ERR_UNSUPPORTED
    assert call(wb=need - 1) == bsq.BSQ_ERR_WORKSPACE_TOO_SMALL
    g = bsq._lib.bsq_moe_route_bwd

    def back(T=4, E=8, ld=8, K=2, ids=FAKE, d=FAKE, ldd=8):
        return g(FAKE, 1, T, E, ld, K, ids, FAKE, FAKE, FAKE, None, None, 1, 1.0, 0.0, d, ldd, None)

    assert back(ids=None) == back(d=None) == back(ld=7) == back(ldd=7) == back(K=9) == bsq.BSQ_ERR_INVALID_ARG
    assert back(d=ODD) == back(E=1025, ld=1025, ldd=1025) == bsq.BSQ_ERR_UNSUPPORTED
    assert back(T=0) == bsq.BSQ_OK


def test_dispatch(bsq):
    f = bsq._lib.bsq_moe_dispatch
    need = bsq.bsq_moe_dispatch_workspace_size(100, 8, 64)
    assert bsq.bsq_moe_dispatch_workspace_size(100, 8, 1025) == 0

    def call(ids=FAKE, T=100, K=8, E=64, off=FAKE, ws=FAKE, wb=need):
        return f(ids, T, K, E, off, FAKE, FAKE, ws, wb, None)

    assert call(ids=None) == call(off=None) == call(ws=None) == bsq.BSQ_ERR_INVALID_ARG
    assert call(T=-1) == call(K=0) == call(E=0) == bsq.BSQ_ERR_INVALID_ARG
    assert call(E=1025) == call(T=1 << 28) == call(ids=ODD) == bsq.BSQ_ERR_UNSUPPORTED
    assert call(wb=need - 1) == bsq.BSQ_ERR_WORKSPACE_TOO_SMALL


def test_combine(bsq):
    f = bsq._lib.bsq_moe_combine

    def call(ye=FAKE, dt=0, M=64, W=64, ld=64, slot=FAKE, T=8, K=8, y=FAKE, ldy=64):
        return f(ye, dt, M, W, ld, slot, None, T, K, y, ldy, None)

    assert call(ye=None) == call(slot=None) == call(y=None) == call(ld=63) == call(ldy=63) == bsq.BSQ_ERR_INVALID_ARG
    assert call(dt=5) == call(M=-1) == call(K=0) == bsq.BSQ_ERR_INVALID_ARG
    assert call(W=60) == call(ld=68) == call(ldy=68) == call(ye=ODD) == call(T=1 << 24) == bsq.BSQ_ERR_UNSUPPORTED
    assert call(T=0) == call(W=0) == bsq.BSQ_OK
    g = bsq._lib.bsq_moe_combine_bwd

    def back(dy=FAKE, W=64, ld=64, ye=FAKE, slot=FAKE, dye=FAKE, ldd=64, dw=FAKE, T=8):
        return g(dy, 1, T, W, ld, ye, 64, 64, slot, None, 8, None, 0, dye, ldd, dw, None)

    assert back(dy=None) == back(ye=None) == back(slot=None) == back(dye=None) == bsq.BSQ_ERR_INVALID_ARG
    assert back(ldd=60) == back(ld=60) == bsq.BSQ_ERR_INVALID_ARG
    assert back(W=0) == back(ld=68) == back(dye=ODD) == back(T=1 << 24) == bsq.BSQ_ERR_UNSUPPORTED


def test_quantize(bsq):
    f = bsq._lib.bsq_quantize_fp8b128

    def call(x=FAKE, src=64, C=64, ld=64, idx=None, R=64, off=FAKE, G=2, c=FAKE, s=FAKE, tc=FAKE, ts=FAKE):
        return f(x, src, C, ld, idx, R, off, G, c, s, tc, ts, None)

    inv, uns = bsq.BSQ_ERR_INVALID_ARG, bsq.BSQ_ERR_UNSUPPORTED
    assert call(x=None) == call(s=None) == call(ts=None) == call(off=None) == call(G=0) == call(R=65) == inv
    assert call(c=None, s=None, tc=None, ts=None) == call(ld=63) == call(R=-1) == inv
    assert call(C=56) == call(ld=68) == call(x=ODD) == call(tc=ODD) == call(idx=ODD) == uns
    assert call(src=BIG, R=BIG) == call(idx=FAKE, R=(1 << 27) + 1) == call(C=1 << 23, ld=1 << 23) == uns
    assert call(src=1 << 24, R=1 << 24, ) == uns                      # token columns beyond the grid
    assert call(C=0, ld=0) == bsq.BSQ_OK
    w = bsq._lib.bsq_quantize_fp8b128_weights
    assert w(None, 2, 64, 64, 64, FAKE, FAKE, FAKE, None) == w(FAKE, 2, 64, 64, 48, FAKE, FAKE, FAKE, None) == inv
    assert w(FAKE, 2, 64, 64, 64, FAKE, FAKE, None, None) == w(FAKE, -1, 64, 64, 64, FAKE, FAKE, FAKE, None) == inv
    assert w(FAKE, 2, 60, 64, 64, FAKE, FAKE, FAKE, None) == w(FAKE, 2, 64, 72, 72, FAKE, FAKE, FAKE, None) == uns
    assert w(FAKE, 70000, 64, 64, 64, FAKE, FAKE, FAKE, None) == w(FAKE, 2, 64, 64, 64, FAKE, ODD, FAKE, None) == uns
    assert w(FAKE, 0, 64, 64, 64, FAKE, FAKE, FAKE, None) == bsq.BSQ_OK


def test_gemm(bsq):
    need = bsq.bsq_grouped_gemm_fp8b128_workspace_size(4)
    assert need > 0 and bsq.bsq_grouped_gemm_fp8b128_workspace_size(0) == 0
    assert bsq.bsq_grouped_gemm_fp8b128_workspace_size(4097) == 0
    inv, uns = bsq.BSQ_ERR_INVALID_ARG, bsq.BSQ_ERR_UNSUPPORTED

    def fwd(a=FAKE, w=FAKE, off=FAKE, E=4, M=64, n=64, k=128, y=FAKE, dt=0, ws=FAKE, wb=need):
        return bsq._lib.bsq_grouped_gemm_fp8b128_fwd(a, FAKE, w, FAKE, off, E, M, n, k, y, dt, ws, wb, None)

    assert fwd(a=None) == fwd(w=None) == fwd(off=None) == fwd(y=None) == fwd(ws=None) == inv
    assert fwd(E=0) == fwd(M=-1) == fwd(dt=2) == inv
    assert fwd(n=0) == fwd(n=72) == fwd(k=120) == fwd(E=4097) == fwd(a=ODD) == fwd(y=ODD) == uns
    assert fwd(k=1 << 23) == fwd(n=1 << 21) == fwd(M=1 << 29) == uns
    assert fwd(wb=need - 1) == bsq.BSQ_ERR_WORKSPACE_TOO_SMALL and fwd(M=0) == bsq.BSQ_OK

    def bwd(flags=3, dy=FAKE, wt=FAKE, dyt=FAKE, xt=FAKE, dx=FAKE, dw=FAKE, M=64, n=64, k=128, dt=0, wb=need):
        return bsq._lib.bsq_grouped_gemm_fp8b128_bwd(dy, FAKE, wt, FAKE, dyt, FAKE, xt, FAKE, FAKE, 4, M, n, k, dx, dt,
                                                     dw, dt, flags, FAKE, wb, None)

    assert bwd(flags=0) == bwd(flags=4) == bwd(dy=None) == bwd(wt=None) == bwd(dyt=None) == bwd(xt=None) == inv
    assert bwd(dx=None) == bwd(dw=None) == bwd(dt=3) == inv
    assert bwd(n=56) == bwd(k=0) == bwd(dw=ODD) == bwd(xt=ODD) == bwd(M=1 << 24) == bwd(k=1 << 21) == uns
    assert bwd(wb=need - 1) == bsq.BSQ_ERR_WORKSPACE_TOO_SMALL
    assert bwd(flags=bsq.BSQ_DGRAD, M=0, dw=None) == bsq.BSQ_OK


def test_binding_refuses_host_tensors_and_shapes(bsq):
    import torch
    with pytest.raises(TypeError):
        bsq.bsq_moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        bsq.bsq_moe_dispatch(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(TypeError):
        bsq.bsq_moe_combine(torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        bsq.bsq_quantize_fp8b128(torch.zeros(4, 16, dtype=torch.bfloat16))
