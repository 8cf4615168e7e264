"""Python binding of libbsq.so: block-scaled MoE expert grouped GEMM on MI355X.

Thin ctypes marshalling over the C ABI declared in ``include/bsq.h``: every
function here has the C entry point's name, checks tensor dtypes, shapes and
devices, passes raw device pointers plus torch's current HIP stream, and turns
a non-OK status into ``RuntimeError``.  All arithmetic runs in the HIP kernels;
torch only provides device memory and streams.  There is no CPU fallback:
importing this package fails if the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbsq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python block_scaled_precision_bsq_amd/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

P = ctypes.c_void_p
I64 = ctypes.c_int64
I32 = ctypes.c_int32
INT = ctypes.c_int
F32 = ctypes.c_float

BSQ_OK, BSQ_ERR_INVALID_ARG, BSQ_ERR_UNSUPPORTED, BSQ_ERR_WORKSPACE_TOO_SMALL, BSQ_ERR_HIP = range(5)
BSQ_BF16, BSQ_F32 = 0, 1
BSQ_ROWWISE, BSQ_COLWISE_T = 0, 1
BSQ_DGRAD, BSQ_WGRAD = 1, 2
BSQ_OP_GEMM_FWD, BSQ_OP_GEMM_BWD = 0, 1

_SIGS = {
    "bsq_quantize_nvfp4v": ([P, I64, I64, I64, P, I32, P, P, P, P], INT),
    "bsq_swiglu_quantize_nvfp4v": ([P, I64, I64, I64, P, I64, P, P, P, P], INT),
    "bsq_quantize_mxfp8_gather": ([P, I64, I64, I64, P, I64, P, P, P], INT),
    "bsq_debug_quantize_nvfp4v_fastdiv": ([P, I64, I64, I64, P, P, P, P], INT),
    "bsq_quantize_mxfp8": ([P, I64, I64, I64, INT, P, I32, P, P, P], INT),
    "bsq_quantize_mxfp8_dual": ([P, I64, I64, I64, P, I32, P, P, P, P, P], INT),
    "bsq_grouped_gemm_fwd": ([P, P, P, P, P, P, P, I32, I64, I64, I64, P, INT, P, ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_fwd_swiglu": ([P, P, P, P, P, P, P, I32, I64, I64, I64, P, I64, P, ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_fwd_noalloc": ([P, P, P, P, P, P, P, I32, I64, I64, I64, P, INT, P], INT),
    "bsq_grouped_gemm_bwd": ([P, P, P, P, P, P, P, P, P, I32, I64, I64, I64, P, INT, P, INT, ctypes.c_uint, P,
                              ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_fwd_mxfp8": ([P, P, P, P, P, I32, I64, I64, I64, P, INT, P, ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_bf16": ([P, P, P, I32, I64, I64, I64, P, INT, P, ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_w4a16": ([P, P, P, P, P, I32, I64, I64, I64, P, INT, P, ctypes.c_size_t, P], INT),
    "bsq_moe_route": ([P, INT, I64, I32, I64, I32, P, P, I32, F32, F32, P, P, P, P, P, P, ctypes.c_size_t, P], INT),
    "bsq_moe_route_workspace_size": ([I64, I32], ctypes.c_size_t),
    "bsq_moe_route_bwd": ([P, INT, I64, I32, I64, I32, P, P, P, P, P, P, I32, F32, F32, P, I64, P], INT),
    "bsq_moe_dispatch": ([P, I64, I32, I32, P, P, P, P, ctypes.c_size_t, P], INT),
    "bsq_moe_dispatch_workspace_size": ([I64, I32, I32], ctypes.c_size_t),
    "bsq_moe_combine": ([P, INT, I64, I64, I64, P, P, I64, I32, P, I64, P], INT),
    "bsq_moe_combine_bwd": ([P, INT, I64, I64, I64, P, I64, I64, P, P, I32, P, I32, P, I64, P, P], INT),
    "bsq_quantize_fp8b128": ([P, I64, I64, I64, P, I64, P, I32, P, P, P, P, P], INT),
    "bsq_quantize_fp8b128_weights": ([P, I32, I64, I64, I64, P, P, P, P], INT),
    "bsq_grouped_gemm_fp8b128_fwd": ([P, P, P, P, P, I32, I64, I64, I64, P, INT, P, ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_fp8b128_bwd": ([P, P, P, P, P, P, P, P, P, I32, I64, I64, I64, P, INT, P, INT, ctypes.c_uint, P,
                                      ctypes.c_size_t, P], INT),
    "bsq_grouped_gemm_fp8b128_workspace_size": ([I32], ctypes.c_size_t),
    "bsq_workspace_size": ([INT, I32, I64, I64, I64], ctypes.c_size_t),
    "bsq_colwise_padded_cols": ([I32, I64], I64),
    "bsq_status_string": ([INT], ctypes.c_char_p),
    "bsq_abi_version": ([], INT),
    "bsq_debug_status": ([P, P, ctypes.POINTER(I32)], INT),
    "bsq_debug_encode_e2m1": ([P, P, I64, P], INT),
    "bsq_debug_encode_e4m3": ([P, P, I64, P], INT),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

ABI_VERSION = _lib.bsq_abi_version()


class BsqError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {_lib.bsq_status_string(status).decode()} (status {status})")
        self.status = status


def _check(fn, status):
    if status != BSQ_OK:
        raise BsqError(fn, status)


def _stream(stream=None):
    # the raw handle: building a torch.cuda.Stream costs 3 us, a third of a small call
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _empty(stream, shape, dtype, device):
    """torch.empty on the caching allocator's pool of ``stream`` when one is
    given: a block freed here (the workspace) or later (an output) is then
    reused only in ``stream``'s order, never while its kernels still run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# Bytes of outputs and workspace up to which one allocation holds all of them (an
# allocation apiece costs such a call more time than its kernel).
_SMALL = 1 << 14


def _carve(stream, dtype, device, sizes, scratch=0):
    """Dense 1-D tensors of the given lengths out of one allocation (4-byte types),
    and the address of ``scratch`` bytes of workspace on 256 bytes (last, where
    wanted).  Each is a tensor of its own (.data): an in-place change of one, an
    all-reduce of counts say, does not count as a change of another that
    autograd has saved."""
    if not scratch:
        return [t.data for t in _empty(stream, (sum(sizes),), dtype, device).split_with_sizes(sizes)]
    n = sum(sizes)
    base = _empty(stream, (n + scratch // 4 + 64,), dtype, device)
    *out, _ = base.split_with_sizes((*sizes, scratch // 4 + 64))
    return [t.data for t in out] + [(base.data_ptr() + 4 * n + 255) & -256]


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _dev(t, name, dtypes):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _rows_ld(x):
    if x.dim() != 2:
        raise ValueError("x must be a 2-D matrix")
    rows, cols = x.shape
    if rows == 0 or cols == 0:
        return rows, cols, cols
    if x.stride(1) != 1 and cols > 1:
        raise ValueError("x must be row-major (unit column stride)")
    return rows, cols, x.stride(0) if rows > 1 else cols


def bsq_workspace_size(op, num_experts, m_total, n, k):
    return int(_lib.bsq_workspace_size(op, num_experts, m_total, n, k))


def bsq_colwise_padded_cols(num_groups, rows):
    return int(_lib.bsq_colwise_padded_cols(num_groups, rows))


def bsq_quantize_nvfp4v(x, codes=None, bscale=None, rscale=None, offsets=None, stream=None):
    """NVFP4-variant quantization of each row of bf16 ``x`` [rows, cols].
    Returns (codes u8 [rows, cols/2], bscale u8 [rows, cols/16], rscale f32 [rows])."""
    _dev(x, "x", _BF16)
    rows, cols, ld = _rows_ld(x)
    dev = x.device
    codes = _empty(stream, (rows, cols // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    bscale = _empty(stream, (rows, cols // 16), dtype=torch.uint8, device=dev) if bscale is None else bscale
    rscale = _empty(stream, (rows,), dtype=torch.float32, device=dev) if rscale is None else rscale
    for t, nm, shape in ((codes, "codes", (rows, cols // 2)), (bscale, "bscale", (rows, cols // 16)),
                         (rscale, "rscale", (rows,))):
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
    ng = 0 if offsets is None else offsets.numel() - 1
    _check("bsq_quantize_nvfp4v",
           _lib.bsq_quantize_nvfp4v(_ptr(x), rows, cols, ld, _ptr(offsets), ng, _ptr(codes), _ptr(bscale),
                                    _ptr(rscale), _stream(stream)))
    return codes, bscale, rscale


def bsq_debug_quantize_nvfp4v_fastdiv(x, stream=None):
    """Ablation: bsq_quantize_nvfp4v with fast approximate divides (reciprocal
    approximation times numerator).  Returns (codes, bscale, rscale)."""
    _dev(x, "x", _BF16)
    rows, cols, ld = _rows_ld(x)
    dev = x.device
    codes = _empty(stream, (rows, cols // 2), dtype=torch.uint8, device=dev)
    bscale = _empty(stream, (rows, cols // 16), dtype=torch.uint8, device=dev)
    rscale = _empty(stream, (rows,), dtype=torch.float32, device=dev)
    _check("bsq_debug_quantize_nvfp4v_fastdiv",
           _lib.bsq_debug_quantize_nvfp4v_fastdiv(_ptr(x), rows, cols, ld, _ptr(codes), _ptr(bscale), _ptr(rscale),
                                                  _stream(stream)))
    return codes, bscale, rscale


def bsq_quantize_mxfp8_gather(x, row_index, codes=None, scale=None, stream=None):
    """MXFP8 ROWWISE quantization of the rows ``x[row_index]`` (int32 device
    indices; out-of-range indices give zero rows) in one pass.
    Returns (codes [rows, cols], scale [cols/32, rows])."""
    _dev(x, "x", _BF16)
    _dev(row_index, "row_index", (torch.int32,))
    src_rows, cols, ld = _rows_ld(x)
    rows = row_index.numel()
    dev = x.device
    codes = _empty(stream, (rows, cols), dtype=torch.uint8, device=dev) if codes is None else codes
    scale = _empty(stream, (cols // 32, rows), dtype=torch.uint8, device=dev) if scale is None else scale
    for t, nm, shape in ((codes, "codes", (rows, cols)), (scale, "scale", (cols // 32, rows))):
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
    _check("bsq_quantize_mxfp8_gather",
           _lib.bsq_quantize_mxfp8_gather(_ptr(x), src_rows, cols, ld, _ptr(row_index), rows, _ptr(codes),
                                          _ptr(scale), _stream(stream)))
    return codes, scale


def bsq_swiglu_quantize_nvfp4v(gu, h=None, write_h=True, codes=None, bscale=None, rscale=None, stream=None):
    """SwiGLU of bf16 ``gu`` [rows, 2*inter] ([gate | up] per row) fused with the
    NVFP4-variant quantization of H = bf16(silu(gate) * up).
    Returns (h bf16 [rows, inter] or None, codes u8 [rows, inter/2],
    bscale u8 [rows, inter/16], rscale f32 [rows])."""
    _dev(gu, "gu", _BF16)
    rows, cols2, ld = _rows_ld(gu)
    if cols2 % 2:
        raise ValueError("gu must have an even number of columns ([gate | up])")
    inter = cols2 // 2
    dev = gu.device
    if write_h and h is None:
        h = _empty(stream, (rows, inter), dtype=torch.bfloat16, device=dev)
    if h is not None:
        _dev(h, "h", _BF16)
        if tuple(h.shape) != (rows, inter) or (rows > 1 and h.stride(1) != 1):
            raise ValueError(f"h must be row-major with shape {(rows, inter)}")
    ldh = 0 if h is None else (h.stride(0) if rows > 1 else inter)
    codes = _empty(stream, (rows, inter // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    bscale = _empty(stream, (rows, inter // 16), dtype=torch.uint8, device=dev) if bscale is None else bscale
    rscale = _empty(stream, (rows,), dtype=torch.float32, device=dev) if rscale is None else rscale
    for t, nm, shape in ((codes, "codes", (rows, inter // 2)), (bscale, "bscale", (rows, inter // 16)),
                         (rscale, "rscale", (rows,))):
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
    _check("bsq_swiglu_quantize_nvfp4v",
           _lib.bsq_swiglu_quantize_nvfp4v(_ptr(gu), rows, inter, ld, _ptr(h), ldh, _ptr(codes), _ptr(bscale),
                                           _ptr(rscale), _stream(stream)))
    return h, codes, bscale, rscale


def bsq_quantize_mxfp8(x, axis=BSQ_ROWWISE, offsets=None, codes=None, scale=None, stream=None):
    """MXFP8 quantization of bf16 ``x`` [rows, cols]; scales are block-major.
    ROWWISE: (codes [rows, cols], scale [cols/32, rows]).
    COLWISE_T (needs int32 device ``offsets``): (codes [cols, P], scale [P/32, cols])."""
    _dev(x, "x", _BF16)
    rows, cols, ld = _rows_ld(x)
    dev = x.device
    if axis == BSQ_ROWWISE:
        shapes = ((rows, cols), (cols // 32, rows))
        ng = 0
    else:
        if offsets is None:
            raise ValueError("COLWISE_T needs offsets")
        _dev(offsets, "offsets", (torch.int32,))
        ng = offsets.numel() - 1
        Pc = bsq_colwise_padded_cols(ng, rows)
        shapes = ((cols, Pc), (Pc // 32, cols))
    codes = _empty(stream, shapes[0], dtype=torch.uint8, device=dev) if codes is None else codes
    scale = _empty(stream, shapes[1], dtype=torch.uint8, device=dev) if scale is None else scale
    for t, nm, shape in ((codes, "codes", shapes[0]), (scale, "scale", shapes[1])):
        if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
    _check("bsq_quantize_mxfp8",
           _lib.bsq_quantize_mxfp8(_ptr(x), rows, cols, ld, axis, _ptr(offsets), ng, _ptr(codes), _ptr(scale),
                                   _stream(stream)))
    return codes, scale


def bsq_quantize_mxfp8_dual(x, offsets, row=None, t=None, stream=None):
    """Both MXFP8 layouts of bf16 ``x`` [rows, cols] from one read: returns
    ((codes [rows, cols], scale [cols/32, rows]) as ROWWISE,
     (codes [cols, P], scale [P/32, cols]) as COLWISE_T with int32 ``offsets``)."""
    _dev(x, "x", _BF16)
    _dev(offsets, "offsets", (torch.int32,))
    rows, cols, ld = _rows_ld(x)
    dev = x.device
    ng = offsets.numel() - 1
    Pc = bsq_colwise_padded_cols(ng, rows)
    shapes = ((rows, cols), (cols // 32, rows), (cols, Pc), (Pc // 32, cols))
    rc, rs = (None, None) if row is None else row
    tc, ts = (None, None) if t is None else t
    outs = []
    for buf, nm, shape in ((rc, "row codes", shapes[0]), (rs, "row scale", shapes[1]),
                           (tc, "t codes", shapes[2]), (ts, "t scale", shapes[3])):
        buf = _empty(stream, shape, dtype=torch.uint8, device=dev) if buf is None else buf
        if tuple(buf.shape) != tuple(shape) or not buf.is_contiguous():
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
        outs.append(buf)
    _check("bsq_quantize_mxfp8_dual",
           _lib.bsq_quantize_mxfp8_dual(_ptr(x), rows, cols, ld, _ptr(offsets), ng, *[_ptr(o) for o in outs],
                                        _stream(stream)))
    return (outs[0], outs[1]), (outs[2], outs[3])


def _workspace(op, E, m_total, n, k, workspace, dev, stream=None):
    need = bsq_workspace_size(op, E, m_total, n, k)
    if workspace is None:
        workspace = _empty(stream, (need,), dtype=torch.uint8, device=dev)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    return workspace


def bsq_grouped_gemm_fwd(a_q, w_q, offsets, n, k, y_dtype=BSQ_BF16, y=None, workspace=None, stream=None):
    """Forward grouped GEMM.  a_q / w_q = (codes, bscale, rscale) of the
    expert-sorted activations [m_total, k] and of the weights [E*n, k]."""
    a_codes, a_bscale, a_rscale = a_q
    w_codes, w_bscale, w_rscale = w_q
    _dev(offsets, "offsets", (torch.int32,))
    E = offsets.numel() - 1
    m_total = a_codes.shape[0]
    if w_codes.shape[0] != E * n:
        raise ValueError("weights must hold num_experts * n rows")
    dev = a_codes.device
    if y is None:
        y = _empty(stream, (m_total, n), dtype=torch.float32 if y_dtype == BSQ_F32 else torch.bfloat16, device=dev)
    workspace = _workspace(BSQ_OP_GEMM_FWD, E, m_total, n, k, workspace, dev, stream)
    _check("bsq_grouped_gemm_fwd",
           _lib.bsq_grouped_gemm_fwd(_ptr(a_codes), _ptr(a_bscale), _ptr(a_rscale), _ptr(w_codes), _ptr(w_bscale),
                                     _ptr(w_rscale), _ptr(offsets), E, m_total, n, k, _ptr(y), y_dtype,
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)))
    return y


def bsq_grouped_gemm_fwd_swiglu(a_q, w_q, offsets, inter, k, h=None, workspace=None, stream=None):
    """Gate/up grouped GEMM with the SwiGLU activation in its epilogue.
    a_q = NVFP4v (codes, bscale, rscale) of the expert-sorted activations
    [m_total, k]; w_q = NVFP4v of the gate/up weights [E*2*inter, k] ([gate;
    up] rows per expert).  Returns h bf16 [m_total, inter]; the gate/up output
    is never written."""
    a_codes, a_bscale, a_rscale = a_q
    w_codes, w_bscale, w_rscale = w_q
    _dev(offsets, "offsets", (torch.int32,))
    E = offsets.numel() - 1
    m_total = a_codes.shape[0]
    if w_codes.shape[0] != E * 2 * inter:
        raise ValueError("weights must hold num_experts * 2 * inter rows")
    dev = a_codes.device
    if h is None:
        h = _empty(stream, (m_total, inter), dtype=torch.bfloat16, device=dev)
    _dev(h, "h", _BF16)
    if tuple(h.shape) != (m_total, inter) or (m_total > 1 and h.stride(1) != 1):
        raise ValueError(f"h must be row-major with shape {(m_total, inter)}")
    ldh = h.stride(0) if m_total > 1 else inter
    workspace = _workspace(BSQ_OP_GEMM_FWD, E, m_total, 2 * inter, k, workspace, dev, stream)
    _check("bsq_grouped_gemm_fwd_swiglu",
           _lib.bsq_grouped_gemm_fwd_swiglu(_ptr(a_codes), _ptr(a_bscale), _ptr(a_rscale), _ptr(w_codes),
                                            _ptr(w_bscale), _ptr(w_rscale), _ptr(offsets), E, m_total, inter, k,
                                            _ptr(h), ldh, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _stream(stream)))
    return h


def bsq_grouped_gemm_fwd_noalloc(a_q, w_q, offsets, n, k, y_dtype=BSQ_BF16, y=None, stream=None):
    """bsq_grouped_gemm_fwd with the planner workspace inside the library (no
    workspace argument; the library allocates nothing).  ``y`` is allocated
    here only when not given."""
    a_codes, a_bscale, a_rscale = a_q
    w_codes, w_bscale, w_rscale = w_q
    _dev(offsets, "offsets", (torch.int32,))
    E = offsets.numel() - 1
    m_total = a_codes.shape[0]
    if w_codes.shape[0] != E * n:
        raise ValueError("weights must hold num_experts * n rows")
    if y is None:
        y = _empty(stream, (m_total, n), dtype=torch.float32 if y_dtype == BSQ_F32 else torch.bfloat16,
                   device=a_codes.device)
    _check("bsq_grouped_gemm_fwd_noalloc",
           _lib.bsq_grouped_gemm_fwd_noalloc(_ptr(a_codes), _ptr(a_bscale), _ptr(a_rscale), _ptr(w_codes),
                                             _ptr(w_bscale), _ptr(w_rscale), _ptr(offsets), E, m_total, n, k, _ptr(y),
                                             y_dtype, _stream(stream)))
    return y


def bsq_grouped_gemm_fwd_mxfp8(x_q, w_q, offsets, n, k, y_dtype=BSQ_BF16, y=None, workspace=None, stream=None):
    """Forward grouped GEMM over MXFP8 operands.  x_q / w_q = ROWWISE (codes,
    scale) of the expert-sorted activations [m_total, k] and of the weights
    [E*n, k] (block-major scales)."""
    x_codes, x_scale = x_q
    w_codes, w_scale = w_q
    _dev(offsets, "offsets", (torch.int32,))
    E = offsets.numel() - 1
    m_total = x_codes.shape[0]
    if w_codes.shape[0] != E * n:
        raise ValueError("weights must hold num_experts * n rows")
    dev = x_codes.device
    if y is None:
        y = _empty(stream, (m_total, n), dtype=torch.float32 if y_dtype == BSQ_F32 else torch.bfloat16, device=dev)
    workspace = _workspace(BSQ_OP_GEMM_FWD, E, m_total, n, k, workspace, dev, stream)
    _check("bsq_grouped_gemm_fwd_mxfp8",
           _lib.bsq_grouped_gemm_fwd_mxfp8(_ptr(x_codes), _ptr(x_scale), _ptr(w_codes), _ptr(w_scale),
                                           _ptr(offsets), E, m_total, n, k, _ptr(y), y_dtype, _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


def bsq_grouped_gemm_bf16(x, w, offsets, n, k, y_dtype=BSQ_BF16, y=None, workspace=None, stream=None):
    """bf16 baseline grouped GEMM: x [m_total, k] bf16, w [E*n, k] bf16."""
    _dev(x, "x", _BF16)
    _dev(w, "w", _BF16)
    _dev(offsets, "offsets", (torch.int32,))
    E = offsets.numel() - 1
    m_total = x.shape[0]
    for t, nm, shape in ((x, "x", (m_total, k)), (w, "w", (E * n, k))):
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
    dev = x.device
    if y is None:
        y = _empty(stream, (m_total, n), dtype=torch.float32 if y_dtype == BSQ_F32 else torch.bfloat16, device=dev)
    workspace = _workspace(BSQ_OP_GEMM_FWD, E, m_total, n, k, workspace, dev, stream)
    _check("bsq_grouped_gemm_bf16",
           _lib.bsq_grouped_gemm_bf16(_ptr(x), _ptr(w), _ptr(offsets), E, m_total, n, k, _ptr(y), y_dtype,
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream)))
    return y


def bsq_grouped_gemm_w4a16(x, w_q, offsets, n, k, y_dtype=BSQ_BF16, y=None, workspace=None, stream=None):
    """Frozen-expert GEMM: x [m_total, k] bf16 against packed weights
    w_q = (codes [E*n, k/2], bscale [E*n, k/16], rscale [E*n]) from
    bsq_quantize_nvfp4v, dequantized to bf16 inside the kernel."""
    _dev(x, "x", _BF16)
    _dev(offsets, "offsets", (torch.int32,))
    w_codes, w_bscale, w_rscale = w_q
    E = offsets.numel() - 1
    m_total = x.shape[0]
    for t, nm, shape, dt in ((x, "x", (m_total, k), None), (w_codes, "w codes", (E * n, k // 2), torch.uint8),
                             (w_bscale, "w bscale", (E * n, k // 16), torch.uint8),
                             (w_rscale, "w rscale", (E * n,), torch.float32)):
        if tuple(t.shape) != shape or not t.is_contiguous() or (dt is not None and t.dtype != dt):
            raise ValueError(f"{nm} must be contiguous with shape {shape}")
    dev = x.device
    if y is None:
        y = _empty(stream, (m_total, n), dtype=torch.float32 if y_dtype == BSQ_F32 else torch.bfloat16, device=dev)
    workspace = _workspace(BSQ_OP_GEMM_FWD, E, m_total, n, k, workspace, dev, stream)
    _check("bsq_grouped_gemm_w4a16",
           _lib.bsq_grouped_gemm_w4a16(_ptr(x), _ptr(w_codes), _ptr(w_bscale), _ptr(w_rscale), _ptr(offsets), E,
                                       m_total, n, k, _ptr(y), y_dtype, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


def bsq_grouped_gemm_bwd(offsets, m_total, n, k, dy_q=None, wt_q=None, dyt_q=None, xt_q=None,
                         flags=BSQ_DGRAD | BSQ_WGRAD, dx_dtype=BSQ_BF16, dw_dtype=BSQ_BF16, dx=None, dw=None,
                         workspace=None, stream=None):
    """Backward grouped GEMMs.  dy_q = ROWWISE (codes, scale) of dY [m_total, n];
    wt_q = COLWISE_T of W [E*n, k] with offsets {0, n, 2n, ..}; dyt_q / xt_q =
    COLWISE_T of dY / X with ``offsets``.  Returns (dx, dw)."""
    _dev(offsets, "offsets", (torch.int32,))
    E = offsets.numel() - 1
    dev = offsets.device
    if flags & BSQ_DGRAD and dx is None and m_total > 0:
        dx = _empty(stream, (m_total, k), dtype=torch.float32 if dx_dtype == BSQ_F32 else torch.bfloat16, device=dev)
    if flags & BSQ_WGRAD and dw is None:
        dw = _empty(stream, (E, n, k), dtype=torch.float32 if dw_dtype == BSQ_F32 else torch.bfloat16, device=dev)
    workspace = _workspace(BSQ_OP_GEMM_BWD, E, m_total, n, k, workspace, dev, stream)
    dy_q = dy_q or (None, None)
    wt_q = wt_q or (None, None)
    dyt_q = dyt_q or (None, None)
    xt_q = xt_q or (None, None)
    _check("bsq_grouped_gemm_bwd",
           _lib.bsq_grouped_gemm_bwd(_ptr(dy_q[0]), _ptr(dy_q[1]), _ptr(wt_q[0]), _ptr(wt_q[1]), _ptr(dyt_q[0]),
                                     _ptr(dyt_q[1]), _ptr(xt_q[0]), _ptr(xt_q[1]), _ptr(offsets), E, m_total, n, k,
                                     _ptr(dx), dx_dtype, _ptr(dw), dw_dtype, flags, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream)))
    return dx, dw


def _dtype_id(t, name):
    _dev(t, name, (torch.bfloat16, torch.float32))
    return BSQ_F32 if t.dtype == torch.float32 else BSQ_BF16


def _shaped(t, name, dtypes, shape, dev):
    """Checks a dense input or output buffer."""
    if type(t) is torch.Tensor and t.dtype in dtypes and t.shape == shape and t.device == dev and t.is_contiguous():
        return t
    _dev(t, name, dtypes)
    if t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)} on {dev}")
    return t


def _scratch(need, workspace, dev, stream):
    if workspace is None:
        return _empty(stream, (max(need, 1),), dtype=torch.uint8, device=dev)  # (0: sizes that the call refuses)
    _dev(workspace, "workspace", (workspace.dtype,))
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    return workspace


def _offsets(offsets, dev):
    _dev(offsets, "offsets", (torch.int32,))
    if offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous() or offsets.device != dev:
        raise ValueError(f"offsets must be contiguous [num_experts + 1] on {dev}")
    return offsets.numel() - 1


def bsq_moe_route_workspace_size(tokens, num_experts):
    return int(_lib.bsq_moe_route_workspace_size(tokens, num_experts))


def bsq_moe_dispatch_workspace_size(tokens, top_k, num_experts):
    return int(_lib.bsq_moe_dispatch_workspace_size(tokens, top_k, num_experts))


def bsq_moe_route(logits, top_k, bias=None, mask=None, normalize=True, scale=1.0, loss_coef=0.0, workspace=None,
                  stream=None):
    """Top-k routing of ``logits`` [tokens, experts] (bf16 or f32) with the balance loss.
    bias f32 [experts] is added for the selection only; mask (uint8 or bool) [tokens]
    is 0 for padding.  Returns (expert_ids i32 [tokens, top_k], weights f32
    [tokens, top_k], lse f32 [tokens], counts i32 [experts + 1], loss f32 [1]);
    counts holds the tokens per expert, then the tokens that go anywhere."""
    dt = _dtype_id(logits, "logits")
    T, E, ld = _rows_ld(logits)
    dev = logits.device
    if bias is not None:
        _shaped(bias, "bias", (torch.float32,), (E,), dev)
    if mask is not None:
        _shaped(mask, "mask", (torch.uint8, torch.bool), (T,), dev)
    need = bsq_moe_route_workspace_size(T, E)
    sizes = T * top_k, T * top_k, T, E + 1, 1
    if workspace is None and 0 < need <= _SMALL - 4 * sum(sizes):
        ids, weights, lse, counts, loss, ws = _carve(stream, torch.float32, dev, sizes, need)
        ids, weights, counts = ids.view(torch.int32).view(T, top_k), weights.view(T, top_k), counts.view(torch.int32)
    else:
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):  # (as _empty, once for all)
            ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
            weights, lse, loss = (torch.empty(n, device=dev, dtype=torch.float32) for n in ((T, top_k), T, 1))
            counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
            workspace = _scratch(need, workspace, dev, None)
        ws, need = _ptr(workspace), workspace.numel() * workspace.element_size()
    _check("bsq_moe_route",
           _lib.bsq_moe_route(_ptr(logits), dt, T, E, ld, top_k, _ptr(bias), _ptr(mask), int(normalize),
                              scale, loss_coef, _ptr(ids), _ptr(weights), _ptr(lse), _ptr(counts), _ptr(loss), ws, need,
                              _stream(stream)))
    return ids, weights, lse, counts, loss


def bsq_moe_route_bwd(logits, expert_ids, weights, lse, counts, dweights=None, dloss=None, normalize=True, scale=1.0,
                      loss_coef=0.0, dlogits=None, stream=None):
    """Gradient of ``logits`` from those of the weights (f32 [tokens, top_k]) and of
    the loss (f32 [1], on the device); either may be None.  The other arguments are
    those and the outputs of bsq_moe_route."""
    dt = _dtype_id(logits, "logits")
    T, E, ld = _rows_ld(logits)
    dev = logits.device
    K = expert_ids.shape[-1]
    _shaped(expert_ids, "expert_ids", (torch.int32,), (T, K), dev)
    _shaped(weights, "weights", (torch.float32,), (T, K), dev)
    _shaped(lse, "lse", (torch.float32,), (T,), dev)
    _shaped(counts, "counts", (torch.int32,), (E + 1,), dev)
    if dweights is not None:
        _shaped(dweights, "dweights", (torch.float32,), (T, K), dev)
    if dloss is not None:
        _dev(dloss, "dloss", (torch.float32,))
        if dloss.numel() != 1 or dloss.device != dev:
            raise ValueError(f"dloss must hold one value on {dev}")
    ldd = E
    if dlogits is None:
        dlogits = _empty(stream, (T, E), dtype=logits.dtype, device=dev)
    else:
        _dev(dlogits, "dlogits", (logits.dtype,))
        if dlogits.shape != (T, E) or dlogits.device != dev:
            raise ValueError(f"dlogits must have shape {(T, E)} on {dev}")
        ldd = _rows_ld(dlogits)[2]
    _check("bsq_moe_route_bwd",
           _lib.bsq_moe_route_bwd(_ptr(logits), dt, T, E, ld, K, _ptr(expert_ids), _ptr(weights), _ptr(lse),
                                  _ptr(counts), _ptr(dweights), _ptr(dloss), int(normalize), scale, loss_coef,
                                  _ptr(dlogits), ldd, _stream(stream)))
    return dlogits


def bsq_moe_dispatch(expert_ids, num_experts, workspace=None, stream=None):
    """Expert-sorted order of the choices ``expert_ids`` (i32 [tokens, top_k]; an id
    outside [0, num_experts) is no choice).  Returns (offsets i32 [num_experts + 1],
    row_index i32 [tokens * top_k], slot i32 [tokens, top_k])."""
    _dev(expert_ids, "expert_ids", (torch.int32,))
    if expert_ids.dim() != 2 or not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be contiguous [tokens, top_k]")
    T, K = expert_ids.shape
    dev = expert_ids.device
    need = bsq_moe_dispatch_workspace_size(T, K, num_experts)
    sizes = num_experts + 1, T * K, T * K
    # (the workspace of a larger call is a small part of the outputs)
    if workspace is None and 0 < need <= max(_SMALL - 4 * sum(sizes), sum(sizes) // 2):
        offsets, row_index, slot, ws = _carve(stream, torch.int32, dev, sizes, need)
    else:
        offsets, row_index, slot = _carve(stream, torch.int32, dev, sizes)
        workspace = _scratch(need, workspace, dev, stream)
        ws, need = _ptr(workspace), workspace.numel() * workspace.element_size()
    slot = slot.view(T, K)
    _check("bsq_moe_dispatch",
           _lib.bsq_moe_dispatch(_ptr(expert_ids), T, K, num_experts, _ptr(offsets), _ptr(row_index), _ptr(slot), ws,
                                 need, _stream(stream)))
    return offsets, row_index, slot


def bsq_moe_combine(ye, slot, weights=None, y=None, stream=None):
    """y[t] = sum_j weights[t, j] * ye[slot[t, j]] (bf16 or f32 rows; weights None:
    ones).  Choices whose slot is outside ye add nothing."""
    dt = _dtype_id(ye, "ye")
    M, W, ld = _rows_ld(ye)
    dev = ye.device
    T, K = slot.shape
    _shaped(slot, "slot", (torch.int32,), (T, K), dev)
    if weights is not None:
        _shaped(weights, "weights", (torch.float32,), (T, K), dev)
    ldy = W
    if y is None:
        y = _empty(stream, (T, W), dtype=ye.dtype, device=dev)
    else:
        _dev(y, "y", (ye.dtype,))
        if y.shape != (T, W) or y.device != dev:
            raise ValueError(f"y must have shape {(T, W)} on {dev}")
        ldy = _rows_ld(y)[2]
    _check("bsq_moe_combine",
           _lib.bsq_moe_combine(_ptr(ye), dt, M, W, ld, _ptr(slot), _ptr(weights), T, K, _ptr(y), ldy,
                                _stream(stream)))
    return y


def bsq_moe_combine_bwd(dy, ye, slot, weights=None, offsets=None, m_total=None, dye=None, need_dweights=True,
                        stream=None):
    """Gradients of bsq_moe_combine: (dye [m_total, width], dweights f32 [tokens, top_k]
    or None).  With ``offsets`` (of the dispatch) the rows of dye that no choice
    owns become zero, without they are left as they are.  ye may be None where
    dweights is not needed; m_total then gives the rows of dye."""
    dt = _dtype_id(dy, "dy")
    T, W, ld = _rows_ld(dy)
    dev = dy.device
    K = slot.shape[-1]
    _shaped(slot, "slot", (torch.int32,), (T, K), dev)
    if weights is not None:
        _shaped(weights, "weights", (torch.float32,), (T, K), dev)
    if ye is None and (need_dweights or m_total is None):
        raise ValueError("without ye, m_total is needed and dweights cannot be computed")
    M = ye.shape[0] if ye is not None else m_total
    ldye = 0
    if ye is not None:
        _dev(ye, "ye", (dy.dtype,))
        if ye.dim() != 2 or ye.shape[1] != W or ye.device != dev:
            raise ValueError(f"ye must have {W} columns on {dev}")
        ldye = _rows_ld(ye)[2]
    E = 0 if offsets is None else _offsets(offsets, dev)
    ldd = W
    if dye is None:
        dye = _empty(stream, (M, W), dtype=dy.dtype, device=dev)
    else:
        _dev(dye, "dye", (dy.dtype,))
        if dye.shape != (M, W) or dye.device != dev:
            raise ValueError(f"dye must have shape {(M, W)} on {dev}")
        ldd = _rows_ld(dye)[2]
    dw = _empty(stream, (T, K), dtype=torch.float32, device=dev) if need_dweights else None
    _check("bsq_moe_combine_bwd",
           _lib.bsq_moe_combine_bwd(_ptr(dy), dt, T, W, ld, _ptr(ye), M, ldye, _ptr(slot), _ptr(weights), K,
                                    _ptr(offsets), E, _ptr(dye), ldd, _ptr(dw), _stream(stream)))
    return dye, dw


def bsq_quantize_fp8b128(x, row_index=None, offsets=None, rows_form=True, row=None, t=None, stream=None):
    """FP8B128 of bf16 ``x`` [src_rows, cols], or of x[row_index] (i32; out-of-range
    indices give zero rows); a block with an infinity or a NaN gets a NaN scale.  Returns (row, t): row = (codes u8 [rows, cols], scale
    f32 [ceil(cols/128), rows]), or None with rows_form=False; t = the
    token-column form (t_codes u8 [cols, P], t_scale f32 [P/128, cols]) where
    ``offsets`` (i32 [groups + 1]) is given, else None."""
    _dev(x, "x", _BF16)
    src_rows, cols, ld = _rows_ld(x)
    dev = x.device
    rows = src_rows
    if row_index is not None:
        rows = row_index.numel()
        _shaped(row_index, "row_index", (torch.int32,), (rows,), dev)
    nb = (cols + 127) // 128
    G = 0
    if not rows_form:
        row = None
    elif row is None:
        row = (_empty(stream, (rows, cols), dtype=torch.uint8, device=dev),
               _empty(stream, (nb, rows), dtype=torch.float32, device=dev))
    else:
        row = (_shaped(row[0], "codes", (torch.uint8,), (rows, cols), dev),
               _shaped(row[1], "scale", (torch.float32,), (nb, rows), dev))
    if offsets is not None:
        G = _offsets(offsets, dev)
        Pc = bsq_colwise_padded_cols(G, rows)
        if t is None:
            t = (_empty(stream, (cols, Pc), dtype=torch.uint8, device=dev),
                 _empty(stream, (Pc // 128, cols), dtype=torch.float32, device=dev))
        else:
            t = (_shaped(t[0], "t codes", (torch.uint8,), (cols, Pc), dev),
                 _shaped(t[1], "t scale", (torch.float32,), (Pc // 128, cols), dev))
    else:
        t = None
    rq, tq = row or (None, None), t or (None, None)
    _check("bsq_quantize_fp8b128",
           _lib.bsq_quantize_fp8b128(_ptr(x), src_rows, cols, ld, _ptr(row_index), rows, _ptr(offsets), G,
                                     _ptr(rq[0]), _ptr(rq[1]), _ptr(tq[0]), _ptr(tq[1]), _stream(stream)))
    return row, t


def bsq_quantize_fp8b128_weights(w, num_experts, transposed=True, codes=None, codes_t=None, scale=None, stream=None):
    """FP8B128 of expert weights ``w`` bf16 [num_experts * n, k] in 128 x 128 blocks:
    (codes u8 [E*n, k], codes_t u8 [E*k, n] or None, scale f32 [E, ceil(n/128), ceil(k/128)])."""
    _dev(w, "w", _BF16)
    rows, k, ld = _rows_ld(w)
    if num_experts < 1 or rows % num_experts:
        raise ValueError("w must hold num_experts * n rows")
    n, dev = rows // num_experts, w.device
    sshape = (num_experts, (n + 127) // 128, (k + 127) // 128)
    u8, f32 = (torch.uint8,), (torch.float32,)
    codes = _empty(stream, (rows, k), dtype=u8[0], device=dev) if codes is None else _shaped(codes, "codes", u8, (rows, k), dev)
    scale = _empty(stream, sshape, dtype=f32[0], device=dev) if scale is None else _shaped(scale, "scale", f32, sshape, dev)
    if codes_t is not None:
        _shaped(codes_t, "codes_t", u8, (num_experts * k, n), dev)
    elif transposed:
        codes_t = _empty(stream, (num_experts * k, n), dtype=u8[0], device=dev)
    _check("bsq_quantize_fp8b128_weights",
           _lib.bsq_quantize_fp8b128_weights(_ptr(w), num_experts, n, k, ld, _ptr(codes), _ptr(codes_t),
                                             _ptr(scale), _stream(stream)))
    return codes, codes_t, scale


def bsq_grouped_gemm_fp8b128_workspace_size(num_experts):
    return int(_lib.bsq_grouped_gemm_fp8b128_workspace_size(num_experts))


_OUT_DTYPE = {BSQ_BF16: torch.bfloat16, BSQ_F32: torch.float32}


def _out(t, name, dtype, shape, dev, stream):
    if t is None:
        return _empty(stream, shape, dtype=_OUT_DTYPE[dtype], device=dev)
    return _shaped(t, name, (_OUT_DTYPE[dtype],), shape, dev)


def bsq_grouped_gemm_fp8b128_fwd(a_q, w_q, offsets, y_dtype=BSQ_BF16, y=None, workspace=None, stream=None):
    """Forward grouped GEMM on FP8B128 operands: a_q = (codes [m_total, k], scale)
    of the expert-sorted activations in row form, w_q = (codes [E*n, k], scale [E,
    ceil(n/128), ceil(k/128)]) of the weights.  Returns y [m_total, n]; a row's bits do
    not depend on the other rows."""
    a_codes, a_scale = a_q
    w_codes, w_scale = w_q
    _dev(a_codes, "a codes", (torch.uint8,))
    dev = a_codes.device
    E = _offsets(offsets, dev)
    M, k = a_codes.shape
    n = w_codes.shape[0] // E
    kb = (k + 127) // 128
    _shaped(a_codes, "a codes", (torch.uint8,), (M, k), dev)
    _shaped(a_scale, "a scale", (torch.float32,), (kb, M), dev)
    _shaped(w_codes, "w codes", (torch.uint8,), (E * n, k), dev)
    _shaped(w_scale, "w scale", (torch.float32,), (E, (n + 127) // 128, kb), dev)
    y = _out(y, "y", y_dtype, (M, n), dev, stream)
    workspace = _scratch(bsq_grouped_gemm_fp8b128_workspace_size(E), workspace, dev, stream)
    _check("bsq_grouped_gemm_fp8b128_fwd",
           _lib.bsq_grouped_gemm_fp8b128_fwd(_ptr(a_codes), _ptr(a_scale), _ptr(w_codes), _ptr(w_scale),
                                             _ptr(offsets), E, M, n, k, _ptr(y), y_dtype, _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


def bsq_grouped_gemm_fp8b128_bwd(offsets, m_total, n, k, dy_q=None, wt_q=None, dyt_q=None, xt_q=None,
                                 flags=BSQ_DGRAD | BSQ_WGRAD, dx_dtype=BSQ_BF16, dw_dtype=BSQ_BF16, dx=None, dw=None,
                                 workspace=None, stream=None):
    """Backward grouped GEMMs on FP8B128 operands.  dy_q = row form of dY [m_total, n];
    wt_q = (codes_t [E*k, n], scale) of the weights; dyt_q / xt_q = token-column
    forms of dY / X with ``offsets``.  Returns (dx, dw)."""
    _dev(offsets, "offsets", (torch.int32,))
    dev = offsets.device
    E = _offsets(offsets, dev)
    nb, kb = (n + 127) // 128, (k + 127) // 128
    u8, f32 = (torch.uint8,), (torch.float32,)
    none = (None, None)
    if flags & BSQ_DGRAD:
        if dy_q is None or wt_q is None:
            raise ValueError("BSQ_DGRAD needs dy_q and wt_q")
        _shaped(dy_q[0], "dy codes", u8, (m_total, n), dev)
        _shaped(dy_q[1], "dy scale", f32, (nb, m_total), dev)
        _shaped(wt_q[0], "wt codes", u8, (E * k, n), dev)
        _shaped(wt_q[1], "w scale", f32, (E, nb, kb), dev)
        dx = _out(dx, "dx", dx_dtype, (m_total, k), dev, stream)
    else:
        dy_q = wt_q = none
    if flags & BSQ_WGRAD:
        if dyt_q is None or xt_q is None:
            raise ValueError("BSQ_WGRAD needs dyt_q and xt_q")
        Pc = bsq_colwise_padded_cols(E, m_total)
        for q, nm, w in ((dyt_q, "dyt", n), (xt_q, "xt", k)):
            _shaped(q[0], nm + " codes", u8, (w, Pc), dev)
            _shaped(q[1], nm + " scale", f32, (Pc // 128, w), dev)
        dw = _out(dw, "dw", dw_dtype, (E, n, k), dev, stream)
    else:
        dyt_q = xt_q = none
    workspace = _scratch(bsq_grouped_gemm_fp8b128_workspace_size(E), workspace, dev, stream)
    _check("bsq_grouped_gemm_fp8b128_bwd",
           _lib.bsq_grouped_gemm_fp8b128_bwd(_ptr(dy_q[0]), _ptr(dy_q[1]), _ptr(wt_q[0]), _ptr(wt_q[1]),
                                             _ptr(dyt_q[0]), _ptr(dyt_q[1]), _ptr(xt_q[0]), _ptr(xt_q[1]),
                                             _ptr(offsets), E, m_total, n, k, _ptr(dx), dx_dtype, _ptr(dw), dw_dtype,
                                             flags, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                             _stream(stream)))
    return dx, dw


def bsq_debug_status(workspace, stream=None):
    v = I32(0)
    _check("bsq_debug_status", _lib.bsq_debug_status(_ptr(workspace), _stream(stream), ctypes.byref(v)))
    return int(v.value)


def bsq_debug_encode_e2m1(x, out=None, stream=None):
    _dev(x, "x", (torch.float32,))
    out = _empty(stream, x.shape, dtype=torch.uint8, device=x.device) if out is None else out
    _check("bsq_debug_encode_e2m1", _lib.bsq_debug_encode_e2m1(_ptr(x), _ptr(out), x.numel(), _stream(stream)))
    return out


def bsq_debug_encode_e4m3(x, out=None, stream=None):
    _dev(x, "x", (torch.float32,))
    out = _empty(stream, x.shape, dtype=torch.uint8, device=x.device) if out is None else out
    _check("bsq_debug_encode_e4m3", _lib.bsq_debug_encode_e4m3(_ptr(x), _ptr(out), x.numel(), _stream(stream)))
    return out
