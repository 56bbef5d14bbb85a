"""Python binding of libmfx, fused transformer MLP and residual epilogues for
GB300 (sm_103a).

Every function here marshals torch tensors into the C ABI declared in
``include/mfx.h`` (device pointers, sizes, the current CUDA stream) and calls
the library; all computation happens in its CUDA kernels.  The names are the
ABI's names and the positional arguments follow the ABI's order.  Tensors must
be contiguous CUDA tensors; the last dimension is the width (hidden, or 2F for
the GLU inputs) and all leading dimensions are flattened into rows, so the
Megatron [seq, batch, hidden] layout is accepted as is.

There is no fallback: if ``libmfx.so`` has not been built, every call raises.
"""
import ctypes as C
import math
import os

import torch

__all__ = [
    "MfxError", "lib", "dtype_code",
    "mfx_bias_gelu_fwd", "mfx_bias_gelu_bwd",
    "mfx_bias_geglu_fwd", "mfx_bias_geglu_bwd",
    "mfx_bias_swiglu_fwd", "mfx_bias_swiglu_bwd",
    "mfx_weighted_squared_relu_fwd", "mfx_weighted_squared_relu_bwd",
    "mfx_scaled_masked_softmax_fwd", "mfx_scaled_upper_triang_masked_softmax_fwd",
    "mfx_scaled_masked_softmax_bwd", "mfx_scaled_upper_triang_masked_softmax_bwd",
    "mfx_relbias_softmax_dropout_fwd", "mfx_relbias_softmax_dropout_bwd",
    "mfx_moe_rows", "mfx_moe_sort", "mfx_moe_permute_fwd", "mfx_moe_permute_bwd",
    "mfx_moe_unpermute_fwd", "mfx_moe_unpermute_bwd",
    "mfx_add_rmsnorm_fwd", "mfx_add_rmsnorm_quant_fwd", "mfx_add_rmsnorm_bwd",
    "mfx_token_logprobs_fwd", "mfx_token_logprobs_bwd",
    "mfx_topk_distill_fwd", "mfx_topk_distill_bwd", "mfx_topk_distill_fwd_bwd",
    "mfx_bias_dropout_add_train", "mfx_bias_dropout_add_inference", "mfx_bias_dropout_add_bwd",
    "mfx_bias_dropout_add_train_packed", "mfx_bias_dropout_add_bwd_packed",
    "mfx_bias_dropout_add_train_nomask", "mfx_dropout_fwd", "mfx_dropout_bwd",
    "mfx_bias_gelu_bwd_dbias", "mfx_bias_geglu_bwd_dbias", "mfx_bias_swiglu_bwd_dbias",
    "mfx_bias_dropout_add_bwd_dbias", "mfx_device_error",
]

# MFX_LIBRARY selects another build of the same library (for example one
# compiled with different tuning knobs); by default the in-tree build is used.
LIB_PATH = os.environ.get("MFX_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmfx.so")

MFX_F32, MFX_BF16, MFX_E4M3, MFX_E5M2, MFX_E8M0 = 0, 1, 2, 3, 4
STATUS = {0: "MFX_OK", 1: "MFX_ERR_NULL", 2: "MFX_ERR_SHAPE", 3: "MFX_ERR_DTYPE",
          4: "MFX_ERR_PROB", 5: "MFX_ERR_ALIAS", 6: "MFX_ERR_CUDA", 7: "MFX_ERR_DEVICE",
          8: "MFX_ERR_WORKSPACE", 9: "MFX_ERR_VALUE"}


class MfxError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().mfx_status_string(status).decode()
        extra = f" (cudaError {lib().mfx_last_cuda_error()})" if status == 6 else ""
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}{extra}")


_lib = None

_P, _I, _I64, _U64, _F = C.c_void_p, C.c_int, C.c_int64, C.c_uint64, C.c_float
_RELBIAS = [_I, _P, _I64, _I64, _I, _P, _I64, _I64, _I64, _I, _I64, _P, _F, _U64, _U64, _U64]
_SIGS = {
    "mfx_bias_gelu_fwd": [_I, _I64, _I64, _P, _P, _P, _P],
    "mfx_bias_gelu_bwd": [_I, _I64, _I64, _P, _P, _P, _P, _P],
    "mfx_bias_geglu_fwd": [_I, _I64, _I64, _P, _P, _P, _P],
    "mfx_bias_geglu_bwd": [_I, _I64, _I64, _P, _P, _P, _P, _P],
    "mfx_bias_swiglu_fwd": [_I, _I64, _I64, _P, _P, _P, _P, _P],
    "mfx_bias_swiglu_bwd": [_I, _I64, _I64, _P, _P, _P, _P, _P, _P, _P],
    "mfx_weighted_squared_relu_fwd": [_I, _I64, _I64, _P, _P, _P, _P],
    "mfx_weighted_squared_relu_bwd": [_I, _I64, _I64, _P, _P, _P, _P, _P, _P],
    "mfx_scaled_masked_softmax_fwd": [_I, _I64, _I64, _I64, _I64, _P, _P, _I64, _I64, _I64, _F, _P, _P],
    "mfx_scaled_upper_triang_masked_softmax_fwd": [_I, _I64, _I64, _P, _F, _P, _P],
    "mfx_scaled_masked_softmax_bwd": [_I, _I64, _I64, _P, _P, _F, _P, _P],
    "mfx_scaled_upper_triang_masked_softmax_bwd": [_I, _I64, _I64, _P, _P, _F, _P, _P],
    "mfx_relbias_softmax_dropout_fwd": [_I, _I64, _I64, _I64, _I64, _P, _F, *_RELBIAS, _P, _P, _P],
    "mfx_relbias_softmax_dropout_bwd": [_I, _I64, _I64, _I64, _I64, _P, _P, _P, _F, *_RELBIAS, _P, _P, _P,
                                        C.POINTER(C.c_size_t), _P],
    "mfx_moe_sort": [_I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, C.POINTER(C.c_size_t), _P],
    "mfx_moe_permute_fwd": [_I, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P],
    "mfx_moe_permute_bwd": [_I, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P],
    "mfx_moe_unpermute_fwd": [_I, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P],
    "mfx_moe_unpermute_bwd": [_I, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P],
    "mfx_add_rmsnorm_fwd": [_I, _I, _I, _I64, _I64, _P, _P, _P, _F, _F, _P, _P, _P, _P],
    "mfx_add_rmsnorm_quant_fwd": [_I, _I, _I, _I64, _I64, _P, _P, _P, _F, _F, _I, _I64, _I, _P, _P, _P, _P, _P],
    "mfx_add_rmsnorm_bwd": [_I, _I, _I, _I64, _I64, _P, _P, _P, _P, _F, _P, _P, _P, _P, _P, C.POINTER(C.c_size_t), _P],
    "mfx_token_logprobs_fwd": [_I, _I64, _I64, _I64, _P, _I, _P, _F, _I64, _P, _P, _P, _P, _P, _P, C.POINTER(C.c_size_t),
                               _P],
    "mfx_token_logprobs_bwd": [_I, _I64, _I64, _I64, _P, _P, _P, _I, _P, _P, _F, _P, _I64, _P],
    "mfx_topk_distill_fwd": [_I, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _P, _F, _P, _P, _P],
    "mfx_topk_distill_bwd": [_I, _I, _I64, _I64, _I64, _I64, _P, _P, _I, _P, _P, _P, _F, _P, _I64, _P],
    "mfx_topk_distill_fwd_bwd": [_I, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _P, _P, _F, _P, _P, _I64, _P],
    "mfx_bias_dropout_add_train": [_I, _I, _I64, _I64, _P, _P, _P, _F, _U64, _U64, _U64, _P, _P, _P],
    "mfx_bias_dropout_add_inference": [_I, _I, _I64, _I64, _P, _P, _P, _F, _U64, _U64, _P],
    "mfx_bias_dropout_add_bwd": [_I, _I, _I64, _I64, _P, _P, _F, _U64, _U64, _U64, _P, _P, _P],
    "mfx_bias_dropout_add_train_packed": [_I, _I, _I64, _I64, _P, _P, _P, _F, _U64, _U64, _U64, _P, _P, _P],
    "mfx_bias_dropout_add_bwd_packed": [_I, _I, _I64, _I64, _P, _P, _F, _P, _P, _P],
    "mfx_bias_dropout_add_train_nomask": [_I, _I, _I64, _I64, _P, _P, _P, _F, _U64, _U64, _U64, _P, _P],
    "mfx_dropout_fwd": [_I, _I64, _P, _F, _U64, _U64, _U64, _P, _P],
    "mfx_dropout_bwd": [_I, _I64, _P, _F, _U64, _U64, _U64, _P, _P],
    "mfx_bias_gelu_bwd_dbias": [_I, _I64, _I64, _P, _P, _P, _P, _P, _P, C.POINTER(C.c_size_t), _P],
    "mfx_bias_gelu_bwd_dbias_noalloc": [_I, _I64, _I64, _P, _P, _P, _P, _P, _P],
    "mfx_bias_geglu_bwd_dbias": [_I, _I64, _I64, _P, _P, _P, _P, _P, _P, C.POINTER(C.c_size_t), _P],
    "mfx_bias_swiglu_bwd_dbias": [_I, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, C.POINTER(C.c_size_t), _P],
    "mfx_bias_dropout_add_bwd_dbias": [_I, _I, _I64, _I64, _P, _P, _F, _U64, _U64, _U64, _P, _P, _P, _P,
                                       C.POINTER(C.c_size_t), _P],
}


def lib():
    """The loaded libmfx.so (ctypes), with argument types set."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libmfx.so is not built ({LIB_PATH} missing): run "
                "`python -c 'import __graft_entry__ as g; g.build()'` first")
        L = C.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = C.c_int
        L.mfx_status_string.argtypes = [C.c_int]
        L.mfx_status_string.restype = C.c_char_p
        L.mfx_last_cuda_error.argtypes = []
        L.mfx_last_cuda_error.restype = C.c_int
        L.mfx_moe_rows.argtypes = [_I64, _I64, _I64, _I64]
        L.mfx_moe_rows.restype = _I64
        L.mfx_version.argtypes = []
        L.mfx_version.restype = C.c_int
        L.mfx_device_error.argtypes = [C.POINTER(C.c_uint)]
        L.mfx_device_error.restype = C.c_int
        _lib = L
    return _lib


def dtype_code(dtype):
    if dtype == torch.bfloat16:
        return MFX_BF16
    if dtype == torch.float32:
        return MFX_F32
    raise TypeError(f"libmfx supports bfloat16 and float32 tensors, got {dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cuda(t, name, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _like(t, name, shape, dtype):
    """A CUDA tensor of the given shape and dtype (an output or gradient buffer)."""
    _cuda(t, name, dtype)
    if t is None or t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return t


def _same_device(t, dev, name):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}, the data's")


# the current stream's raw handle without building a Stream object per call
# (torch's own raw-stream query where this torch has it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, t):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(t.get_device())
        return torch.cuda.current_stream(t.device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream, device):
    """Context in which allocations belong to `stream` (as _stream() takes it)."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    """Memory of a call's own.  It belongs to the stream that the call runs
    on, so that it is given to nobody else while the call may use it, and to
    the call while nobody else may."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(t, stream):
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _rows_cols(t):
    cols = t.shape[-1] if t.dim() else 1
    rows = t.numel() // cols if cols else 0
    return rows, cols


def mfx_device_error():
    """Code of any bounded wait that ran out since the last call (0 = none);
    synchronises the current device and clears the word."""
    code = C.c_uint(0)
    lib().mfx_device_error(C.byref(code))
    return code.value


def _call(name, *args):
    st = getattr(_lib or lib(), name)(*args)
    if st != 0:
        raise MfxError(st, name)


# ---------------------------------------------------------------------------
# bias-GeLU
# ---------------------------------------------------------------------------
def mfx_bias_gelu_fwd(bias, y, out=None, stream=None):
    """out = gelu_tanh(y + bias); returns out (allocated if not given)."""
    _cuda(y, "y")
    _cuda(bias, "bias", y.dtype)
    out = torch.empty_like(y) if out is None else _cuda(out, "out", y.dtype)
    rows, cols = _rows_cols(y)
    _call("mfx_bias_gelu_fwd", dtype_code(y.dtype), rows, cols, _ptr(bias), _ptr(y), _ptr(out),
          _stream(stream, y))
    return out


def mfx_bias_gelu_bwd(g, bias, y, dy=None, stream=None):
    """dy = g * gelu_tanh'(y + bias); returns dy."""
    _cuda(y, "y")
    _cuda(g, "g", y.dtype)
    _cuda(bias, "bias", y.dtype)
    if g.shape != y.shape:
        raise ValueError("g and y must have the same shape")
    dy = torch.empty_like(y) if dy is None else _cuda(dy, "dy", y.dtype)
    rows, cols = _rows_cols(y)
    _call("mfx_bias_gelu_bwd", dtype_code(y.dtype), rows, cols, _ptr(g), _ptr(bias), _ptr(y),
          _ptr(dy), _stream(stream, y))
    return dy


# ---------------------------------------------------------------------------
# GLU
# ---------------------------------------------------------------------------
def _glu_shape(x):
    rows, two_f = _rows_cols(x)
    if two_f % 2:
        raise ValueError("the GLU input width must be even (2F)")
    return rows, two_f // 2


def _half_shape(x):
    return (*x.shape[:-1], x.shape[-1] // 2)


def mfx_bias_geglu_fwd(x, bias, out=None, stream=None):
    _cuda(x, "x")
    _cuda(bias, "bias", x.dtype)
    rows, F = _glu_shape(x)
    out = x.new_empty(_half_shape(x)) if out is None else _cuda(out, "out", x.dtype)
    _call("mfx_bias_geglu_fwd", dtype_code(x.dtype), rows, F, _ptr(x), _ptr(bias), _ptr(out),
          _stream(stream, x))
    return out


def mfx_bias_geglu_bwd(g, x, bias, dx=None, stream=None):
    _cuda(x, "x")
    _cuda(g, "g", x.dtype)
    _cuda(bias, "bias", x.dtype)
    rows, F = _glu_shape(x)
    dx = torch.empty_like(x) if dx is None else _cuda(dx, "dx", x.dtype)
    _call("mfx_bias_geglu_bwd", dtype_code(x.dtype), rows, F, _ptr(g), _ptr(x), _ptr(bias),
          _ptr(dx), _stream(stream, x))
    return dx


def mfx_bias_swiglu_fwd(x, bias, weight=None, out=None, stream=None):
    _cuda(x, "x")
    _cuda(bias, "bias", x.dtype)
    _cuda(weight, "weight", torch.float32)
    rows, F = _glu_shape(x)
    out = x.new_empty(_half_shape(x)) if out is None else _cuda(out, "out", x.dtype)
    _call("mfx_bias_swiglu_fwd", dtype_code(x.dtype), rows, F, _ptr(x), _ptr(bias), _ptr(weight),
          _ptr(out), _stream(stream, x))
    return out


def mfx_bias_swiglu_bwd(g, x, bias, weight=None, dx=None, dweight=None, stream=None):
    """Returns (dx, dweight); dweight is None without a weight."""
    _cuda(x, "x")
    _cuda(g, "g", x.dtype)
    _cuda(bias, "bias", x.dtype)
    _cuda(weight, "weight", torch.float32)
    rows, F = _glu_shape(x)
    dx = torch.empty_like(x) if dx is None else _cuda(dx, "dx", x.dtype)
    if weight is not None and dweight is None:
        dweight = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
    _cuda(dweight, "dweight", torch.float32)
    _call("mfx_bias_swiglu_bwd", dtype_code(x.dtype), rows, F, _ptr(g), _ptr(x), _ptr(bias),
          _ptr(weight), _ptr(dx), _ptr(dweight), _stream(stream, x))
    return dx, dweight


# ---------------------------------------------------------------------------
# weighted squared ReLU
# ---------------------------------------------------------------------------
def _row_weight(weight, rows):
    _cuda(weight, "weight", torch.float32)
    if weight is None or weight.numel() != rows:
        raise ValueError(f"weight must be a float32 CUDA tensor of {rows} elements (one per row)")
    return weight


def mfx_weighted_squared_relu_fwd(x, weight, out=None, stream=None):
    _cuda(x, "x")
    rows, cols = _rows_cols(x)
    _row_weight(weight, rows)
    out = torch.empty_like(x) if out is None else _cuda(out, "out", x.dtype)
    _call("mfx_weighted_squared_relu_fwd", dtype_code(x.dtype), rows, cols, _ptr(x), _ptr(weight),
          _ptr(out), _stream(stream, x))
    return out


def mfx_weighted_squared_relu_bwd(g, x, weight, dx=None, dweight=None, stream=None):
    """Returns (dx, dweight)."""
    _cuda(x, "x")
    _cuda(g, "g", x.dtype)
    rows, cols = _rows_cols(x)
    _row_weight(weight, rows)
    dx = torch.empty_like(x) if dx is None else _cuda(dx, "dx", x.dtype)
    if dweight is None:
        dweight = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
    _cuda(dweight, "dweight", torch.float32)
    _call("mfx_weighted_squared_relu_bwd", dtype_code(x.dtype), rows, cols, _ptr(g), _ptr(x), _ptr(weight),
          _ptr(dx), _ptr(dweight), _stream(stream, x))
    return dx, dweight


# ---------------------------------------------------------------------------
# scale-mask-softmax
# ---------------------------------------------------------------------------
def mfx_scaled_masked_softmax_fwd(x, scale, mask=None, y=None, stream=None):
    """Softmax over the last dim of x * scale (+ mask).  x: [b, np, sq, sk]
    (or any shape whose leading dims flatten into rows when mask is None);
    mask: additive, 4 dims [1|b, 1|np, 1|sq, sk], x's dtype."""
    _cuda(x, "x")
    _cuda(mask, "mask", x.dtype)
    if mask is not None:
        if x.dim() != 4 or mask.dim() != 4:
            raise ValueError("with a mask, x and mask must have 4 dims [b, np, sq, sk]")
        b, np_, sq, sk = x.shape
        mb, mnp, msq, msk = mask.shape
    else:
        sk = x.shape[-1] if x.dim() else 1
        b, np_, sq = 1, 1, (x.numel() // sk if sk else 0)
        mb = mnp = msq = 1
        msk = sk
    if msk != sk:
        raise ValueError("mask's last dim must equal x's")
    y = torch.empty_like(x) if y is None else _cuda(y, "y", x.dtype)
    _call("mfx_scaled_masked_softmax_fwd", dtype_code(x.dtype), b, np_, sq, sk, _ptr(x), _ptr(mask),
          mb, mnp, msq, float(scale), _ptr(y), _stream(stream, x))
    return y


def _causal_dims(t):
    if t.dim() != 3 or t.shape[1] != t.shape[2]:
        raise ValueError("the causal softmax takes [attn_batches, sq, sq]")
    return t.shape[0], t.shape[1]


def mfx_scaled_upper_triang_masked_softmax_fwd(x, scale, y=None, stream=None):
    _cuda(x, "x")
    ab, sq = _causal_dims(x)
    y = torch.empty_like(x) if y is None else _cuda(y, "y", x.dtype)
    _call("mfx_scaled_upper_triang_masked_softmax_fwd", dtype_code(x.dtype), ab, sq, _ptr(x), float(scale),
          _ptr(y), _stream(stream, x))
    return y


def mfx_scaled_masked_softmax_bwd(dy, y, scale, dx=None, stream=None):
    _cuda(y, "y")
    _cuda(dy, "dy", y.dtype)
    if dy.shape != y.shape:
        raise ValueError("dy and y must have the same shape")
    rows, sk = _rows_cols(y)
    dx = torch.empty_like(y) if dx is None else _cuda(dx, "dx", y.dtype)
    _call("mfx_scaled_masked_softmax_bwd", dtype_code(y.dtype), rows, sk, _ptr(dy), _ptr(y), float(scale),
          _ptr(dx), _stream(stream, y))
    return dx


def mfx_scaled_upper_triang_masked_softmax_bwd(dy, y, scale, dx=None, stream=None):
    _cuda(y, "y")
    _cuda(dy, "dy", y.dtype)
    if dy.shape != y.shape:
        raise ValueError("dy and y must have the same shape")
    ab, sq = _causal_dims(y)
    dx = torch.empty_like(y) if dx is None else _cuda(dx, "dx", y.dtype)
    _call("mfx_scaled_upper_triang_masked_softmax_bwd", dtype_code(y.dtype), ab, sq, _ptr(dy), _ptr(y),
          float(scale), _ptr(dx), _stream(stream, y))
    return dx


# ---------------------------------------------------------------------------
# scale-mask-softmax with a learned relative position bias and dropout
# ---------------------------------------------------------------------------
def _relbias_args(x, table, mask, max_distance, bidirectional, causal, q_start, seq_start, p, seed, offset, elem_base):
    """x's shape and the arguments that forward and backward share, from
    table_dt on."""
    _cuda(x, "x")
    if x.dim() != 4:
        raise ValueError("x must have 4 dims [b, np, sq, sk]")
    shape = b, np_, _, sk = tuple(x.shape)
    dev, tdt, tptr, buckets = x.get_device(), MFX_F32, None, 0
    if table is not None:
        _cuda(table, "table")
        if table.dim() != 2 or table.shape[1] != np_:
            raise ValueError("table must have the shape [num_buckets, np]")
        _same_device(table, dev, "table")
        tdt, tptr, buckets = dtype_code(table.dtype), table.data_ptr(), table.shape[0]
    mptr, mb, mnp, msq = None, 1, 1, 1
    if mask is not None:
        _cuda(mask, "mask", x.dtype)
        if mask.dim() != 4 or mask.shape[3] != sk:
            raise ValueError("mask must have the shape [1 or b, 1 or np, 1 or sq, sk]")
        _same_device(mask, dev, "mask")
        mptr, (mb, mnp, msq, _) = mask.data_ptr(), mask.shape
    sptr = None
    if seq_start is not None:
        _like(seq_start, "seq_start", (b,), torch.int32)
        _same_device(seq_start, dev, "seq_start")
        sptr = seq_start.data_ptr()
    return shape, (tdt, tptr, buckets, int(max_distance), 1 if bidirectional else 0, mptr, mb, mnp, msq,
                   1 if causal else 0, int(q_start), sptr, float(p), int(seed) % 2**64, int(offset) % 2**64,
                   int(elem_base))


def mfx_relbias_softmax_dropout_fwd(x, scale, table=None, mask=None, max_distance=128, bidirectional=True,
                                    causal=False, q_start=0, seq_start=None, p=0.0, seed=0, offset=0, elem_base=0,
                                    y=None, stats=None, need_stats=True, stream=None):
    """y = dropout(softmax(x * scale + table[bucket(k - pos)] + mask), p) over
    the last dim of x [b, np, sq, sk]; table: [num_buckets, np] (x's dtype or
    float32); pos = q_start + seq_start[b] + q.  Returns (y, stats); stats
    [b, np, sq, 3] is what the backward needs (None with need_stats=False)."""
    shape, shared = _relbias_args(x, table, mask, max_distance, bidirectional, causal, q_start, seq_start, p, seed,
                                  offset, elem_base)
    y = _empty_like(x, stream) if y is None else _like(y, "y", shape, x.dtype)
    if stats is not None:
        _like(stats, "stats", (*shape[:3], 3), torch.float32)
    elif need_stats:
        stats = _empty((*shape[:3], 3), torch.float32, x.device, stream)
    _call("mfx_relbias_softmax_dropout_fwd", dtype_code(x.dtype), *shape, x.data_ptr(), float(scale), *shared,
          y.data_ptr(), _ptr(stats), _stream(stream, x))
    return y, stats


def mfx_relbias_softmax_dropout_bwd(dy, x, stats, scale, table=None, mask=None, max_distance=128, bidirectional=True,
                                    causal=False, q_start=0, seq_start=None, p=0.0, seed=0, offset=0, elem_base=0,
                                    dx=None, dtable=None, need_dtable=True, workspace=None, stream=None):
    """(dx, dtable) from the forward's inputs and stats; dtable has table's
    shape and dtype (None without a table or with need_dtable=False)."""
    shape, shared = _relbias_args(x, table, mask, max_distance, bidirectional, causal, q_start, seq_start, p, seed,
                                  offset, elem_base)
    _like(dy, "dy", shape, x.dtype)
    _like(stats, "stats", (*shape[:3], 3), torch.float32)
    dx = _empty_like(x, stream) if dx is None else _like(dx, "dx", shape, x.dtype)
    if dtable is not None:
        if table is None:
            raise ValueError("dtable needs a table")
        _like(dtable, "dtable", table.shape, table.dtype)
    elif table is not None and need_dtable:
        dtable = _empty_like(table, stream)
    head = (dtype_code(x.dtype), *shape, dy.data_ptr(), x.data_ptr(), stats.data_ptr(), float(scale), *shared,
            dx.data_ptr(), _ptr(dtable))
    st = _stream(stream, x)
    if dtable is None:
        _call("mfx_relbias_softmax_dropout_bwd", *head, None, None, st)
    else:
        _with_workspace("mfx_relbias_softmax_dropout_bwd", head, (st,), x.device, workspace,
                        (x.get_device(), *shape, table.shape[0]), stream=stream)
    return dx, dtable


# ---------------------------------------------------------------------------
# tokens sorted by expert and back
# ---------------------------------------------------------------------------
def mfx_moe_rows(tokens, topk, experts, align=1):
    """Rows that the sorted layout of tokens x topk slots needs at most."""
    n = lib().mfx_moe_rows(int(tokens), int(topk), int(experts), int(align))
    if n < 0:
        raise MfxError(2, "mfx_moe_rows")
    return n


def mfx_moe_sort(expert_of, experts, align=1, capacity=0, rows=None, row_of=None, slot_of=None, offsets=None,
                 counts=None, workspace=None, stream=None):
    """(row_of [tokens, topk], slot_of [rows], offsets [experts + 1], counts
    [experts]), all int32, of the layout of expert_of's slots (int32 [tokens,
    topk]) by expert; rows defaults to mfx_moe_rows()."""
    _cuda(expert_of, "expert_of", torch.int32)
    if expert_of.dim() != 2:
        raise ValueError("expert_of must have the shape [tokens, topk]")
    tokens, topk = expert_of.shape
    experts, align, capacity = int(experts), int(align), int(capacity)
    if rows is not None:
        rows = int(rows)
    else:
        rows = slot_of.numel() if slot_of is not None else mfx_moe_rows(tokens, topk, experts, align)
    slots = tokens * topk
    new = lambda t, name, shape: (_empty(shape, torch.int32, expert_of.device, stream) if t is None  # noqa: E731
                                  else _like(t, name, shape, torch.int32))
    row_of, slot_of = new(row_of, "row_of", (tokens, topk)), new(slot_of, "slot_of", (rows,))
    offsets, counts = new(offsets, "offsets", (max(experts, 0) + 1,)), new(counts, "counts", (max(experts, 0),))
    _with_workspace("mfx_moe_sort", (tokens, topk, experts, align, capacity, rows, expert_of.data_ptr(),
                                     row_of.data_ptr(), slot_of.data_ptr(), offsets.data_ptr(), counts.data_ptr()),
                    (_stream(stream, expert_of),), expert_of.device, workspace, (slots, experts), none=True, stream=stream)
    return row_of, slot_of, offsets, counts


def _moe_maps(x, row_of, slot_of=None):
    """(tokens, topk) of the maps, which must be int32 and on x's device."""
    _cuda(row_of, "row_of", torch.int32)
    if row_of.dim() != 2:
        raise ValueError("row_of must have the shape [tokens, topk]")
    dev = x.get_device()
    _same_device(row_of, dev, "row_of")
    if slot_of is not None:
        _cuda(slot_of, "slot_of", torch.int32)
        if slot_of.dim() != 1:
            raise ValueError("slot_of must have the shape [rows]")
        _same_device(slot_of, dev, "slot_of")
    return row_of.shape


def _moe_data(t, name, rows=None):
    _cuda(t, name)
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must have the shape [{'rows' if rows is None else rows}, cols]")
    return t.shape


def mfx_moe_permute_fwd(x, row_of, slot_of, weight=None, out=None, out_weight=None, stream=None):
    """(out [rows, cols], out_weight [rows]): x [tokens, cols] by the maps of
    mfx_moe_sort, padding rows zero; out_weight is None without weight
    [tokens, topk] (fp32)."""
    tokens, topk = _moe_maps(x, row_of, slot_of)
    _, cols = _moe_data(x, "x", tokens)
    rows = slot_of.shape[0]
    out = _empty((rows, cols), x.dtype, x.device, stream) if out is None else _like(out, "out", (rows, cols), x.dtype)
    if weight is not None:
        _like(weight, "weight", (tokens, topk), torch.float32)
        out_weight = (_empty(rows, torch.float32, x.device, stream) if out_weight is None
                      else _like(out_weight, "out_weight", (rows,), torch.float32))
    elif out_weight is not None:
        raise ValueError("out_weight needs a weight")
    _call("mfx_moe_permute_fwd", dtype_code(x.dtype), tokens, topk, cols, rows, _ptr(x), _ptr(row_of), _ptr(slot_of),
          _ptr(weight), _ptr(out), _ptr(out_weight), _stream(stream, x))
    return out, out_weight


def mfx_moe_permute_bwd(g, row_of, g_weight=None, dx=None, dweight=None, stream=None):
    """(dx [tokens, cols], dweight [tokens, topk]) from the gradients g [rows,
    cols] and g_weight [rows] of mfx_moe_permute_fwd's outputs; dweight is
    None without g_weight."""
    tokens, topk = _moe_maps(g, row_of)
    rows, cols = _moe_data(g, "g")
    dx = _empty((tokens, cols), g.dtype, g.device, stream) if dx is None else _like(dx, "dx", (tokens, cols), g.dtype)
    if g_weight is not None:
        _like(g_weight, "g_weight", (rows,), torch.float32)
        dweight = (_empty((tokens, topk), torch.float32, g.device, stream) if dweight is None
                   else _like(dweight, "dweight", (tokens, topk), torch.float32))
    elif dweight is not None:
        raise ValueError("dweight needs g_weight")
    _call("mfx_moe_permute_bwd", dtype_code(g.dtype), tokens, topk, cols, rows, _ptr(g), _ptr(row_of), _ptr(g_weight),
          _ptr(dx), _ptr(dweight), _stream(stream, g))
    return dx, dweight


def mfx_moe_unpermute_fwd(y, row_of, weight=None, out=None, stream=None):
    """out [tokens, cols] = sum over a token's rows of y [rows, cols], times
    weight [tokens, topk] (fp32) where given."""
    tokens, topk = _moe_maps(y, row_of)
    rows, cols = _moe_data(y, "y")
    if weight is not None:
        _like(weight, "weight", (tokens, topk), torch.float32)
    out = _empty((tokens, cols), y.dtype, y.device, stream) if out is None else _like(out, "out", (tokens, cols), y.dtype)
    _call("mfx_moe_unpermute_fwd", dtype_code(y.dtype), tokens, topk, cols, rows, _ptr(y), _ptr(row_of), _ptr(weight),
          _ptr(out), _stream(stream, y))
    return out


def mfx_moe_unpermute_bwd(g, y, row_of, slot_of, weight=None, dy=None, dweight=None, need_dweight=None, stream=None):
    """(dy [rows, cols], dweight [tokens, topk]) from the gradient g [tokens,
    cols] of mfx_moe_unpermute_fwd's output.  dweight is formed where weight
    is given (need_dweight overrides); without it y may be None."""
    tokens, topk = _moe_maps(g, row_of, slot_of)
    _, cols = _moe_data(g, "g", tokens)
    rows = slot_of.shape[0]
    if weight is not None:
        _like(weight, "weight", (tokens, topk), torch.float32)
    if y is not None:
        _like(y, "y", (rows, cols), g.dtype)
    if need_dweight is None:
        need_dweight = weight is not None or dweight is not None
    if need_dweight:
        if y is None:
            raise ValueError("dweight needs y")
        dweight = (_empty((tokens, topk), torch.float32, g.device, stream) if dweight is None
                   else _like(dweight, "dweight", (tokens, topk), torch.float32))
    else:
        dweight = None
    dy = _empty((rows, cols), g.dtype, g.device, stream) if dy is None else _like(dy, "dy", (rows, cols), g.dtype)
    _call("mfx_moe_unpermute_bwd", dtype_code(g.dtype), tokens, topk, cols, rows, _ptr(g), _ptr(y), _ptr(row_of),
          _ptr(slot_of), _ptr(weight), _ptr(dy), _ptr(dweight), _stream(stream, g))
    return dy, dweight


# ---------------------------------------------------------------------------
# root-mean-square norm with the residual's addition
# ---------------------------------------------------------------------------
_DTYPES = {torch.bfloat16: MFX_BF16, torch.float32: MFX_F32}
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _buf(t, name, shape, dtype, dev):
    """The address of t, a contiguous tensor of this shape and dtype on device
    dev; says what is wrong otherwise."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    _like(t, name, shape, dtype)
    _same_device(t, dev, name)
    return t.data_ptr()


def _new(t, name, shape, dtype, dev, like, stream):
    """(t or memory of the call's own, its address)."""
    if t is not None:
        return t, _buf(t, name, shape, dtype, dev)
    t = (torch.empty(shape, dtype=dtype, device=like.device) if stream is None
         else _empty(shape, dtype, like.device, stream))
    return t, t.data_ptr()


def _run(name, dev, *args):
    """A call whose kernels go to device dev, whichever is the current one."""
    fn = getattr(_lib or lib(), name)
    if dev == _current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != 0:
        raise MfxError(st, name)


def _run_with_workspace(name, dev, head, tail, device, workspace, sizes, stream):
    """The same for a call with a workspace, which may need none."""
    if dev == _current_device():
        _with_workspace(name, head, tail, device, workspace, sizes, none=True, stream=stream)
    else:
        with torch.cuda.device(dev):
            _with_workspace(name, head, tail, device, workspace, sizes, none=True, stream=stream)


def _stream_of(stream, t, dev):
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream, t)


def _float_code(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _DTYPES.get(t.dtype)
    return dtype_code(t.dtype) if code is None else code


def _norm_data(x, name):
    """(type code, device, shape, rows, cols) of the norm's data."""
    code = _float_code(x, name)
    dev, shape = x.get_device(), x.shape
    if dev < 0 or not x.is_contiguous() or not shape:
        _cuda(x, name)
        raise ValueError(f"{name} must have at least one dim")
    cols = shape[-1]
    return code, dev, shape, x.numel() // cols if cols else math.prod(shape[:-1]), cols


def mfx_add_rmsnorm_fwd(x, weight, residual=None, eps=1e-6, weight_offset=0.0, y=None, h=None, rstd=None,
                        need_rstd=True, stream=None):
    """(y, h, rstd): h = x + residual in the residual's dtype (None without a
    residual), y = h * rstd * (weight + weight_offset) over the last dim with
    rstd = 1 / sqrt(mean(h^2) + eps) ([rows], None with need_rstd=False).
    weight [cols] may be None."""
    xdt, dev, shape, rows, cols = _norm_data(x, "x")
    rdt = wdt = xdt
    rptr = wptr = hptr = sptr = None
    if weight is not None:
        wdt = _float_code(weight, "weight")
        wptr = _buf(weight, "weight", (cols,), weight.dtype, dev)
    if residual is not None:
        rdt = _float_code(residual, "residual")
        rptr = _buf(residual, "residual", shape, residual.dtype, dev)
        h, hptr = _new(h, "h", shape, residual.dtype, dev, x, stream)
    elif h is not None:
        raise ValueError("h needs a residual")
    y, yptr = _new(y, "y", shape, x.dtype, dev, x, stream)
    if need_rstd or rstd is not None:
        rstd, sptr = _new(rstd, "rstd", (rows,), torch.float32, dev, x, stream)
    _run("mfx_add_rmsnorm_fwd", dev, xdt, rdt, wdt, rows, cols, x.data_ptr(), rptr, wptr, float(eps),
         float(weight_offset), yptr, hptr, sptr, _stream_of(stream, x, dev))
    return y, h, rstd


_Q_DTYPES = {torch.float8_e4m3fn: MFX_E4M3, torch.float8_e5m2: MFX_E5M2}
_SCALE_DTYPES = {torch.float32: MFX_F32, torch.float8_e8m0fnu: MFX_E8M0}


def mfx_add_rmsnorm_quant_fwd(x, weight, residual=None, eps=1e-6, weight_offset=0.0, group=0,
                              q_dtype=torch.float8_e4m3fn, scale_dtype=torch.float32, q=None, scale=None, h=None,
                              rstd=None, need_rstd=False, stream=None):
    """(q, scale, h, rstd): mfx_add_rmsnorm_fwd with y in 8 bits, y ~ q *
    scale.  One scale per row (group=0) or per 32 or 128 columns of it, scale
    [..., groups]; float8_e8m0fnu scales are powers of two."""
    xdt, dev, shape, rows, cols = _norm_data(x, "x")
    qdt, sdt = _Q_DTYPES.get(q_dtype), _SCALE_DTYPES.get(scale_dtype)
    if qdt is None or sdt is None:
        raise TypeError("q is float8_e4m3fn or float8_e5m2, scale float32 or float8_e8m0fnu")
    group = int(group)
    if group not in (0, 32, 128):
        raise MfxError(9, "mfx_add_rmsnorm_quant_fwd")
    rdt = wdt = xdt
    rptr = wptr = hptr = sptr = None
    if weight is not None:
        wdt = _float_code(weight, "weight")
        wptr = _buf(weight, "weight", (cols,), weight.dtype, dev)
    if residual is not None:
        rdt = _float_code(residual, "residual")
        rptr = _buf(residual, "residual", shape, residual.dtype, dev)
        h, hptr = _new(h, "h", shape, residual.dtype, dev, x, stream)
    elif h is not None:
        raise ValueError("h needs a residual")
    groups = -(-cols // group) if group else min(cols, 1)
    q, qptr = _new(q, "q", shape, q_dtype, dev, x, stream)
    scale, scptr = _new(scale, "scale", (*shape[:-1], groups), scale_dtype, dev, x, stream)
    if need_rstd or rstd is not None:
        rstd, sptr = _new(rstd, "rstd", (rows,), torch.float32, dev, x, stream)
    _run("mfx_add_rmsnorm_quant_fwd", dev, xdt, rdt, wdt, rows, cols, x.data_ptr(), rptr, wptr, float(eps),
         float(weight_offset), qdt, group, sdt, qptr, scptr, hptr, sptr, _stream_of(stream, x, dev))
    return q, scale, h, rstd


def mfx_add_rmsnorm_bwd(dy, h, rstd, weight, dh=None, weight_offset=0.0, dx=None, dresidual=None, residual_dtype=None,
                        dweight=None, need_dweight=True, workspace=None, stream=None):
    """(dx, dresidual, dweight) from the forward's h (x where there was no
    residual) and rstd, the gradient dy of y and, where given, dh of h.
    dresidual is produced when a buffer is given or residual_dtype (h's dtype)
    is set; with dy's dtype and no buffer it is dx itself.  dweight is None
    without a weight or with need_dweight=False."""
    xdt, dev, shape, rows, cols = _norm_data(dy, "dy")
    rdt, wdt = _float_code(h, "h"), xdt
    hptr = _buf(h, "h", shape, h.dtype, dev)
    sptr = _buf(rstd, "rstd", (rows,), torch.float32, dev)
    wptr = eptr = rptr = dwptr = None
    if weight is not None:
        wdt = _float_code(weight, "weight")
        wptr = _buf(weight, "weight", (cols,), weight.dtype, dev)
    if dh is not None:
        eptr = _buf(dh, "dh", shape, h.dtype, dev)
    dx, xptr = _new(dx, "dx", shape, dy.dtype, dev, dy, stream)
    if dresidual is not None or residual_dtype is not None:
        if residual_dtype is not None and residual_dtype != h.dtype:
            raise TypeError(f"residual_dtype must be h's, {h.dtype}")
        if dresidual is None and rdt == xdt:
            dresidual = dx
        else:
            dresidual, rptr = _new(dresidual, "dresidual", shape, h.dtype, dev, dy, stream)
    if dweight is not None and weight is None:
        raise ValueError("dweight needs a weight")
    if dweight is not None or (weight is not None and need_dweight):
        dweight, dwptr = _new(dweight, "dweight", (cols,), weight.dtype, dev, dy, stream)
    head = (xdt, rdt, wdt, rows, cols, dy.data_ptr(), hptr, sptr, wptr, float(weight_offset), eptr, xptr, rptr, dwptr)
    _run_with_workspace("mfx_add_rmsnorm_bwd", dev, head, (_stream_of(stream, dy, dev),), dy.device, workspace,
                        (dev, xdt, rdt, rows, cols, dwptr is None), stream)
    return dx, dresidual, dweight


# ---------------------------------------------------------------------------
# operators on logits
# ---------------------------------------------------------------------------
_INDEX_BITS = {torch.int32: 32, torch.int64: 64}


def _logit_rows(t, name):
    """(type code, device, rows, vocab, ld) of [rows, vocab] data whose rows lie
    ld elements apart."""
    code = _float_code(t, name)
    dev, shape = t.get_device(), t.shape
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if len(shape) != 2:
        raise ValueError(f"{name} must have the shape [rows, vocab]")
    rows, vocab = shape
    if t.is_contiguous():
        return code, dev, rows, vocab, vocab
    ld, step = t.stride()
    if vocab > 1 and step != 1:
        raise ValueError(f"{name}'s columns must be contiguous")
    if rows > 1 and ld < vocab:
        raise ValueError(f"{name}'s rows must not overlap")
    return code, dev, rows, vocab, ld if rows > 1 else vocab


def _columns(t, name, shape, dev):
    """(bits, address) of an index array of the given shape."""
    bits = _INDEX_BITS.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if bits is None:
        raise TypeError(f"{name} must be an int32 or int64 tensor")
    return bits, _buf(t, name, shape, t.dtype, dev)


def _dlogits(dlogits, logits, dev, rows, vocab, stream):
    """(buffer, its address, its ld): contiguous if it is allocated here."""
    if dlogits is None:
        return *_new(None, "dlogits", (rows, vocab), logits.dtype, dev, logits, stream), vocab
    if not isinstance(dlogits, torch.Tensor) or dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits must be a {logits.dtype} tensor")
    _, _, r, v, ld = _logit_rows(dlogits, "dlogits")
    if (r, v) != (rows, vocab):
        raise ValueError("dlogits must have the logits' shape")
    _same_device(dlogits, dev, "dlogits")
    return dlogits, dlogits.data_ptr(), ld


def mfx_token_logprobs_fwd(logits, tokens, scale=1.0, top=0, logprob=None, entropy=None, top_logprob=None,
                           top_index=None, stats=None, need_stats=True, workspace=None, stream=None):
    """(logprob [rows], entropy [rows], top_logprob [rows, top], top_index
    [rows, top], stats [rows, 3]) of softmax(scale * logits [rows, vocab]) at
    tokens [rows] (int32 or int64; one outside the vocabulary leaves its row
    out).  The alternatives are None with top=0, stats with need_stats=False.
    logits' rows may lie further apart than the vocabulary is wide."""
    code, dev, rows, vocab, ld = _logit_rows(logits, "logits")
    bits, kptr = _columns(tokens, "tokens", (rows,), dev)
    top, f32 = int(top), torch.float32
    vptr = iptr = sptr = None
    logprob, lptr = _new(logprob, "logprob", (rows,), f32, dev, logits, stream)
    entropy, eptr = _new(entropy, "entropy", (rows,), f32, dev, logits, stream)
    if top > 0:
        top_logprob, vptr = _new(top_logprob, "top_logprob", (rows, top), f32, dev, logits, stream)
        top_index, iptr = _new(top_index, "top_index", (rows, top), torch.int32, dev, logits, stream)
    elif top_logprob is not None or top_index is not None:
        raise ValueError("top_logprob and top_index need top")
    if stats is not None or need_stats:
        stats, sptr = _new(stats, "stats", (rows, 3), f32, dev, logits, stream)
    head = (code, rows, vocab, ld, logits.data_ptr(), bits, kptr, float(scale), top, lptr, eptr, vptr, iptr, sptr)
    st = _stream_of(stream, logits, dev)
    if top > 0:
        _run_with_workspace("mfx_token_logprobs_fwd", dev, head, (st,), logits.device, workspace, (dev, code, rows, vocab), stream)
    else:
        _run("mfx_token_logprobs_fwd", dev, *head, None, None, st)
    return logprob, entropy, top_logprob, top_index, stats


def mfx_token_logprobs_bwd(g_logprob, g_entropy, logits, tokens, stats, scale=1.0, dlogits=None, stream=None):
    """dlogits [rows, vocab] from the gradients of logprob and entropy (either
    may be None) and the forward's inputs and stats; dlogits may be logits."""
    code, dev, rows, vocab, ld = _logit_rows(logits, "logits")
    bits, kptr = _columns(tokens, "tokens", (rows,), dev)
    g = None if g_logprob is None else _buf(g_logprob, "g_logprob", (rows,), torch.float32, dev)
    ge = None if g_entropy is None else _buf(g_entropy, "g_entropy", (rows,), torch.float32, dev)
    sptr = _buf(stats, "stats", (rows, 3), torch.float32, dev)
    dlogits, dptr, ldo = _dlogits(dlogits, logits, dev, rows, vocab, stream)
    _run("mfx_token_logprobs_bwd", dev, code, rows, vocab, ld, g, ge, logits.data_ptr(), bits, kptr, sptr, float(scale), dptr,
         ldo, _stream_of(stream, logits, dev))
    return dlogits


def _distill_args(logits, index, teacher, teacher_lse):
    """(device, rows, arguments up to k, logits' to teacher's, teacher_lse's address)."""
    code, dev, rows, vocab, ld = _logit_rows(logits, "logits")
    tdt = _float_code(teacher, "teacher")
    if teacher.dim() != 2:
        raise ValueError("teacher must have the shape [rows, k]")
    k = teacher.shape[1]
    tptr = _buf(teacher, "teacher", (rows, k), teacher.dtype, dev)
    bits, iptr = _columns(index, "index", (rows, k), dev)
    lse = None if teacher_lse is None else _buf(teacher_lse, "teacher_lse", (rows,), torch.float32, dev)
    return dev, rows, (code, tdt, rows, vocab, ld, k), (logits.data_ptr(), bits, iptr, tptr), lse


def mfx_topk_distill_fwd(logits, index, teacher, scale=1.0, teacher_lse=None, loss=None, stats=None, need_stats=True,
                         stream=None):
    """(loss [rows], stats [rows, 4]): sum of q (log q - log p) over the
    teacher's entries, p = softmax(scale * logits [rows, vocab]) and q the same
    of teacher [rows, k] at the columns index [rows, k] (int32 or int64,
    negative for no entry), or exp(scale * teacher - teacher_lse [rows]).  A row
    without entries has loss 0 and a gradient of zeros."""
    dev, rows, head, data, lse = _distill_args(logits, index, teacher, teacher_lse)
    loss, lptr = _new(loss, "loss", (rows,), torch.float32, dev, logits, stream)
    sptr = None
    if stats is not None or need_stats:
        stats, sptr = _new(stats, "stats", (rows, 4), torch.float32, dev, logits, stream)
    _run("mfx_topk_distill_fwd", dev, *head, *data, lse, float(scale), lptr, sptr, _stream_of(stream, logits, dev))
    return loss, stats


def mfx_topk_distill_bwd(g, logits, index, teacher, stats, scale=1.0, teacher_lse=None, dlogits=None, stream=None):
    """dlogits [rows, vocab] from the gradient g [rows] of the loss and the
    forward's inputs and stats (which hold what teacher_lse says); dlogits may
    be logits."""
    dev, rows, head, data, _ = _distill_args(logits, index, teacher, teacher_lse)
    gptr = _buf(g, "g", (rows,), torch.float32, dev)
    sptr = _buf(stats, "stats", (rows, 4), torch.float32, dev)
    dlogits, dptr, ldo = _dlogits(dlogits, logits, dev, rows, head[3], stream)
    _run("mfx_topk_distill_bwd", dev, *head, gptr, *data, sptr, float(scale), dptr, ldo, _stream_of(stream, logits, dev))
    return dlogits


def mfx_topk_distill_fwd_bwd(logits, index, teacher, weight, scale=1.0, teacher_lse=None, loss=None, dlogits=None,
                             stream=None):
    """(loss [rows], dlogits [rows, vocab]) in one call, where the gradient
    weight [rows] of each row's loss is known before it; dlogits may be
    logits."""
    dev, rows, head, data, lse = _distill_args(logits, index, teacher, teacher_lse)
    gptr = _buf(weight, "weight", (rows,), torch.float32, dev)
    loss, lptr = _new(loss, "loss", (rows,), torch.float32, dev, logits, stream)
    dlogits, dptr, ldo = _dlogits(dlogits, logits, dev, rows, head[3], stream)
    _run("mfx_topk_distill_fwd_bwd", dev, *head, *data, lse, gptr, float(scale), lptr, dptr, ldo,
         _stream_of(stream, logits, dev))
    return loss, dlogits


# ---------------------------------------------------------------------------
# bias-dropout-add
# ---------------------------------------------------------------------------
def mfx_bias_dropout_add_train(x, bias, residual, p, seed, offset=0, elem_base=0, out=None,
                               keep_mask=None, stream=None):
    """Returns (out, keep_mask); keep_mask is uint8 (1 = kept)."""
    _cuda(x, "x")
    _cuda(bias, "bias", x.dtype)
    _cuda(residual, "residual")
    if residual.shape != x.shape:
        raise ValueError("residual must have x's shape")
    out = torch.empty_like(x) if out is None else _cuda(out, "out", x.dtype)
    keep_mask = (torch.empty(x.shape, dtype=torch.uint8, device=x.device) if keep_mask is None
                 else _cuda(keep_mask, "keep_mask", torch.uint8))
    rows, cols = _rows_cols(x)
    _call("mfx_bias_dropout_add_train", dtype_code(x.dtype), dtype_code(residual.dtype), rows, cols,
          _ptr(x), _ptr(bias), _ptr(residual), float(p), int(seed) % 2**64, int(offset) % 2**64,
          int(elem_base), _ptr(out), _ptr(keep_mask), _stream(stream, x))
    return out, keep_mask


def mfx_bias_dropout_add_inference(x, bias, residual, p=0.0, seed=0, offset=0, stream=None):
    """x = (x + bias) + residual.to(x.dtype), in place; returns x."""
    _cuda(x, "x")
    _cuda(bias, "bias", x.dtype)
    _cuda(residual, "residual")
    if residual.shape != x.shape:
        raise ValueError("residual must have x's shape")
    rows, cols = _rows_cols(x)
    _call("mfx_bias_dropout_add_inference", dtype_code(x.dtype), dtype_code(residual.dtype), rows,
          cols, _ptr(x), _ptr(bias), _ptr(residual), float(p), int(seed) % 2**64,
          int(offset) % 2**64, _stream(stream, x))
    return x


def mfx_bias_dropout_add_bwd(g, keep_mask, p, seed=0, offset=0, elem_base=0, dx=None, dresidual=None,
                             residual_dtype=None, stream=None):
    """Returns (dx, dresidual).  keep_mask None regenerates the forward's mask
    from (seed, offset, elem_base, p).  dresidual is produced when a buffer
    is given or residual_dtype is set (and differs from g's dtype; with the
    same dtype the residual gradient is g itself)."""
    _cuda(g, "g")
    _cuda(keep_mask, "keep_mask", torch.uint8)
    dx = torch.empty_like(g) if dx is None else _cuda(dx, "dx", g.dtype)
    if dresidual is None and residual_dtype is not None:
        dresidual = g if residual_dtype == g.dtype else torch.empty(g.shape, dtype=residual_dtype,
                                                                     device=g.device)
    _cuda(dresidual, "dresidual")
    rdt = dtype_code(dresidual.dtype) if dresidual is not None else dtype_code(g.dtype)
    rows, cols = _rows_cols(g)
    _call("mfx_bias_dropout_add_bwd", dtype_code(g.dtype), rdt, rows, cols, _ptr(g), _ptr(keep_mask),
          float(p), int(seed) % 2**64, int(offset) % 2**64, int(elem_base), _ptr(dx), _ptr(dresidual),
          _stream(stream, g))
    return dx, dresidual


def mfx_bias_dropout_add_train_packed(x, bias, residual, p, seed, offset=0, elem_base=0, out=None,
                                      keep_bits=None, stream=None):
    """Returns (out, keep_bits): the keep mask as bits, element i at bit i % 8
    of byte i // 8 (uint8, ceil(numel / 8) bytes)."""
    _cuda(x, "x")
    _cuda(bias, "bias", x.dtype)
    _cuda(residual, "residual")
    if residual.shape != x.shape:
        raise ValueError("residual must have x's shape")
    out = torch.empty_like(x) if out is None else _cuda(out, "out", x.dtype)
    nbytes = (x.numel() + 7) // 8
    keep_bits = (torch.empty(nbytes, dtype=torch.uint8, device=x.device) if keep_bits is None
                 else _cuda(keep_bits, "keep_bits", torch.uint8))
    if keep_bits.numel() < nbytes:
        raise ValueError(f"keep_bits needs {nbytes} bytes")
    rows, cols = _rows_cols(x)
    _call("mfx_bias_dropout_add_train_packed", dtype_code(x.dtype), dtype_code(residual.dtype), rows, cols,
          _ptr(x), _ptr(bias), _ptr(residual), float(p), int(seed) % 2**64, int(offset) % 2**64,
          int(elem_base), _ptr(out), _ptr(keep_bits), _stream(stream, x))
    return out, keep_bits


def mfx_bias_dropout_add_bwd_packed(g, keep_bits, p, dx=None, dresidual=None, residual_dtype=None, stream=None):
    """(dx, dresidual) from the bit mask of mfx_bias_dropout_add_train_packed."""
    _cuda(g, "g")
    _cuda(keep_bits, "keep_bits", torch.uint8)
    if keep_bits.numel() < (g.numel() + 7) // 8:
        raise ValueError("keep_bits is shorter than the mask")
    dx = torch.empty_like(g) if dx is None else _cuda(dx, "dx", g.dtype)
    if dresidual is None and residual_dtype is not None:
        dresidual = g if residual_dtype == g.dtype else torch.empty(g.shape, dtype=residual_dtype,
                                                                     device=g.device)
    _cuda(dresidual, "dresidual")
    rdt = dtype_code(dresidual.dtype) if dresidual is not None else dtype_code(g.dtype)
    rows, cols = _rows_cols(g)
    _call("mfx_bias_dropout_add_bwd_packed", dtype_code(g.dtype), rdt, rows, cols, _ptr(g), _ptr(keep_bits),
          float(p), _ptr(dx), _ptr(dresidual), _stream(stream, g))
    return dx, dresidual


def mfx_bias_dropout_add_train_nomask(x, bias, residual, p, seed, offset=0, elem_base=0, out=None, stream=None):
    """out of mfx_bias_dropout_add_train, without writing a mask; the backward
    regenerates it (mfx_bias_dropout_add_bwd with keep_mask=None)."""
    _cuda(x, "x")
    _cuda(bias, "bias", x.dtype)
    _cuda(residual, "residual")
    if residual.shape != x.shape:
        raise ValueError("residual must have x's shape")
    out = _empty_like(x, stream) if out is None else _like(out, "out", x.shape, x.dtype)
    rows, cols = _rows_cols(x)
    if bias is not None and bias.numel() != cols:
        raise ValueError("bias must have one element per column of x")
    _call("mfx_bias_dropout_add_train_nomask", dtype_code(x.dtype), dtype_code(residual.dtype), rows, cols, _ptr(x),
          _ptr(bias), _ptr(residual), float(p), int(seed) % 2**64, int(offset) % 2**64, int(elem_base), _ptr(out),
          _stream(stream, x))
    return out


def _dropout(name, x, p, seed, offset, elem_base, out, what, stream):
    _cuda(x, what[0])
    out = _empty_like(x, stream) if out is None else _like(out, what[1], x.shape, x.dtype)
    _call(name, dtype_code(x.dtype), x.numel(), _ptr(x), float(p), int(seed) % 2**64, int(offset) % 2**64,
          int(elem_base), _ptr(out), _stream(stream, x))
    return out


def mfx_dropout_fwd(x, p, seed, offset=0, elem_base=0, out=None, stream=None):
    """out = dropout(x, p); the mask is a function of (seed, offset, element
    index) and is not stored."""
    return _dropout("mfx_dropout_fwd", x, p, seed, offset, elem_base, out, ("x", "out"), stream)


def mfx_dropout_bwd(g, p, seed, offset=0, elem_base=0, dx=None, stream=None):
    """dx of mfx_dropout_fwd from the gradient g and the forward's p, seed,
    offset and elem_base."""
    return _dropout("mfx_dropout_bwd", g, p, seed, offset, elem_base, dx, ("g", "dx"), stream)


# ---------------------------------------------------------------------------
# fused bias gradients (workspace protocol: query the size, then run)
# ---------------------------------------------------------------------------
_workspace_bytes = {}  # (entry point, sizes) -> bytes, for calls that say which sizes theirs goes by
_WORKSPACE_SIZES = 1024  # most of them (lengths may differ from call to call): then they are asked for anew


def _with_workspace(name, args_before_ws, tail, device, workspace=None, sizes=None, none=False, stream=None):
    """Query the workspace size, allocate it and run `name`.  `workspace` is
    None (a fresh uint8 tensor of the call's stream, `stream` as its caller
    gave it), a uint8 CUDA tensor, or a callable that takes the byte count and
    returns one (a caller's own allocator).
    `sizes`: what the workspace's size depends on, so that it is asked for
    once; `none`: a call whose workspace is empty takes none."""
    need = _workspace_bytes.get((name, sizes)) if sizes is not None else None
    if need is None:
        size = C.c_size_t(0)
        _call(name, *args_before_ws, None, C.byref(size), *tail)
        need = int(size.value)
        if sizes is not None:
            if len(_workspace_bytes) >= _WORKSPACE_SIZES:
                _workspace_bytes.clear()
            _workspace_bytes[(name, sizes)] = need
    if workspace is not None:
        if callable(workspace):
            workspace = workspace(max(need, 16))
        _cuda(workspace, "workspace", torch.uint8)
        if workspace.numel() == 0:  # a null pointer would ask for the size again, and nothing would run
            if not none or need:
                raise MfxError(8, name)
            workspace = None
    if workspace is None:
        if none and need == 0:
            _call(name, *args_before_ws, None, None, *tail)
            return None
        workspace = _empty(max(need, 16), torch.uint8, device, stream)
    size = C.c_size_t(workspace.numel())
    _call(name, *args_before_ws, workspace.data_ptr(), C.byref(size), *tail)
    return workspace


def mfx_bias_gelu_bwd_dbias(g, bias, y, dy=None, dbias=None, workspace=None, stream=None):
    """(dy, dbias): bias-GeLU backward and the bias gradient sum_r dy[r, :]."""
    _cuda(y, "y")
    _cuda(g, "g", y.dtype)
    _cuda(bias, "bias", y.dtype)
    rows, cols = _rows_cols(y)
    dy = torch.empty_like(y) if dy is None else _cuda(dy, "dy", y.dtype)
    dbias = y.new_empty((cols,)) if dbias is None else _cuda(dbias, "dbias", y.dtype)
    st = _stream(stream, y)
    _with_workspace("mfx_bias_gelu_bwd_dbias",
                    (dtype_code(y.dtype), rows, cols, _ptr(g), _ptr(bias), _ptr(y), _ptr(dy), _ptr(dbias)),
                    (st,), y.device, workspace, stream=stream)
    return dy, dbias


def mfx_bias_gelu_bwd_dbias_noalloc(g, bias, y, dy=None, dbias=None, stream=None):
    """(dy, dbias) as mfx_bias_gelu_bwd_dbias, with the library's fixed
    device scratch instead of a caller workspace (widths up to the scratch
    size; concurrent calls on the GPU must be serialised)."""
    _cuda(y, "y")
    _cuda(g, "g", y.dtype)
    _cuda(bias, "bias", y.dtype)
    rows, cols = _rows_cols(y)
    dy = torch.empty_like(y) if dy is None else _cuda(dy, "dy", y.dtype)
    dbias = y.new_empty((cols,)) if dbias is None else _cuda(dbias, "dbias", y.dtype)
    _call("mfx_bias_gelu_bwd_dbias_noalloc", dtype_code(y.dtype), rows, cols, _ptr(g), _ptr(bias), _ptr(y),
          _ptr(dy), _ptr(dbias), _stream(stream, y))
    return dy, dbias


def mfx_bias_geglu_bwd_dbias(g, x, bias, dx=None, dbias=None, workspace=None, stream=None):
    """(dx, dbias): GEGLU backward and the bias gradient over the width 2F."""
    _cuda(x, "x")
    _cuda(g, "g", x.dtype)
    _cuda(bias, "bias", x.dtype)
    rows, F = _glu_shape(x)
    dx = torch.empty_like(x) if dx is None else _cuda(dx, "dx", x.dtype)
    dbias = x.new_empty((2 * F,)) if dbias is None else _cuda(dbias, "dbias", x.dtype)
    _with_workspace("mfx_bias_geglu_bwd_dbias",
                    (dtype_code(x.dtype), rows, F, _ptr(g), _ptr(x), _ptr(bias), _ptr(dx), _ptr(dbias)),
                    (_stream(stream, x),), x.device, workspace, stream=stream)
    return dx, dbias


def mfx_bias_swiglu_bwd_dbias(g, x, bias, weight=None, dx=None, dweight=None, dbias=None, workspace=None,
                              stream=None):
    """(dx, dweight, dbias): SwiGLU backward (optionally weighted) and the bias
    gradient over the width 2F."""
    _cuda(x, "x")
    _cuda(g, "g", x.dtype)
    _cuda(bias, "bias", x.dtype)
    _cuda(weight, "weight", torch.float32)
    rows, F = _glu_shape(x)
    dx = torch.empty_like(x) if dx is None else _cuda(dx, "dx", x.dtype)
    if weight is not None and dweight is None:
        dweight = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
    dbias = x.new_empty((2 * F,)) if dbias is None else _cuda(dbias, "dbias", x.dtype)
    _with_workspace("mfx_bias_swiglu_bwd_dbias",
                    (dtype_code(x.dtype), rows, F, _ptr(g), _ptr(x), _ptr(bias), _ptr(weight), _ptr(dx),
                     _ptr(dweight), _ptr(dbias)), (_stream(stream, x),), x.device, workspace, stream=stream)
    return dx, dweight, dbias


def mfx_bias_dropout_add_bwd_dbias(g, keep_mask, p, seed=0, offset=0, elem_base=0, dx=None, dresidual=None,
                                   residual_dtype=None, dbias=None, workspace=None, stream=None):
    """(dx, dresidual, dbias): bias-dropout-add backward and the bias
    gradient sum_r dx[r, :]."""
    _cuda(g, "g")
    _cuda(keep_mask, "keep_mask", torch.uint8)
    dx = torch.empty_like(g) if dx is None else _cuda(dx, "dx", g.dtype)
    if dresidual is None and residual_dtype is not None:
        dresidual = g if residual_dtype == g.dtype else torch.empty(g.shape, dtype=residual_dtype,
                                                                     device=g.device)
    _cuda(dresidual, "dresidual")
    rdt = dtype_code(dresidual.dtype) if dresidual is not None else dtype_code(g.dtype)
    rows, cols = _rows_cols(g)
    dbias = g.new_empty((cols,)) if dbias is None else _cuda(dbias, "dbias", g.dtype)
    _with_workspace("mfx_bias_dropout_add_bwd_dbias",
                    (dtype_code(g.dtype), rdt, rows, cols, _ptr(g), _ptr(keep_mask), float(p),
                     int(seed) % 2**64, int(offset) % 2**64, int(elem_base), _ptr(dx), _ptr(dresidual),
                     _ptr(dbias)), (_stream(stream, g),), g.device, workspace, stream=stream)
    return dx, dresidual, dbias
