"""ctypes binding of libbsq.so (declared in include/bsq.h): same entry-point names, argument
marshalling only.  Every computation runs in the library's CUDA kernels; there is no
fallback path -- if the library or a GPU is missing, the calls raise.

Tensors are torch tensors on the current CUDA device; a packed operand is any object
with the attributes ``fmt, data, scale, tensor_scale, batch, rows, cols`` (for example
``block_scaled_gemm_fp8_gb300.synth.Packed``).
"""

import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbsq.so")
HEADER_PATH = os.path.join(HERE, "..", "include", "bsq.h")

BSQ_BF16, BSQ_FP8_E4M3_B128, BSQ_MXFP4, BSQ_NVFP4, BSQ_FP8_E4M3_TENSOR, BSQ_FP8_E5M2_TENSOR = 0, 1, 2, 3, 4, 5
BSQ_OK, BSQ_ERR_INVALID_ARG, BSQ_ERR_UNSUPPORTED, BSQ_ERR_CUDA, BSQ_ERR_TIMEOUT = 0, 1, 2, 3, 4
BSQ_NEEDS_GRAD_X, BSQ_NEEDS_GRAD_W = 1, 2
BSQ_DT_BF16, BSQ_DT_F32 = 0, 1

_c_void_p, _i64, _i32, _f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double

SIGNATURES = {
    "bsq_dequant": [_i32, _c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p],
    "bsq_linear_dgrad": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p],
    "bsq_linear_wgrad": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p],
    "bsq_grouped_dgrad": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i64, _i64, _c_void_p,
                          _c_void_p, _c_void_p],
    "bsq_grouped_wgrad": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _i64,
                          _c_void_p, _c_void_p],
    "bsq_linear_backward": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                            _c_void_p, _c_void_p, _i64, ctypes.c_uint32, _c_void_p, _c_void_p, _c_void_p],
    "bsq_linear_forward": [_i32, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i64,
                           _i64, _c_void_p, _c_void_p],
    "bsq_linear_dgrad_smallm_noalloc": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i64,
                                        _c_void_p, _c_void_p],
    "bsq_quantize_e5m2": [_c_void_p, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "bsq_linear_backward_e5m2": [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                                 _c_void_p, _c_void_p, _i64, ctypes.c_uint32, _i32, _c_void_p, _c_void_p,
                                 _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "bsq_quantize_e4m3": [_i32, _c_void_p, _i64, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p],
    "bsq_fp8_forward": [_c_void_p, _c_void_p, _i64, _i32, _c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p],
    "bsq_fp8_dgrad": [_c_void_p, _c_void_p, _i64, _i32, _c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p],
    "bsq_fp8_grouped_forward": [_c_void_p, _c_void_p, _i64, _i32, _c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p,
                                _c_void_p, _c_void_p],
    "bsq_fp8_grouped_dgrad": [_c_void_p, _c_void_p, _i64, _i32, _c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p,
                              _c_void_p, _c_void_p],
    "bsq_adamw": [_c_void_p, _i32, _i32, _i32, _i64, _f64, _f64, _f64, _f64, _c_void_p, ctypes.c_uint32, _c_void_p],
    "bsq_status_string": [_i32],
    "bsq_last_error": [],
    "bsq_get_device_error": [ctypes.POINTER(_i32), _c_void_p],
    "bsq_num_sms": [],
}
_RESTYPES = {"bsq_status_string": ctypes.c_char_p, "bsq_last_error": ctypes.c_char_p}


class BsqError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


_lib = None


def lib():
    """Load libbsq.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_scaled_gemm_fp8_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _RESTYPES.get(name, _i32)
        _lib = L
    return _lib


def header_entry_points():
    """Names of the functions include/bsq.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bsq_[a-z_]+)\s*\(", text)))


def status_string(s):
    return lib().bsq_status_string(int(s)).decode()


def last_error():
    return lib().bsq_last_error().decode()


def _check(status):
    if status != BSQ_OK:
        raise BsqError(status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def num_sms():
    return int(lib().bsq_num_sms())


def get_device_error(stream=None):
    """(status, code): synchronizes the stream and reads/clears the device error word."""
    code = _i32(0)
    st = lib().bsq_get_device_error(ctypes.byref(code), _stream(stream))
    return st, code.value


def _empty(shape, dtype, like, stream):
    """A new tensor on `like`'s device for a kernel on `stream`: of that stream's memory, so that no work
    queued elsewhere still uses it; reused, once freed, after what the current stream does with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def dequant(p, out=None, stream=None):
    """BF16 [batch, rows, cols] from a packed operand."""
    if out is None:
        out = _empty((p.batch, p.rows, p.cols), torch.bfloat16, p.data, stream)
    _check(lib().bsq_dequant(p.fmt, _ptr(p.data), _ptr(p.scale), _ptr(p.tensor_scale), p.batch, p.rows, p.cols,
                             _ptr(out), _stream(stream)))
    return out


def linear_dgrad(grad_out, w, out=None, stream=None):
    """grad_x[M,K] = grad_out[M,N] @ deq(W)[N,K]."""
    M, N = grad_out.shape
    if out is None:
        out = _empty((M, w.cols), torch.bfloat16, grad_out, stream)
    _check(lib().bsq_linear_dgrad(_ptr(grad_out), M, N, w.fmt, _ptr(w.data), _ptr(w.scale), _ptr(w.tensor_scale),
                                  w.cols, _ptr(out), _stream(stream)))
    return out


def linear_dgrad_smallm_noalloc(grad_out, w, out=None, stream=None):
    """grad_x[M,K] = grad_out[M,N] @ deq(W)[N,K] for M <= 16 without any device allocation
    (split-K scratch in a static device array of the library; K <= 16384)."""
    M, N = grad_out.shape
    if out is None:
        out = _empty((M, w.cols), torch.bfloat16, grad_out, stream)
    _check(lib().bsq_linear_dgrad_smallm_noalloc(_ptr(grad_out), M, N, w.fmt, _ptr(w.data), _ptr(w.scale),
                                                 _ptr(w.tensor_scale), w.cols, _ptr(out), _stream(stream)))
    return out


def linear_wgrad(grad_out, x, out=None, stream=None):
    """grad_w[N,K] = grad_out[M,N]^T @ deq(X)[M,K]."""
    M, N = grad_out.shape
    if out is None:
        out = _empty((N, x.cols), torch.bfloat16, grad_out, stream)
    _check(lib().bsq_linear_wgrad(_ptr(grad_out), M, N, x.fmt, _ptr(x.data), _ptr(x.scale), _ptr(x.tensor_scale),
                                  x.cols, _ptr(out), _stream(stream)))
    return out


def linear_backward(grad_out, w, x, needs=BSQ_NEEDS_GRAD_X | BSQ_NEEDS_GRAD_W, grad_x=None, grad_w=None,
                    stream=None):
    """(grad_x, grad_w): grad_out @ deq(W) and grad_out^T @ deq(X), each only when `needs` asks
    for it (None otherwise); one launch when both are wanted and W and X share a format."""
    M, N = grad_out.shape
    K = (w if w is not None else x).cols
    if needs & BSQ_NEEDS_GRAD_X and grad_x is None:
        grad_x = _empty((M, K), torch.bfloat16, grad_out, stream)
    if needs & BSQ_NEEDS_GRAD_W and grad_w is None:
        grad_w = _empty((N, K), torch.bfloat16, grad_out, stream)
    f = lambda p, a: None if p is None else getattr(p, a)
    _check(lib().bsq_linear_backward(
        _ptr(grad_out), M, N, f(w, "fmt") or 0, _ptr(f(w, "data")), _ptr(f(w, "scale")), _ptr(f(w, "tensor_scale")),
        f(x, "fmt") or 0, _ptr(f(x, "data")), _ptr(f(x, "scale")), _ptr(f(x, "tensor_scale")), K, needs,
        _ptr(grad_x) if needs & BSQ_NEEDS_GRAD_X else None, _ptr(grad_w) if needs & BSQ_NEEDS_GRAD_W else None,
        _stream(stream)))
    return (grad_x if needs & BSQ_NEEDS_GRAD_X else None), (grad_w if needs & BSQ_NEEDS_GRAD_W else None)


def quantize_e5m2(g, margin=0, codes=None, deq=None, want_deq=True, stream=None):
    """Per-tensor E5M2 quantization of a BF16 gradient with its current amax:
    (codes u8, step f32[1], amax f32[1], deq bf16 or None), all on g's device."""
    if codes is None:
        codes = _empty(g.shape, torch.uint8, g, stream)
    if deq is None and want_deq:
        deq = _empty(g.shape, torch.bfloat16, g, stream)
    step = _empty(1, torch.float32, g, stream)
    amax = _empty(1, torch.float32, g, stream)
    _check(lib().bsq_quantize_e5m2(_ptr(g), g.numel(), margin, _ptr(codes), _ptr(deq), _ptr(step), _ptr(amax),
                                   _stream(stream)))
    return codes, step, amax, deq


def linear_backward_e5m2(grad_out, w, x, needs=BSQ_NEEDS_GRAD_X | BSQ_NEEDS_GRAD_W, margin=0, grad_x=None,
                         grad_w=None, stream=None):
    """(grad_x, grad_w, step, amax): the backward on grad_out quantized once to E5M2 (step and
    amax are the quantization's, f32[1] on the device)."""
    M, N = grad_out.shape
    K = (w if w is not None else x).cols
    if needs & BSQ_NEEDS_GRAD_X and grad_x is None:
        grad_x = _empty((M, K), torch.bfloat16, grad_out, stream)
    if needs & BSQ_NEEDS_GRAD_W and grad_w is None:
        grad_w = _empty((N, K), torch.bfloat16, grad_out, stream)
    codes = _empty((M, N), torch.uint8, grad_out, stream)
    deq = _empty((M, N), torch.bfloat16, grad_out, stream)
    step = _empty(1, torch.float32, grad_out, stream)
    amax = _empty(1, torch.float32, grad_out, stream)
    f = lambda p, a: None if p is None else getattr(p, a)
    _check(lib().bsq_linear_backward_e5m2(
        _ptr(grad_out), M, N, f(w, "fmt") or 0, _ptr(f(w, "data")), _ptr(f(w, "scale")), _ptr(f(w, "tensor_scale")),
        f(x, "fmt") or 0, _ptr(f(x, "data")), _ptr(f(x, "scale")), _ptr(f(x, "tensor_scale")), K, needs, margin,
        _ptr(codes), _ptr(deq), _ptr(step), _ptr(amax),
        _ptr(grad_x) if needs & BSQ_NEEDS_GRAD_X else None, _ptr(grad_w) if needs & BSQ_NEEDS_GRAD_W else None,
        _stream(stream)))
    return (grad_x if needs & BSQ_NEEDS_GRAD_X else None), (grad_w if needs & BSQ_NEEDS_GRAD_W else None), step, amax


def linear_forward(x, w, out=None, stream=None):
    """y[M,N] = deq(X)[M,K] @ deq(W)[N,K]^T; W packed, X packed of W's kind or BF16 (fmt 0)."""
    if out is None:
        out = _empty((x.rows, w.rows), torch.bfloat16, x.data, stream)
    _check(lib().bsq_linear_forward(x.fmt, _ptr(x.data), _ptr(x.scale), _ptr(x.tensor_scale), x.rows, w.fmt,
                                    _ptr(w.data), _ptr(w.scale), _ptr(w.tensor_scale), w.rows, x.cols, _ptr(out),
                                    _stream(stream)))
    return out


def grouped_dgrad(grad_out, w, offsets, out=None, stream=None):
    """Per expert e: grad_x[r0:r1] = grad_out[r0:r1] @ deq(W[e]); rows past offsets[-1] untouched."""
    S, N = grad_out.shape
    if out is None:
        out = _empty((S, w.cols), torch.bfloat16, grad_out, stream)
    _check(lib().bsq_grouped_dgrad(_ptr(grad_out), S, N, w.fmt, _ptr(w.data), _ptr(w.scale), _ptr(w.tensor_scale),
                                   w.batch, w.cols, _ptr(offsets), _ptr(out), _stream(stream)))
    return out


def grouped_wgrad(grad_out, x, offsets, E, out=None, stream=None):
    """Per expert e: grad_w[e] = grad_out[r0:r1]^T @ deq(X)[r0:r1]; empty experts give zeros."""
    S, N = grad_out.shape
    if out is None:
        out = _empty((E, N, x.cols), torch.bfloat16, grad_out, stream)
    _check(lib().bsq_grouped_wgrad(_ptr(grad_out), S, N, x.fmt, _ptr(x.data), _ptr(x.scale), _ptr(x.tensor_scale),
                                   x.cols, _ptr(offsets), E, _ptr(out), _stream(stream)))
    return out


def _dense(t, dtypes, what):
    """t is a contiguous CUDA tensor of one of `dtypes`."""
    if t is None:
        raise ValueError(f"{what}: a CUDA tensor is wanted, not None")
    if not (t.dtype in dtypes and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{what}: a contiguous CUDA tensor of {' or '.join(map(str, dtypes))} is wanted, not "
                         f"{t.dtype} on {t.device}, strides {t.stride()}")


def _out(out, shape, dtype, like, stream, what):
    """`out` checked, or a new tensor for `stream`."""
    if out is not None:
        _dense(out, (dtype,), what)
        if out.shape != torch.Size(shape):
            raise ValueError(f"{what}: shape {tuple(out.shape)}, {tuple(shape)} is wanted")
        if out.get_device() != like.get_device():
            raise ValueError(f"{what}: on {out.device}, the operands are on {like.device}")
        return out
    return _empty(shape, dtype, like, stream)


# Index of the current device, without the checks torch.cuda.current_device() makes first.
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: -1)


def _refuse_device(name, t):
    raise ValueError(f"{name}: the operands are on {t.device}, kernels are launched on the current device, cuda:{_current_device()}")


def _raw_stream(stream, like):
    """The stream's handle; None: the current stream of `like`'s device, without building its object."""
    return torch._C._cuda_getCurrentRawStream(like.get_device()) if stream is None else stream.cuda_stream


_CODES = (torch.uint8, torch.float8_e4m3fn)
_F32 = (torch.float32,)
_DTYPES = {torch.bfloat16: BSQ_DT_BF16, torch.float32: BSQ_DT_F32}


def quantize_e4m3(x, block_rows=1, codes=None, scale=None, stream=None):
    """(codes u8, scale f32) of x (BF16 or float32, [rows, cols] or [batch, rows, cols]) in blocks of
    block_rows x 128, block_rows 1 (activations, gradients) or 128 (weights)."""
    dtype = _DTYPES.get(x.dtype)
    if dtype is None or not (x.is_cuda and x.is_contiguous()):
        _dense(x, _DTYPES, "quantize_e4m3: x")   # says what is wrong
    if x.get_device() != _current_device():
        _refuse_device("quantize_e4m3", x)
    shape = x.shape
    if len(shape) == 3:
        batch, rows, cols = shape
        blocks = (batch, rows if block_rows == 1 else (rows + 127) // 128, (cols + 127) // 128)
    elif len(shape) == 2:
        batch, (rows, cols) = 1, shape
        blocks = (rows if block_rows == 1 else (rows + 127) // 128, (cols + 127) // 128)
    else:
        raise ValueError(f"quantize_e4m3: x has {len(shape)} dimensions, 2 or 3 are wanted")
    if stream is None and codes is None and scale is None:
        codes = torch.empty(shape, dtype=torch.uint8, device=x.device)
        scale = torch.empty(blocks, dtype=torch.float32, device=x.device)
    else:
        codes = _out(codes, shape, torch.uint8, x, stream, "quantize_e4m3: codes")
        scale = _out(scale, blocks, torch.float32, x, stream, "quantize_e4m3: scale")
    status = (_lib or lib()).bsq_quantize_e4m3(dtype, x.data_ptr(), batch, rows, cols, block_rows, codes.data_ptr(),
                                               scale.data_ptr(), _raw_stream(stream, x))
    if status:
        _check(status)
    return codes, scale


def _fp8(name, codes, scale, w, inner, outer, offsets, out, stream):
    wd, ws, batch, n, k = w.data, w.scale, w.batch, w.rows, w.cols
    dev, rows, blocks = codes.get_device(), codes.shape[0], (inner + 127) // 128
    # one expression for the common case; what is wrong is looked for only when it fails
    if not (dev >= 0 and wd is not None and ws is not None and scale.get_device() == wd.get_device() == ws.get_device() == dev and codes.dtype in _CODES
            and wd.dtype in _CODES and scale.dtype is torch.float32 and ws.dtype is torch.float32
            and codes.shape == (rows, inner) and scale.shape == (rows, blocks) and codes.is_contiguous()
            and scale.is_contiguous() and wd.is_contiguous() and ws.is_contiguous() and wd.numel() == batch * n * k
            and (w.fmt != BSQ_FP8_E4M3_B128 or ws.numel() == batch * ((n + 127) // 128) * ((k + 127) // 128))):
        for t, dtypes, what in ((codes, _CODES, "codes"), (scale, _F32, "scale"), (wd, _CODES, "w.data"), (ws, _F32, "w.scale")):
            _dense(t, dtypes, f"{name}: {what}")
        raise ValueError(f"{name}: codes {tuple(codes.shape)} on {codes.device}, scale {tuple(scale.shape)} on {scale.device}; "
                         f"[rows, {inner}] and [rows, {blocks}] are wanted; w holds {wd.numel()} codes and {ws.numel()} scales "
                         f"on {wd.device} and {ws.device} for [{batch}, {n}, {k}]")
    if dev != _current_device():
        _refuse_device(name, codes)
    if stream is None and out is None:
        out = torch.empty((rows, outer), dtype=torch.bfloat16, device=codes.device)
    else:
        out = _out(out, (rows, outer), torch.bfloat16, codes, stream, name)
    fn = getattr(_lib or lib(), "bsq_" + name)
    raw = _raw_stream(stream, codes)
    if offsets is None:
        if batch != 1:
            raise ValueError(f"{name}: one weight is wanted, not {batch}")
        status = fn(codes.data_ptr(), scale.data_ptr(), rows, w.fmt, wd.data_ptr(), ws.data_ptr(), n, k, out.data_ptr(), raw)
    else:
        _dense(offsets, (torch.int32,), name)
        if offsets.numel() != batch or offsets.get_device() != dev:
            raise ValueError(f"{name}: {offsets.numel()} offsets on {offsets.device} for {batch} experts")
        status = fn(codes.data_ptr(), scale.data_ptr(), rows, w.fmt, wd.data_ptr(), ws.data_ptr(), batch, n, k,
                    offsets.data_ptr(), out.data_ptr(), raw)
    if status:
        _check(status)
    return out


def fp8_forward(x_codes, x_scale, w, out=None, stream=None):
    """y[M,N] (BF16) = X W^T of E4M3 operands: X from quantize_e4m3, W packed in 128x128 blocks."""
    return _fp8("fp8_forward", x_codes, x_scale, w, w.cols, w.rows, None, out, stream)


def fp8_dgrad(g_codes, g_scale, w, out=None, stream=None):
    """grad_x[M,K] (BF16) = G W of E4M3 operands: G = grad_out from quantize_e4m3."""
    return _fp8("fp8_dgrad", g_codes, g_scale, w, w.rows, w.cols, None, out, stream)


def fp8_grouped_forward(x_codes, x_scale, w, offsets, out=None, stream=None):
    """Per expert e: y[r0:r1] = X[r0:r1] W[e]^T; rows past offsets[-1] untouched."""
    return _fp8("fp8_grouped_forward", x_codes, x_scale, w, w.cols, w.rows, offsets, out, stream)


def fp8_grouped_dgrad(g_codes, g_scale, w, offsets, out=None, stream=None):
    """Per expert e: grad_x[r0:r1] = G[r0:r1] W[e]; rows past offsets[-1] untouched."""
    return _fp8("fp8_grouped_dgrad", g_codes, g_scale, w, w.rows, w.cols, offsets, out, stream)


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("param", _c_void_p), ("grad", _c_void_p), ("m", _c_void_p), ("v", _c_void_p), ("m_scale", _c_void_p),
                ("v_scale", _c_void_p), ("copy", _c_void_p), ("n", _i64), ("weight_decay", ctypes.c_float),
                ("counter", ctypes.c_uint32)]


# Whether tensors[i] still starts at addresses[i], for the given i.
_at_addresses = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal",
                        lambda tensors, addresses, which: all(tensors[i].data_ptr() == addresses[i] for i in which))


class AdamwTable:
    """The tensors of an optimizer, checked and laid out once, with the memory they had then.

    Moving or resharding a module gives its parameters other memory (``p.data = ...``), so every step
    compares the addresses of the parameters and their copies and refuses when one has changed
    (32 ns each on the GPU's host).  Gradients and states are taken where they were: they are to be
    written in place, and tensors that replace them (``zero_grad(set_to_none=True)``) need another
    table.  Their memory is held, whatever their owner does with them."""

    def __init__(self, items, grad_dtype, state_bits, keep):
        self.items, self.count, self.grad_dtype, self.state_bits, self.keep = items, len(items), grad_dtype, state_bits, keep
        self.address, self.like = ctypes.addressof(items), keep["params"][0] if keep["params"] else None
        self.watched = keep["params"] + keep.get("copies", [])
        self.addresses = [e.param or 0 for e in items] + ([e.copy or 0 for e in items] if "copies" in keep else [])
        self.places = list(range(len(self.watched)))
        self.held = [t.untyped_storage() for name, seq in keep.items() if name not in ("params", "copies", "weight_decay") for t in seq]

    def check(self):
        """Raises when a parameter or a copy is not where the table found it."""
        if not _at_addresses(self.watched, self.addresses, self.places):
            i = next(i for i in self.places if self.watched[i].data_ptr() != self.addresses[i])
            name, i = ("params", i) if i < self.count else ("copies", i - self.count)
            raise ValueError(f"adamw: {name}[{i}] has other memory than when the table was built; build another one")


def adamw_table(params, grads, ms, vs, m_scales=None, v_scales=None, copies=None, weight_decay=0.0):
    """The table `adamw` steps over.  params: float32; grads: all BF16 or all float32; states: float32,
    or uint8 E4M3 codes with scales of one float32 per 128 elements (new states: zero codes, any
    scale); copies: BF16 tensors that receive the updated parameters.  weight_decay: one number or
    one per tensor.  In the random sequence each tensor takes its length rounded up to 128."""
    n = len(params)
    s8 = m_scales is not None
    if (v_scales is not None) != s8:
        raise ValueError("adamw_table: m_scales and v_scales come together")
    decays = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * n
    lists = dict(params=list(params), grads=list(grads), ms=list(ms), vs=list(vs), weight_decay=decays)
    if s8:
        lists.update(m_scales=list(m_scales), v_scales=list(v_scales))
    if copies is not None:
        lists.update(copies=list(copies))
    for name, seq in lists.items():
        if len(seq) != n:
            raise ValueError(f"adamw_table: {len(seq)} {name} for {n} params")
    grad_dtype = grads[0].dtype if n else torch.float32
    if grad_dtype not in _DTYPES:
        raise ValueError(f"adamw_table: gradients of {grad_dtype}")
    wanted = dict(params=(torch.float32,), grads=(grad_dtype,), ms=(torch.uint8,) if s8 else (torch.float32,),
                  m_scales=(torch.float32,), copies=(torch.bfloat16,))
    wanted.update(vs=wanted["ms"], v_scales=wanted["m_scales"])
    items = (_AdamwTensor * n)()
    counter, dev = 0, params[0].get_device() if n else 0
    columns = [(name, seq, wanted[name], name.endswith("_scales")) for name, seq in lists.items() if name != "weight_decay"]
    for i in range(n):
        size = params[i].numel()
        blocks = -(-size // 128)
        for name, seq, dtypes, scales in columns:
            t = seq[i]
            if not (t.dtype in dtypes and t.get_device() == dev >= 0 and t.is_contiguous()
                    and t.numel() == (blocks if scales else size)):
                _dense(t, dtypes, f"adamw_table: {name}[{i}]")
                raise ValueError(f"adamw_table: {name}[{i}] holds {t.numel()} elements on {t.device}; params[{i}] has {size} "
                                 f"and params[0] is on {params[0].device}")
        p = lambda seq: None if seq is None else seq[i].data_ptr()
        items[i] = _AdamwTensor(p(params), p(grads), p(ms), p(vs), p(m_scales), p(v_scales), p(copies), size, decays[i],
                                counter & 0xFFFFFFFF)
        counter += 128 * blocks
    return AdamwTable(items, _DTYPES[grad_dtype], 8 if s8 else 32, lists)


def adamw(table, step, lr, betas=(0.9, 0.999), eps=1e-8, grad_scale=None, seed=0, stream=None):
    """One AdamW step over the tensors of `table`, in place; step counts from 1.  grad_scale: a device
    float32 that multiplies the gradients (clipping, loss scaling), or None.  step, lr and seed are
    the call's: a captured graph repeats them."""
    if grad_scale is not None:
        _dense(grad_scale, _F32, "adamw: grad_scale")
        if grad_scale.numel() != 1:
            raise ValueError("adamw: grad_scale is one number")
    if table.like is None:
        return
    dev = table.like.get_device()
    if dev != _current_device():
        _refuse_device("adamw", table.like)
    if grad_scale is not None and grad_scale.get_device() != dev:
        raise ValueError(f"adamw: grad_scale on {grad_scale.device}, the tensors are on {table.like.device}")
    table.check()
    _check(lib().bsq_adamw(table.address, table.count, table.grad_dtype, table.state_bits, step, lr, betas[0], betas[1], eps,
                           None if grad_scale is None else grad_scale.data_ptr(), seed & 0xFFFFFFFF,
                           _raw_stream(stream, table.like)))
