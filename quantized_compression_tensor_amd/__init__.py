"""Python binding of the C ABI declared in include/taco.h.

Argument marshalling only: every function below forwards to the function of
the same name in libtaco.so (hand-written gfx950 HIP kernels). Tensors may be
passed as torch tensors (their data_ptr is used) or as raw integer addresses;
the stream defaults to torch's current HIP stream. A nonzero status raises
TacoError. There is no fallback path: if the library cannot be built or
loaded, importing this package fails.
"""

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libtaco.so")

TACO_OK = 0
TACO_ERR_INVALID_ARG = -1
TACO_ERR_SHAPE = -2
TACO_ERR_FORMAT = -3
TACO_ERR_ALIGN = -4
TACO_ERR_WORKSPACE = -5
TACO_ERR_HIP = -6

TACO_FMT_FP8_DUAL = 1
TACO_FMT_INT8_SYM = 2
TACO_FMT_INT4_ASYM = 3
TACO_FMT_INT8_ASYM = 4
TACO_FMT_FP8E5_DUAL = 5
FP8_FORMATS = (TACO_FMT_FP8_DUAL, TACO_FMT_FP8E5_DUAL)

TACO_SCALE_AUTO = 0.0
TACO_SCALE_DELAYED = -1.0
TACO_MAX_SHARDS = 16
TACO_WORKSPACE_BYTES = 32768

TACO_F32 = 0
TACO_BF16 = 1
TACO_I8 = 2
TACO_NORM_MAX_COLS = 16384
TACO_ACT_NONE = 0
TACO_ACT_GELU = 1
TACO_ACT_SILU = 2
TACO_ACT_RELU = 3
TACO_LINEAR_MAX_DIM = 1 << 20
TACO_LINEAR_MAX_STRIDE = 1 << 21
TACO_INT8_MAX_K = 131071
TACO_MAX_GROUPS = 1024

# Entry points declared in include/taco.h (checked by the ABI tests).
EXPORTS = (
    "taco_layout", "taco_compressed_bytes", "taco_workspace_bytes", "taco_compress",
    "taco_compress_debug", "taco_decompress_reduce", "taco_ring_hop", "taco_requantize", "taco_decompress",
    "taco_e4m3_encode", "taco_e5m2_encode", "taco_status_string", "taco_compress_noalloc",
    "taco_set_launch_limit", "taco_chunk_order", "taco_compress_reordered", "taco_decompress_reordered",
    "taco_decompress_gemm", "taco_layer_norm", "taco_layer_norm_backward",
    "taco_layer_norm_backward_workspace_bytes", "taco_linear", "taco_linear_workspace_bytes", "taco_linear_backward",
    "taco_linear_backward_workspace_bytes", "taco_gated_linear", "taco_gated_linear_workspace_bytes",
    "taco_gated_linear_backward", "taco_gated_linear_backward_workspace_bytes",
    "taco_quantize_rows", "taco_linear_int8", "taco_linear_int8_workspace_bytes", "taco_gated_linear_int8",
    "taco_gated_linear_int8_workspace_bytes",
    "taco_grouped_linear", "taco_grouped_linear_workspace_bytes", "taco_grouped_linear_backward",
    "taco_grouped_linear_backward_workspace_bytes", "taco_grouped_gated_linear",
    "taco_grouped_gated_linear_workspace_bytes", "taco_grouped_gated_linear_backward",
    "taco_grouped_gated_linear_backward_workspace_bytes",
)


class taco_codec(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("block", ctypes.c_int32),
                ("hadamard", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def __repr__(self):
        return f"taco_codec(format={self.format}, block={self.block}, hadamard={self.hadamard})"


class taco_layout_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "codes_off", "codes_bytes", "scale_off", "scale_bytes", "aux_off", "aux_bytes",
        "tensor_off", "tensor_bytes", "total_bytes")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class taco_array(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def codec(fmt, block, hadamard=0):
    return taco_codec(int(fmt), int(block), int(hadamard), 0)


class TacoError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {taco_status_string(status)} ({status})")


def _load():
    # torch ships its own HIP runtime (same soname as /opt/rocm's). Loading it
    # first makes libtaco.so bind to that one runtime; loading libtaco.so first
    # would map a second runtime that does not know torch's streams or memory.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        from . import build as _build
        _build.build()
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    C, A = taco_codec, taco_array
    sig = {
        "taco_layout": (ctypes.c_int, [C, I64, I64, ctypes.POINTER(taco_layout_t)]),
        "taco_compressed_bytes": (I64, [C, I64, I64]),
        "taco_workspace_bytes": (SZ, [C, I64, I64]),
        "taco_compress": (ctypes.c_int, [C, P, I64, I64, F32, P, P, SZ, P]),
        "taco_compress_noalloc": (ctypes.c_int, [C, P, I64, I64, F32, P, P]),
        "taco_compress_debug": (ctypes.c_int, [C, P, I64, I64, F32, P, P, SZ, P, P]),
        "taco_decompress_reduce": (ctypes.c_int, [C, ctypes.POINTER(P), I32, I64, I64, P, C, P, P]),
        "taco_ring_hop": (ctypes.c_int, [C, P, P, I64, I64, P, C, P, P]),
        "taco_requantize": (ctypes.c_int, [C, P, I64, I64, F32, P, P, SZ, P]),
        "taco_decompress": (ctypes.c_int, [C, P, I64, I64, P, I32, P]),
        "taco_e4m3_encode": (ctypes.c_int, [P, P, I64, P]),
        "taco_e5m2_encode": (ctypes.c_int, [P, P, I64, P]),
        "taco_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "taco_set_launch_limit": (ctypes.c_int, [I32, ctypes.POINTER(I32)]),
        "taco_chunk_order": (ctypes.c_int, [P, I64, I64, P, P]),
        "taco_compress_reordered": (ctypes.c_int, [C, P, I64, I64, F32, P, P, SZ, P, P]),
        "taco_decompress_reordered": (ctypes.c_int, [C, P, I64, I64, P, I32, P, P]),
        "taco_decompress_gemm": (ctypes.c_int, [C, P, I64, I64, P, I64, P, I32, P]),
        "taco_layer_norm": (ctypes.c_int, [A, I64, I64, A, A, F32, A, P, P, P]),
        "taco_layer_norm_backward": (ctypes.c_int, [A, A, I64, I64, A, P, P, A, A, A, P, SZ, P]),
        "taco_layer_norm_backward_workspace_bytes": (SZ, [I64, I64]),
        "taco_linear": (ctypes.c_int, [A, A, A, I32, A, A, A, I64, I64, I64, P, SZ, P]),
        "taco_linear_backward": (ctypes.c_int, [A, A, A, I32, A, A, A, A, I64, I64, I64, P, SZ, P]),
        "taco_gated_linear": (ctypes.c_int, [A, A, I32, A, A, I64, I64, I64, P, SZ, P]),
        "taco_gated_linear_backward": (ctypes.c_int, [A, A, A, I32, A, A, A, I64, I64, I64, P, SZ, P]),
        "taco_quantize_rows": (ctypes.c_int, [A, I64, I64, A, P, P]),
        "taco_linear_int8": (ctypes.c_int, [A, P, A, P, A, I32, A, A, I64, I64, I64, P, SZ, P]),
        "taco_gated_linear_int8": (ctypes.c_int, [A, P, A, P, I32, A, I64, I64, I64, P, SZ, P]),
        "taco_grouped_linear": (ctypes.c_int, [A, A, A, I32, P, I32, A, A, I64, I64, I64, P, SZ, P]),
        "taco_grouped_linear_backward": (ctypes.c_int, [A, A, A, I32, A, P, I32, A, A, A, I64, I64, I64, P, SZ, P]),
        "taco_grouped_gated_linear": (ctypes.c_int, [A, A, I32, P, I32, A, A, I64, I64, I64, P, SZ, P]),
        "taco_grouped_gated_linear_backward": (ctypes.c_int, [A, A, A, I32, A, P, I32, A, A, I64, I64, I64, P, SZ, P]),
        **{f"taco_{n}_workspace_bytes": (SZ, [I64, I64, I64])
           for n in ("linear", "linear_backward", "gated_linear", "gated_linear_backward", "linear_int8",
                     "gated_linear_int8")},
        **{f"taco_grouped_{n}_workspace_bytes": (SZ, [I32, I64, I64, I64])
           for n in ("linear", "linear_backward", "gated_linear", "gated_linear_backward")},
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()
import torch  # noqa: E402  (loaded there)


def lib():
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _current_stream is None:
        _find_current_stream()
    return _current_stream() if _current_stream is not None else None


_current_stream = None   # gives the handle of torch's current stream, once torch has initialised the GPU


def _find_current_stream():
    """torch builds a Stream object for torch.cuda.current_stream() (about 3 us,
    as long as a launch); the plain handle is taken from the functions beneath
    where torch has them (0.1 us)."""
    import torch
    global _current_stream
    if not torch.cuda.is_initialized():
        return
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None:
        _current_stream = lambda: raw(device())   # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream   # noqa: E731


def _check(status, where):
    if status != TACO_OK:
        raise TacoError(status, where)
    return status


# ------------------------------------------------------------- host only --

def taco_status_string(status):
    return _lib.taco_status_string(int(status)).decode()


def taco_layout(c, rows, cols):
    L = taco_layout_t()
    _check(_lib.taco_layout(c, rows, cols, ctypes.byref(L)), "taco_layout")
    return L


def taco_compressed_bytes(c, rows, cols):
    n = _lib.taco_compressed_bytes(c, rows, cols)
    if n < 0:
        raise TacoError(int(n), "taco_compressed_bytes")
    return n


def taco_workspace_bytes(c, rows, cols):
    return _lib.taco_workspace_bytes(c, rows, cols)


def taco_set_launch_limit(max_workgroups):
    """Cap the workgroups of every later launch from this host thread (0 = no
    cap); returns the cap that was in force."""
    prev = ctypes.c_int32(0)
    _check(_lib.taco_set_launch_limit(int(max_workgroups), ctypes.byref(prev)), "taco_set_launch_limit")
    return prev.value


class launch_limit:
    """Context manager: ``with launch_limit(k): ...`` runs the block's calls on
    grids of at most k workgroups and restores the previous cap after."""

    def __init__(self, max_workgroups):
        self.k = max_workgroups

    def __enter__(self):
        self.prev = taco_set_launch_limit(self.k)
        return self

    def __exit__(self, *exc):
        taco_set_launch_limit(self.prev)
        return False


# ------------------------------------------------------------ device ops --

def taco_compress(c, x_bf16, rows, cols, tensor_scale, out, workspace=None, ws_bytes=None, stream=None):
    wsb = ws_bytes if ws_bytes is not None else (TACO_WORKSPACE_BYTES if workspace is not None else 0)
    return _check(_lib.taco_compress(c, _ptr(x_bf16), rows, cols, float(tensor_scale), _ptr(out),
                                     _ptr(workspace), wsb, _stream(stream)), "taco_compress")


def taco_compress_noalloc(c, x_bf16, rows, cols, tensor_scale, out, stream=None):
    return _check(_lib.taco_compress_noalloc(c, _ptr(x_bf16), rows, cols, float(tensor_scale), _ptr(out),
                                             _stream(stream)), "taco_compress_noalloc")


def taco_compress_debug(c, x_bf16, rows, cols, tensor_scale, out, prequant, workspace=None, ws_bytes=None,
                        stream=None):
    wsb = ws_bytes if ws_bytes is not None else (TACO_WORKSPACE_BYTES if workspace is not None else 0)
    return _check(_lib.taco_compress_debug(c, _ptr(x_bf16), rows, cols, float(tensor_scale), _ptr(out),
                                           _ptr(workspace), wsb, _ptr(prequant), _stream(stream)),
                  "taco_compress_debug")


def taco_decompress_reduce(c_in, shards, rows, cols, sum_fp32=None, c_out=None, requant_out=None, stream=None):
    arr = (ctypes.c_void_p * max(1, len(shards)))(*[_ptr(s) for s in shards])
    co = c_out if c_out is not None else taco_codec(0, 0, 0, 0)
    return _check(_lib.taco_decompress_reduce(c_in, arr, len(shards), rows, cols, _ptr(sum_fp32), co,
                                              _ptr(requant_out), _stream(stream)), "taco_decompress_reduce")


def taco_ring_hop(c_in, incoming, local_bf16, rows, cols, sum_fp32=None, c_out=None, requant_out=None,
                  stream=None):
    co = c_out if c_out is not None else taco_codec(0, 0, 0, 0)
    return _check(_lib.taco_ring_hop(c_in, _ptr(incoming), _ptr(local_bf16), rows, cols, _ptr(sum_fp32), co,
                                     _ptr(requant_out), _stream(stream)), "taco_ring_hop")


def taco_requantize(c_out, x_fp32, rows, cols, tensor_scale, out, workspace=None, ws_bytes=None, stream=None):
    wsb = ws_bytes if ws_bytes is not None else (TACO_WORKSPACE_BYTES if workspace is not None else 0)
    return _check(_lib.taco_requantize(c_out, _ptr(x_fp32), rows, cols, float(tensor_scale), _ptr(out),
                                       _ptr(workspace), wsb, _stream(stream)), "taco_requantize")


def taco_decompress(c, inp, rows, cols, out, out_dtype=0, stream=None):
    return _check(_lib.taco_decompress(c, _ptr(inp), rows, cols, _ptr(out), int(out_dtype), _stream(stream)),
                  "taco_decompress")


def taco_chunk_order(stats_bf16, rows, cols, order, stream=None):
    return _check(_lib.taco_chunk_order(_ptr(stats_bf16), rows, cols, _ptr(order), _stream(stream)),
                  "taco_chunk_order")


def taco_compress_reordered(c, x_bf16, rows, cols, tensor_scale, out, order, workspace=None, ws_bytes=None,
                            stream=None):
    wsb = ws_bytes if ws_bytes is not None else (TACO_WORKSPACE_BYTES if workspace is not None else 0)
    return _check(_lib.taco_compress_reordered(c, _ptr(x_bf16), rows, cols, float(tensor_scale), _ptr(out),
                                               _ptr(workspace), wsb, _ptr(order), _stream(stream)),
                  "taco_compress_reordered")


def taco_decompress_reordered(c, inp, rows, cols, out, order, out_dtype=0, stream=None):
    return _check(_lib.taco_decompress_reordered(c, _ptr(inp), rows, cols, _ptr(out), int(out_dtype), _ptr(order),
                                                 _stream(stream)), "taco_decompress_reordered")


def taco_decompress_gemm(c, a, M, K, w_bf16, N, out, out_dtype=0, stream=None):
    """out[M, N] = decode(a)[M, K] @ w_bf16[N, K]^T, the decode fused into the GEMM."""
    return _check(_lib.taco_decompress_gemm(c, _ptr(a), M, K, _ptr(w_bf16), N, _ptr(out), int(out_dtype),
                                            _stream(stream)), "taco_decompress_gemm")


def taco_e4m3_encode(x, codes, n, stream=None):
    return _check(_lib.taco_e4m3_encode(_ptr(x), _ptr(codes), n, _stream(stream)), "taco_e4m3_encode")


def taco_e5m2_encode(x, codes, n, stream=None):
    return _check(_lib.taco_e5m2_encode(_ptr(x), _ptr(codes), n, _stream(stream)), "taco_e5m2_encode")


# ---------------------------------------------------------------- layers --
# These take torch tensors: matrices [rows, cols] with unit column stride and
# any row stride, vectors [n]; sizes, strides and element types come from them.

_ABSENT = taco_array(None, 0, TACO_F32, 0)
_DTYPES = {}   # torch dtype -> TACO_F32 / TACO_BF16, filled on first use


def _dtype(t, what):
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: TACO_F32, torch.bfloat16: TACO_BF16})
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what}: {t.dtype} is neither float32 nor bfloat16")
    return dt


def _on_gpu(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what}: must be on the GPU")


def _matrix(t, rows, cols, what):
    if t is None:
        return _ABSENT
    if not t.is_cuda:
        _on_gpu(t, what)
    if t.shape != (rows, cols):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous (strides {t.stride()})")
    dt = _DTYPES.get(t.dtype)
    return taco_array(t.data_ptr(), stride, _dtype(t, what) if dt is None else dt, 0)


def _vector(t, n, what):
    if t is None:
        return _ABSENT
    if not t.is_cuda:
        _on_gpu(t, what)
    if t.shape != (n,):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {(n,)}")
    if n > 1 and not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    dt = _DTYPES.get(t.dtype)
    return taco_array(t.data_ptr(), n, _dtype(t, what) if dt is None else dt, 0)


def _floats(t, n, what):
    if t is None:
        return None
    if not t.is_cuda:
        _on_gpu(t, what)
    if t.shape != (n,) or (n > 1 and not t.is_contiguous()):
        raise ValueError(f"{what}: expected {n} contiguous values, got shape {tuple(t.shape)}")
    if _dtype(t, what) != TACO_F32:
        raise TypeError(f"{what}: must be float32")
    return t.data_ptr()


def _workspace(t):
    """Address and bytes of a workspace tensor."""
    if t is None:
        return None, 0
    _on_gpu(t, "workspace")
    if not t.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def taco_layer_norm(x, weight, bias, eps, y, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * weight + bias by row of x [rows, cols]; weight and
    bias [cols] or None; mean and rstd (float32 [rows]) are kept where given."""
    rows, cols = x.shape
    return _check(_lib.taco_layer_norm(_matrix(x, rows, cols, "x"), rows, cols, _vector(weight, cols, "weight"),
                                       _vector(bias, cols, "bias"), eps, _matrix(y, rows, cols, "y"),
                                       _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd"), _stream(stream)),
                  "taco_layer_norm")


def taco_layer_norm_backward_workspace_bytes(rows, cols):
    return _lib.taco_layer_norm_backward_workspace_bytes(rows, cols)


def taco_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None,
                             stream=None):
    """Gradients of taco_layer_norm, each where its tensor is given."""
    rows, cols = x.shape
    return _check(_lib.taco_layer_norm_backward(
        _matrix(dy, rows, cols, "dy"), _matrix(x, rows, cols, "x"), rows, cols, _vector(weight, cols, "weight"),
        _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd"), _matrix(dx, rows, cols, "dx"),
        _vector(dweight, cols, "dweight"), _vector(dbias, cols, "dbias"), *_workspace(workspace),
        _stream(stream)), "taco_layer_norm_backward")


def taco_linear_workspace_bytes(M, N, K):
    return _lib.taco_linear_workspace_bytes(M, N, K)


def taco_linear(x, w, out, bias=None, act=TACO_ACT_NONE, residual=None, preact=None, workspace=None, stream=None):
    """out = act(x w^T + bias) + residual; x bf16 [M, K], w bf16 [N, K]; preact,
    where given, receives x w^T + bias."""
    (M, K), N = x.shape, w.shape[0]
    return _check(_lib.taco_linear(
        _matrix(x, M, K, "x"), _matrix(w, N, K, "w"), _vector(bias, N, "bias"), act,
        _matrix(residual, M, N, "residual"), _matrix(out, M, N, "out"), _matrix(preact, M, N, "preact"), M, N, K,
        *_workspace(workspace), _stream(stream)), "taco_linear")


def taco_linear_backward_workspace_bytes(M, N, K):
    return _lib.taco_linear_backward_workspace_bytes(M, N, K)


def taco_linear_backward(dout, x, w, act=TACO_ACT_NONE, preact=None, dx=None, dw=None, dbias=None, workspace=None,
                         stream=None):
    """Gradients of taco_linear, each where its tensor is given."""
    (M, K), N = x.shape, w.shape[0]
    return _check(_lib.taco_linear_backward(
        _matrix(dout, M, N, "dout"), _matrix(x, M, K, "x"), _matrix(w, N, K, "w"), act,
        _matrix(preact, M, N, "preact"), _matrix(dx, M, K, "dx"), _matrix(dw, N, K, "dw"),
        _vector(dbias, N, "dbias"), M, N, K, *_workspace(workspace), _stream(stream)),
        "taco_linear_backward")


def taco_gated_linear_workspace_bytes(M, F, K):
    return _lib.taco_gated_linear_workspace_bytes(M, F, K)


def taco_gated_linear(x, w, out, act=TACO_ACT_SILU, preact=None, workspace=None, stream=None):
    """out = act(z[:, :F]) * z[:, F:] with z = x w^T; w bf16 [2 F, K], the gate's
    rows first; preact, where given, receives z."""
    (M, K), F = x.shape, w.shape[0] // 2
    return _check(_lib.taco_gated_linear(
        _matrix(x, M, K, "x"), _matrix(w, 2 * F, K, "w"), act, _matrix(out, M, F, "out"),
        _matrix(preact, M, 2 * F, "preact"), M, F, K, *_workspace(workspace), _stream(stream)),
        "taco_gated_linear")


def taco_gated_linear_backward_workspace_bytes(M, F, K):
    return _lib.taco_gated_linear_backward_workspace_bytes(M, F, K)


def taco_gated_linear_backward(dout, x, w, act=TACO_ACT_SILU, preact=None, dx=None, dw=None, workspace=None,
                               stream=None):
    """Gradients of taco_gated_linear, each where its tensor is given."""
    (M, K), F = x.shape, w.shape[0] // 2
    return _check(_lib.taco_gated_linear_backward(
        _matrix(dout, M, F, "dout"), _matrix(x, M, K, "x"), _matrix(w, 2 * F, K, "w"), act,
        _matrix(preact, M, 2 * F, "preact"), _matrix(dx, M, K, "dx"), _matrix(dw, 2 * F, K, "dw"), M, F, K,
        *_workspace(workspace), _stream(stream)), "taco_gated_linear_backward")


# ------------------------------------------------ projections in 8 bits --

def _codes(t, rows, cols, what):
    """An int8 matrix."""
    if not t.is_cuda:
        _on_gpu(t, what)
    if t.shape != (rows, cols):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous (strides {t.stride()})")
    if t.dtype is not torch.int8:
        raise TypeError(f"{what}: {t.dtype} is not int8")
    return taco_array(t.data_ptr(), stride, TACO_I8, 0)


def taco_quantize_rows(x, q, scale, stream=None):
    """q (int8 [rows, cols]) and scale (float32 [rows]) of the rows of x: scale =
    max |x| / 127, q = x * ((1 / max |x|) * 127) to the nearest."""
    rows, cols = x.shape
    return _check(_lib.taco_quantize_rows(_matrix(x, rows, cols, "x"), rows, cols, _codes(q, rows, cols, "q"),
                                          _floats(scale, rows, "scale"), _stream(stream)), "taco_quantize_rows")


def taco_linear_int8_workspace_bytes(M, N, K):
    return _lib.taco_linear_int8_workspace_bytes(M, N, K)


def taco_linear_int8(x, x_scale, w, w_scale, out, bias=None, act=TACO_ACT_NONE, residual=None, workspace=None,
                     stream=None):
    """out = act((x w^T) x_scale w_scale + bias) + residual; x int8 [M, K], w int8
    [N, K], x_scale float32 [M], w_scale float32 [N]."""
    (M, K), N = x.shape, w.shape[0]
    return _check(_lib.taco_linear_int8(
        _codes(x, M, K, "x"), _floats(x_scale, M, "x_scale"), _codes(w, N, K, "w"), _floats(w_scale, N, "w_scale"),
        _vector(bias, N, "bias"), act, _matrix(residual, M, N, "residual"), _matrix(out, M, N, "out"), M, N, K,
        *_workspace(workspace), _stream(stream)), "taco_linear_int8")


def taco_gated_linear_int8_workspace_bytes(M, F, K):
    return _lib.taco_gated_linear_int8_workspace_bytes(M, F, K)


def taco_gated_linear_int8(x, x_scale, w, w_scale, out, act=TACO_ACT_SILU, workspace=None, stream=None):
    """out = act(z[:, :F]) * z[:, F:] with z = (x w^T) x_scale w_scale; w int8
    [2 F, K], the gate's rows first, w_scale float32 [2 F]."""
    (M, K), F = x.shape, w.shape[0] // 2
    return _check(_lib.taco_gated_linear_int8(
        _codes(x, M, K, "x"), _floats(x_scale, M, "x_scale"), _codes(w, 2 * F, K, "w"),
        _floats(w_scale, 2 * F, "w_scale"), act, _matrix(out, M, F, "out"), M, F, K, *_workspace(workspace),
        _stream(stream)), "taco_gated_linear_int8")


# ------------------------------------------------- projections by group --
# Weights are [groups, rows, K] tensors, a group's matrix right after another's
# (any row stride); offsets int32 [groups + 1] on the GPU.

def _groups_of(t, groups, rows, cols, what):
    """A [groups, rows, cols] tensor as the matrix [groups * rows, cols]."""
    if t is None:
        return _ABSENT
    if not t.is_cuda:
        _on_gpu(t, what)
    if t.shape != (groups, rows, cols):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {(groups, rows, cols)}")
    apart, stride, inner = t.stride()
    if rows == 1:
        stride = apart
    if (inner != 1 and cols > 1) or (groups > 1 and apart != rows * stride):
        raise ValueError(f"{what}: rows must be contiguous and evenly spaced over all groups (strides {t.stride()})")
    dt = _DTYPES.get(t.dtype)
    return taco_array(t.data_ptr(), stride, _dtype(t, what) if dt is None else dt, 0)


def _offsets(t, groups):
    if not t.is_cuda:
        _on_gpu(t, "offsets")
    if t.shape != (groups + 1,) or not t.is_contiguous():
        raise ValueError(f"offsets: expected {groups + 1} contiguous values, got shape {tuple(t.shape)}")
    if t.dtype is not torch.int32:
        raise TypeError(f"offsets: {t.dtype} is not int32")
    return t.data_ptr()


def taco_grouped_linear_workspace_bytes(groups, M, N, K):
    return _lib.taco_grouped_linear_workspace_bytes(groups, M, N, K)


def taco_grouped_linear(x, w, offsets, out, bias=None, act=TACO_ACT_NONE, preact=None, workspace=None, stream=None):
    """out = act(x w[g]^T + bias[g]) for the rows offsets[g] ... offsets[g + 1] of
    x [M, K]; w bf16 [groups, N, K], bias [groups, N]; preact receives what act is
    taken of. Rows of no group stay as they are."""
    (M, K), (G, N, _) = x.shape, w.shape
    return _check(_lib.taco_grouped_linear(
        _matrix(x, M, K, "x"), _groups_of(w, G, N, K, "w"), _matrix(bias, G, N, "bias"), act, _offsets(offsets, G), G,
        _matrix(out, M, N, "out"), _matrix(preact, M, N, "preact"), M, N, K, *_workspace(workspace), _stream(stream)),
        "taco_grouped_linear")


def taco_grouped_linear_backward_workspace_bytes(groups, M, N, K):
    return _lib.taco_grouped_linear_backward_workspace_bytes(groups, M, N, K)


def taco_grouped_linear_backward(dout, x, w, offsets, act=TACO_ACT_NONE, preact=None, dx=None, dw=None, dbias=None,
                                 workspace=None, stream=None):
    """Gradients of taco_grouped_linear, each where its tensor is given."""
    (M, K), (G, N, _) = x.shape, w.shape
    return _check(_lib.taco_grouped_linear_backward(
        _matrix(dout, M, N, "dout"), _matrix(x, M, K, "x"), _groups_of(w, G, N, K, "w"), act,
        _matrix(preact, M, N, "preact"), _offsets(offsets, G), G, _matrix(dx, M, K, "dx"),
        _groups_of(dw, G, N, K, "dw"), _matrix(dbias, G, N, "dbias"), M, N, K, *_workspace(workspace),
        _stream(stream)), "taco_grouped_linear_backward")


def taco_grouped_gated_linear_workspace_bytes(groups, M, F, K):
    return _lib.taco_grouped_gated_linear_workspace_bytes(groups, M, F, K)


def taco_grouped_gated_linear(x, w, offsets, out, act=TACO_ACT_SILU, preact=None, workspace=None, stream=None):
    """out = act(z[:, :F]) * z[:, F:] with z = x w[g]^T for the rows of group g; w
    bf16 [groups, 2 F, K], of each group the gate's rows first; preact receives z."""
    (M, K), G, F = x.shape, w.shape[0], w.shape[1] // 2
    return _check(_lib.taco_grouped_gated_linear(
        _matrix(x, M, K, "x"), _groups_of(w, G, 2 * F, K, "w"), act, _offsets(offsets, G), G,
        _matrix(out, M, F, "out"), _matrix(preact, M, 2 * F, "preact"), M, F, K, *_workspace(workspace),
        _stream(stream)), "taco_grouped_gated_linear")


def taco_grouped_gated_linear_backward_workspace_bytes(groups, M, F, K):
    return _lib.taco_grouped_gated_linear_backward_workspace_bytes(groups, M, F, K)


def taco_grouped_gated_linear_backward(dout, x, w, offsets, act=TACO_ACT_SILU, preact=None, dx=None, dw=None,
                                       workspace=None, stream=None):
    """Gradients of taco_grouped_gated_linear, each where its tensor is given."""
    (M, K), G, F = x.shape, w.shape[0], w.shape[1] // 2
    return _check(_lib.taco_grouped_gated_linear_backward(
        _matrix(dout, M, F, "dout"), _matrix(x, M, K, "x"), _groups_of(w, G, 2 * F, K, "w"), act,
        _matrix(preact, M, 2 * F, "preact"), _offsets(offsets, G), G, _matrix(dx, M, K, "dx"),
        _groups_of(dw, G, 2 * F, K, "dw"), M, F, K, *_workspace(workspace), _stream(stream)),
        "taco_grouped_gated_linear_backward")


# ------------------------------------------------- buffer plumbing (torch) --

def empty_compressed(c, rows, cols, device="cuda"):
    """A uint8 device tensor sized for one compressed [rows, cols] tensor."""
    import torch
    return torch.empty(max(1, taco_compressed_bytes(c, rows, cols)), dtype=torch.uint8, device=device)


def regions(buf, c, rows, cols):
    """Views of a compressed buffer's regions (codes, scale, aux, tensor), as laid
    out by taco_layout: codes uint8; scale int8 (FP8) or float32; aux uint8;
    tensor float32[4] (FP8) -- for tests and inspection."""
    import torch
    L = taco_layout(c, rows, cols)
    codes = buf[L.codes_off:L.codes_off + L.codes_bytes]
    sc = buf[L.scale_off:L.scale_off + L.scale_bytes]
    sc = sc.view(torch.int8) if c.format in FP8_FORMATS else sc.view(torch.float32)
    aux = buf[L.aux_off:L.aux_off + L.aux_bytes]
    ten = buf[L.tensor_off:L.tensor_off + L.tensor_bytes].view(torch.float32)
    return codes, sc, aux, ten


WS_TICKET_GROUPS = 64   # workspace ticket counters (kernel-side constants)
WS_BANK_LINES = 32      # workspace record lines per bank (three banks)
WS_LINE = 32            # uint32 words per 128-byte line
WS_SHARE_SHIFT = 24     # each call adds 2^24 to every ticket counter


def workspace_history(ws):
    """Read an FP8 tensor-scale workspace (a device tensor of
    TACO_WORKSPACE_BYTES) between calls: returns (calls made, abs-max recorded
    by the most recent call, that call's bank). Layout (uint32 words, 32 per
    line): line 0 unused; line 1 + g, words 0-1: ticket counter g (64, uint64);
    line 65 + 32 b + l, word 0: record line l of bank b (3 banks of 32).
    Inspection only."""
    import numpy as np
    w = ws.detach().cpu().numpy().view(np.uint32).reshape(-1)
    calls = int(w[WS_LINE:WS_LINE + 2].view(np.uint64)[0]) >> WS_SHARE_SHIFT
    if calls == 0:
        return 0, 0.0, None
    bank = (calls - 1) % 3
    amax = bank_lines(w)[bank].copy().view(np.float32).max()
    return calls, float(amax), bank


def bank_lines(words):
    """The record words of a workspace given as uint32 words: [3 banks, 32 lines]."""
    base = WS_LINE * (1 + WS_TICKET_GROUPS)
    return words[base: base + WS_LINE * 3 * WS_BANK_LINES].reshape(3, WS_BANK_LINES, WS_LINE)[:, :, 0]
