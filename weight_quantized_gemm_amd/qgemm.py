"""Thin Python binding of libqgemm's C ABI (include/qgemm.h).

Same names as the C entry points; this module only marshals arguments
(numpy arrays for the host-side quantiser and packer, torch tensors for
device buffers, torch's current HIP stream). Every step of the GEMM runs in
the library's HIP kernels. There is no fallback: if libqgemm.so is missing or
a call fails, an exception is raised.

torch is imported before the library is loaded so that the process uses one
HIP runtime (torch's), which the library then binds to by its soname.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

import torch  # noqa: F401  (must be loaded before libqgemm.so; see module doc)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemm.so")

# Format ids (0-3: the MNN GemmSpeed page's mode numbers; 4: fp16 weights;
# 5: Int4-Block0 with fp16 activations; 6, 8: MXFP4 weights with fp16 / MXFP4
# activations) and names.
QGEMM_F32, QGEMM_INT4_B64, QGEMM_INT8_B0, QGEMM_W4A8, QGEMM_F16, QGEMM_INT4_B0 = 0, 1, 2, 3, 4, 5
QGEMM_MXFP4, QGEMM_MXFP4_A4 = 6, 8
FORMATS = {"f32": QGEMM_F32, "int4b64": QGEMM_INT4_B64, "int8b0": QGEMM_INT8_B0,
           "w4a8": QGEMM_W4A8, "f16": QGEMM_F16, "int4b0": QGEMM_INT4_B0,
           "mxfp4": QGEMM_MXFP4, "mxfp4a4": QGEMM_MXFP4_A4}

STATUS = {0: "QGEMM_OK", 1: "QGEMM_ERR_NULL", 2: "QGEMM_ERR_SHAPE", 3: "QGEMM_ERR_FORMAT",
          4: "QGEMM_ERR_ALIGN", 5: "QGEMM_ERR_NOMEM", 6: "QGEMM_ERR_DEVICE",
          7: "QGEMM_ERR_LAUNCH", 8: "QGEMM_ERR_SIZE", 9: "QGEMM_ERR_VALUE"}

# Every symbol include/qgemm.h declares.
EXPORTS = ["qgemm_status_string", "qgemm_abi_version", "qgemm_canonical_size",
           "qgemm_quantize_weights", "qgemm_packed_size", "qgemm_pack_weights",
           "qgemm_unpack_weights", "qgemm_workspace_size", "qgemm_run", "qgemm_run_ws",
           "qgemm_run_ex", "qgemm_run_noalloc", "qgemm_w4a8_debug", "qgemm_set_gemv_max_m",
           "qgemm_quantize_weights_device", "qgemm_quantize_pack_device",
           "qgemm_mx_quantize", "qgemm_mx_quantize_device", "qgemm_mx_dequantize_device",
           "qgemm_mx_pack", "qgemm_mx_pack_device", "qgemm_group_plan_size", "qgemm_group_plan",
           "qgemm_grouped_workspace_size", "qgemm_run_grouped", "qgemm_group_combine"]


class QGemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libqgemm.so; raises if it has not been built."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m weight_quantized_gemm_amd.build_lib` "
            "(there is no fallback path)")
    lib = ctypes.CDLL(path)
    P, I, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
    ZP = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "qgemm_status_string": ([I], ctypes.c_char_p),
        "qgemm_abi_version": ([], I),
        "qgemm_canonical_size": ([I, I, I, ZP, ZP], I),
        "qgemm_quantize_weights": ([I, I, I, P, P, Z, P, Z], I),
        "qgemm_packed_size": ([I, I, I, ZP, ZP], I),
        "qgemm_pack_weights": ([I, I, I, P, P, P, Z, P, Z], I),
        "qgemm_unpack_weights": ([I, I, I, P, Z, P, Z, P, P], I),
        "qgemm_workspace_size": ([I, I, I, I, ZP], I),
        "qgemm_run": ([I, I, I, I, P, P, P, P, P], I),
        "qgemm_run_ws": ([I, I, I, I, P, P, P, P, P, Z, P], I),
        "qgemm_run_ex": ([I, I, I, I, P, P, P, P, ctypes.POINTER(Epilogue), P, Z, P], I),
        "qgemm_run_noalloc": ([I, I, I, I, P, P, P, P, ctypes.POINTER(Epilogue), P], I),
        "qgemm_w4a8_debug": ([I, I, I, P, P, P, P, P, P, P, P, P, Z, P], I),
        "qgemm_set_gemv_max_m": ([I], I),
        "qgemm_quantize_weights_device": ([I, I, I, P, P, P, P], I),
        "qgemm_quantize_pack_device": ([I, I, I, P, P, P, P], I),
        "qgemm_mx_quantize": ([I, I, P, P, P], I),
        "qgemm_mx_quantize_device": ([I, I, I, P, L, P, P, P], I),
        "qgemm_mx_dequantize_device": ([I, I, P, P, I, P, L, P], I),
        "qgemm_mx_pack": ([I, I, P, P, P, Z, P, Z], I),
        "qgemm_mx_pack_device": ([I, I, I, P, P, P, P, P], I),
        "qgemm_group_plan_size": ([I, I, I, ZP], I),
        "qgemm_group_plan": ([I, I, I, P, I, P, P, P, P, Z, P], I),
        "qgemm_grouped_workspace_size": ([I, I, I, I, I, I, ZP], I),
        "qgemm_run_grouped": ([I, I, I, I, I, I, P, P, P, P, P, P, ctypes.POINTER(Epilogue), P, Z, P], I),
        "qgemm_group_combine": ([I, I, I, I, P, I, P, P, P, I, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path == LIB_PATH:
        _lib = lib
    return lib


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
OUT_TYPES = {"f32": 0, "f16": 1}


class Epilogue(ctypes.Structure):
    """Mirror of qgemm_epilogue: C = act(A x B + bias + residual), C fp32 or fp16."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("activation", ctypes.c_int), ("out_type", ctypes.c_int)]


QGEMM_INT4_BLOCK_BASE = 0x10000
QGEMM_INT8_BLOCK_BASE = 0x2000000


def QGEMM_INT4_BLOCK(b: int) -> int:
    """Format id of Int4 weights with one pair per b K-elements."""
    return QGEMM_INT4_BLOCK_BASE + b


def QGEMM_INT8_BLOCK(b: int) -> int:
    """Format id of Int8 weights with one pair per b K-elements."""
    return QGEMM_INT8_BLOCK_BASE + b


def _fmt(f) -> int:
    """Format id from a name ("int4b64", "int8b0", ..., "int4b<b>" / "int8b<b>"
    for any other Int4 / Int8 block size b) or an id."""
    if not isinstance(f, str):
        return int(f)
    if f in FORMATS:
        return FORMATS[f]
    if f.startswith("int4b") and f[5:].isdigit():
        return QGEMM_INT4_BLOCK(int(f[5:]))
    if f.startswith("int8b") and f[5:].isdigit() and int(f[5:]) > 0:
        return QGEMM_INT8_BLOCK(int(f[5:]))
    raise ValueError(f"unknown format {f}")


def is_int8(fmt) -> bool:
    """Whether a format stores one byte per code (Int8-Block0 and blocked Int8)."""
    f = _fmt(fmt)
    return f == QGEMM_INT8_B0 or f > QGEMM_INT8_BLOCK_BASE


def pairs_per_channel(fmt, K: int) -> int:
    """Canonical pairs per channel of a quantised format."""
    f = _fmt(fmt)
    if f == QGEMM_INT4_B64:
        return K // 64
    if f > QGEMM_INT8_BLOCK_BASE:
        return K // (f - QGEMM_INT8_BLOCK_BASE)
    if f > QGEMM_INT4_BLOCK_BASE:
        return K // (f - QGEMM_INT4_BLOCK_BASE)
    return 1


def _check(st: int, where: str):
    if st != 0:
        raise QGemmError(st, where)


def _np_ptr(a: np.ndarray | None):
    if a is None:
        return None
    assert a.flags["C_CONTIGUOUS"]
    return a.ctypes.data_as(ctypes.c_void_p)


def _dev_ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("device buffers must be contiguous GPU tensors")
    return t.data_ptr()


_TORCH_DTYPE_NAMES = {torch.float32: "float32", torch.float16: "float16", torch.uint8: "uint8",
                      torch.int8: "int8", torch.int32: "int32"}


def _need(t, name: str, dtypes, numel: int | None = None, nbytes: int | None = None):
    """Checks a device-buffer argument before anything reaches the library:
    its dtype (one of `dtypes`, or any when None), at least `numel` elements
    and at least `nbytes` bytes. Raw integer addresses and None pass through
    (the C side checks for NULL). Raises ValueError. The kernels would
    otherwise read or write past a buffer that is too small or of the wrong
    element type."""
    if t is None or isinstance(t, int):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch tensor or a device address, got {type(t).__name__}")
    n = t.numel()
    if n == 0 and not numel and not nbytes:
        return   # an empty placeholder for an operand the shape never reads
    if (dtypes is None or t.dtype in dtypes) and (numel is None or n >= numel) and \
            (nbytes is None or n * t.element_size() >= nbytes):
        return
    if dtypes is not None and t.dtype not in dtypes:
        want = " or ".join(_TORCH_DTYPE_NAMES.get(d, str(d)) for d in dtypes)
        raise ValueError(f"{name}: dtype {t.dtype} where {want} is required")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {numel} required")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, at least {nbytes} required")


def _check_run_args(M: int, K: int, N: int, fmt, A, Bq, scales, C, out_type=0, bias=None,
                    residual=None, workspace=None, ws_bytes: int = 0):
    """Dtype and size checks shared by the run entry points: A fp32 for the
    fp32 format, fp16 otherwise, [M][K]; C (and the residual) fp32, or fp16
    with the fp16 output; the packed buffers at least the packed sizes of
    (K, N, fmt); the bias [N] fp32; the workspace at least ws_bytes."""
    f = _fmt(fmt)
    if M < 0 or N < 0 or K < 0:
        raise ValueError(f"negative shape M={M} K={K} N={N}")
    if M == 0 or N == 0:
        return
    a_dt = torch.float32 if f == QGEMM_F32 else torch.float16
    _need(A, "A", (a_dt,), numel=M * K)
    c_dt = torch.float16 if out_type in (1, "f16") else torch.float32
    _need(C, "C", (c_dt,), numel=M * N)
    _need(residual, "residual", (c_dt,), numel=M * N)
    _need(bias, "bias", (torch.float32,), numel=N)
    try:
        wb, sb = qgemm_packed_size(K, N, f)
    except QGemmError:
        wb = sb = None   # the library reports the bad shape or format itself
    if f == QGEMM_F32 and wb is not None:
        # the fp32 format's B is the float [K][N] matrix itself, read no
        # further than its K*N elements (the packed size rounds it up to 256)
        wb = K * N * 4
    _need(Bq, "Bq", None, nbytes=wb)
    _need(scales, "scales", None, nbytes=sb)
    if isinstance(workspace, torch.Tensor) and workspace.numel() * workspace.element_size() < ws_bytes:
        raise ValueError(f"workspace: {workspace.numel() * workspace.element_size()} bytes, "
                         f"ws_bytes={ws_bytes} claimed")


# The current stream's handle without building a Stream object for every call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------------------
def qgemm_status_string(status: int) -> str:
    return load().qgemm_status_string(status).decode()


def qgemm_abi_version() -> int:
    return load().qgemm_abi_version()


def qgemm_canonical_size(K: int, N: int, fmt) -> tuple[int, int]:
    q, p = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qgemm_canonical_size(K, N, _fmt(fmt), ctypes.byref(q), ctypes.byref(p)),
           "qgemm_canonical_size")
    return q.value, p.value


@functools.lru_cache(maxsize=4096)
def qgemm_packed_size(K: int, N: int, fmt) -> tuple[int, int]:
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qgemm_packed_size(K, N, _fmt(fmt), ctypes.byref(w), ctypes.byref(s)),
           "qgemm_packed_size")
    return w.value, s.value


def qgemm_workspace_size(M: int, K: int, N: int, fmt) -> int:
    b = ctypes.c_size_t()
    _check(load().qgemm_workspace_size(M, K, N, _fmt(fmt), ctypes.byref(b)),
           "qgemm_workspace_size")
    return b.value


def qgemm_quantize_weights(W: np.ndarray, fmt):
    """Float W [N][K] -> (canonical codes uint8, pairs float32 [N][nblk][2])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    qb, pf = qgemm_canonical_size(K, N, fmt)
    q = np.empty(qb, dtype=np.uint8)
    pairs = np.empty(pf, dtype=np.float32)
    _check(load().qgemm_quantize_weights(K, N, _fmt(fmt), _np_ptr(W), _np_ptr(q), qb,
                                         _np_ptr(pairs), pf), "qgemm_quantize_weights")
    f = _fmt(fmt)
    qshape = (N, K) if is_int8(f) else (N, K // 2)
    return q.reshape(qshape), pairs.reshape(N, pairs_per_channel(f, K), 2)


def qgemm_pack_weights(K: int, N: int, fmt, w_canonical: np.ndarray,
                       pairs_canonical: np.ndarray | None):
    """Canonical host arrays -> (packed weights uint8, packed pairs uint8), host."""
    wb, sb = qgemm_packed_size(K, N, fmt)
    wp = np.empty(wb, dtype=np.uint8)
    sp = np.empty(max(sb, 1), dtype=np.uint8)
    wc = np.ascontiguousarray(w_canonical)
    pc = None if pairs_canonical is None else np.ascontiguousarray(pairs_canonical, dtype=np.float32)
    _check(load().qgemm_pack_weights(K, N, _fmt(fmt), _np_ptr(wc), _np_ptr(pc), _np_ptr(wp), wb,
                                     _np_ptr(sp), sb), "qgemm_pack_weights")
    return wp, sp[:sb]


def qgemm_unpack_weights(K: int, N: int, fmt, w_packed: np.ndarray, s_packed: np.ndarray):
    f = _fmt(fmt)
    qb, pf = qgemm_canonical_size(K, N, f)
    q = np.empty(max(qb, 1), dtype=np.uint8)
    pairs = np.empty(max(pf, 1), dtype=np.float32)
    sp = s_packed if s_packed.size else np.zeros(1, np.uint8)
    _check(load().qgemm_unpack_weights(K, N, f, _np_ptr(w_packed), w_packed.nbytes, _np_ptr(sp),
                                       s_packed.nbytes, _np_ptr(q), _np_ptr(pairs)),
           "qgemm_unpack_weights")
    return q[:qb], pairs[:pf]


def qgemm_run(M: int, K: int, N: int, fmt, A, Bq, scales, C, stream=None) -> None:
    """C = A x B on the GPU (torch tensors or raw device addresses)."""
    _check_run_args(M, K, N, fmt, A, Bq, scales, C)
    _check(load().qgemm_run(M, K, N, _fmt(fmt), _dev_ptr(A), _dev_ptr(Bq), _dev_ptr(scales),
                            _dev_ptr(C), _stream(stream)), "qgemm_run")


def qgemm_run_ws(M: int, K: int, N: int, fmt, A, Bq, scales, C, workspace, ws_bytes: int,
                 stream=None) -> None:
    _check_run_args(M, K, N, fmt, A, Bq, scales, C, workspace=workspace, ws_bytes=ws_bytes)
    _check(load().qgemm_run_ws(M, K, N, _fmt(fmt), _dev_ptr(A), _dev_ptr(Bq), _dev_ptr(scales),
                               _dev_ptr(C), _dev_ptr(workspace), ws_bytes, _stream(stream)),
           "qgemm_run_ws")


def qgemm_run_ex(M: int, K: int, N: int, fmt, A, Bq, scales, C, bias=None, residual=None,
                 activation="none", out_type="f32", workspace=None, ws_bytes: int = 0,
                 stream=None) -> None:
    """C = act(A x B + bias + residual) on the GPU; C (and residual) fp32 or fp16
    per out_type. With no workspace the library allocates any scratch the shape
    needs in stream order."""
    _check_run_args(M, K, N, fmt, A, Bq, scales, C, out_type=out_type, bias=bias,
                    residual=residual, workspace=workspace, ws_bytes=ws_bytes)
    epi = Epilogue(_dev_ptr(bias), _dev_ptr(residual),
                   ACTIVATIONS[activation] if isinstance(activation, str) else int(activation),
                   OUT_TYPES[out_type] if isinstance(out_type, str) else int(out_type))
    _check(load().qgemm_run_ex(M, K, N, _fmt(fmt), _dev_ptr(A), _dev_ptr(Bq), _dev_ptr(scales),
                               _dev_ptr(C), ctypes.byref(epi), _dev_ptr(workspace), ws_bytes,
                               _stream(stream)), "qgemm_run_ex")


NOALLOC_SCRATCH_BYTES = 32 << 20   # QGEMM_NOALLOC_SCRATCH_BYTES


def qgemm_run_noalloc(M: int, K: int, N: int, fmt, A, Bq, scales, C, bias=None, residual=None,
                      activation="none", out_type="f32", stream=None) -> None:
    """qgemm_run_ex without any allocation: the scratch the shape needs lives in
    the library's fixed per-GPU array (NOALLOC_SCRATCH_BYTES); calls that may
    overlap on one GPU must be serialised by the caller."""
    _check_run_args(M, K, N, fmt, A, Bq, scales, C, out_type=out_type, bias=bias,
                    residual=residual)
    epi = Epilogue(_dev_ptr(bias), _dev_ptr(residual),
                   ACTIVATIONS[activation] if isinstance(activation, str) else int(activation),
                   OUT_TYPES[out_type] if isinstance(out_type, str) else int(out_type))
    _check(load().qgemm_run_noalloc(M, K, N, _fmt(fmt), _dev_ptr(A), _dev_ptr(Bq), _dev_ptr(scales),
                                    _dev_ptr(C), ctypes.byref(epi), _stream(stream)),
           "qgemm_run_noalloc")


def qgemm_w4a8_debug(M: int, K: int, N: int, A, Bq, scales, C, qa, sa, S, D, workspace,
                     ws_bytes: int, stream=None) -> None:
    _check_run_args(M, K, N, QGEMM_W4A8, A, Bq, scales, C, workspace=workspace, ws_bytes=ws_bytes)
    _need(qa, "qa", (torch.int8, torch.uint8), numel=M * K)
    _need(sa, "sa", (torch.float32,), numel=M)
    _need(S, "S", (torch.int32,), numel=M)
    _need(D, "D", (torch.int32,), numel=M * N)
    _check(load().qgemm_w4a8_debug(M, K, N, _dev_ptr(A), _dev_ptr(Bq), _dev_ptr(scales),
                                   _dev_ptr(C), _dev_ptr(qa), _dev_ptr(sa), _dev_ptr(S),
                                   _dev_ptr(D), _dev_ptr(workspace), ws_bytes, _stream(stream)),
           "qgemm_w4a8_debug")


def qgemm_quantize_weights_device(W, fmt, q=None, pairs=None, stream=None):
    """Device float W [N][K] -> (canonical codes uint8, pairs float32 [N][nblk][2]),
    both device tensors (allocated here unless given)."""
    f = _fmt(fmt)
    N, K = W.shape
    qb, pf = qgemm_canonical_size(K, N, f)
    if q is None:
        q = torch.empty(max(qb, 1), dtype=torch.uint8, device=W.device)
    if pairs is None:
        pairs = torch.empty(max(pf, 1), dtype=torch.float32, device=W.device)
    _check(load().qgemm_quantize_weights_device(K, N, f, _dev_ptr(W), _dev_ptr(q), _dev_ptr(pairs),
                                                _stream(stream)), "qgemm_quantize_weights_device")
    qshape = (N, K) if is_int8(f) else (N, K // 2)
    return q[:qb].view(qshape), pairs[:pf].view(N, pairs_per_channel(f, K), 2)


def qgemm_quantize_pack_device(W, fmt, Bq=None, scales=None, stream=None):
    """Device float W [N][K] -> (packed weights uint8, packed pairs uint8), both
    device tensors in the layout qgemm_run reads."""
    f = _fmt(fmt)
    N, K = W.shape
    wb, sb = qgemm_packed_size(K, N, f)
    if Bq is None:
        Bq = torch.empty(wb, dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty(sb, dtype=torch.uint8, device=W.device)
    _check(load().qgemm_quantize_pack_device(K, N, f, _dev_ptr(W), _dev_ptr(Bq), _dev_ptr(scales),
                                             _stream(stream)), "qgemm_quantize_pack_device")
    return Bq, scales


def qgemm_set_gemv_max_m(max_m: int) -> int:
    return load().qgemm_set_gemv_max_m(max_m)


# ---------------------------------------------------------------------------
# MXFP4 conversions and mixture of experts. These take torch tensors only: the
# sizes come from their shapes, and the call runs on the tensors' own device
# (on its current stream unless one is given).
# ---------------------------------------------------------------------------
TYPES = {"f32": 0, "f16": 1, "bf16": 2}                  # qgemm_type
_TORCH_TYPES = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}
_TYPE_IDS = {d: t for t, d in _TORCH_TYPES.items()}


def _same_device(**tensors):
    """Checks that the tensors (None passes) are GPU tensors of one device and
    returns it."""
    first, index = None, -1
    for name, t in tensors.items():
        if t is None:
            continue
        i = t.get_device() if isinstance(t, torch.Tensor) else -1      # -1: on the host
        if i == index >= 0:
            continue
        if i < 0:
            raise ValueError(f"{name}: expected a GPU tensor")
        if first is not None:
            raise ValueError(f"{name}: on {t.device}, the other tensors on {first.device}")
        first, index = t, i
    return None if first is None else first.device


def _exact(t, name: str, dtypes, shape):
    """Checks a tensor's dtype, shape and contiguity."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        want = " or ".join(_TORCH_DTYPE_NAMES.get(d, str(d)) for d in dtypes)
        raise ValueError(f"{name}: dtype {t.dtype} where {want} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _call(name: str, dev, stream, *args):
    """Calls an entry point whose last argument is the stream, with `dev` as the
    current device."""
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return _call(name, dev, stream, *args)
    if stream is None:
        handle = _raw_stream(dev.index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    status = getattr(load(), name)(*args, handle)
    if status:
        raise QGemmError(status, name)


def _empty(shape, dtype, dev, stream):
    """A new tensor for a call on `stream` (None: the current one). Its memory
    belongs to that stream: memory of the current one may still be in use by
    work queued there, which a call on another stream does not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _row_stride(t, name: str) -> int:
    """Row stride of a [R][K] tensor whose rows are contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name}: expected [R][K] with contiguous, ascending rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def qgemm_mx_quantize(X: np.ndarray):
    """Host float X [R][K] -> (MXFP4 codes uint8 [R][K/2], scales uint8 [R][K/32])."""
    X = np.ascontiguousarray(X, dtype=np.float32)
    R, K = X.shape
    q = np.zeros((R, K // 2), np.uint8)
    scales = np.zeros((R, K // 32), np.uint8)
    _check(load().qgemm_mx_quantize(R, K, _np_ptr(X), _np_ptr(q), _np_ptr(scales)), "qgemm_mx_quantize")
    return q, scales


def qgemm_mx_quantize_device(X, q=None, scales=None, stream=None):
    """Device X [R][K] (fp32, fp16 or bf16, rows may be strided) -> (MXFP4 codes
    uint8 [R][K/2], scales uint8 [R][K/32]), allocated here unless given."""
    dev = _same_device(X=X, q=q, scales=scales)
    if X.dtype not in _TYPE_IDS:
        raise ValueError(f"X: dtype {X.dtype} where float32, float16 or bfloat16 is required")
    ld = _row_stride(X, "X")
    R, K = X.shape
    if q is None:
        q = _empty((R, K // 2), torch.uint8, dev, stream)
    else:
        _exact(q, "q", (torch.uint8,), (R, K // 2))
    if scales is None:
        scales = _empty((R, K // 32), torch.uint8, dev, stream)
    else:
        _exact(scales, "scales", (torch.uint8,), (R, K // 32))
    _call("qgemm_mx_quantize_device", dev, stream, R, K, _TYPE_IDS[X.dtype], X.data_ptr(), ld, q.data_ptr(),
          scales.data_ptr())
    return q, scales


def qgemm_mx_dequantize_device(q, scales, dtype="f32", Y=None, stream=None):
    """Device MXFP4 codes [R][K/2] and scales [R][K/32] -> their values [R][K]
    in dtype ("f32", "f16", "bf16"), or into Y (whose rows may be strided)."""
    dev = _same_device(q=q, scales=scales, Y=Y)
    if q.dim() != 2:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [R][K/2]")
    R, K = q.shape[0], 2 * q.shape[1]
    _exact(q, "q", (torch.uint8,), (R, K // 2))
    _exact(scales, "scales", (torch.uint8,), (R, K // 32))
    if Y is None:
        if dtype not in TYPES:
            raise ValueError(f"unknown type {dtype}")
        Y, ld = _empty((R, K), _TORCH_TYPES[TYPES[dtype]], dev, stream), K
    else:
        if Y.dtype not in _TYPE_IDS or Y.shape != (R, K):
            raise ValueError(f"Y: {Y.dtype} {tuple(Y.shape)}, expected a float tensor of shape {(R, K)}")
        ld = _row_stride(Y, "Y")
    _call("qgemm_mx_dequantize_device", dev, stream, R, K, q.data_ptr(), scales.data_ptr(), _TYPE_IDS[Y.dtype],
          Y.data_ptr(), ld)
    return Y


def qgemm_mx_pack(K: int, N: int, q: np.ndarray, scales: np.ndarray):
    """Host canonical MXFP4 codes [N][K/2] and scales [N][K/32] -> (packed
    weights uint8, packed scales uint8), host."""
    wb, sb = qgemm_packed_size(K, N, QGEMM_MXFP4)
    q = np.ascontiguousarray(q, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.uint8)
    if q.size != N * (K // 2) or scales.size != N * (K // 32):
        raise ValueError(f"q, scales: {q.size} and {scales.size} bytes, expected {N * (K // 2)} and {N * (K // 32)}")
    wp, sp = np.empty(wb, np.uint8), np.empty(sb, np.uint8)
    _check(load().qgemm_mx_pack(K, N, _np_ptr(q), _np_ptr(scales), _np_ptr(wp), wb, _np_ptr(sp), sb),
           "qgemm_mx_pack")
    return wp, sp


def qgemm_mx_pack_device(K: int, N: int, q, scales, E: int = 1, Bq=None, Sp=None, stream=None):
    """Device canonical MXFP4 codes [E][N][K/2] and scales [E][N][K/32] (or
    without the first axis) -> (packed weights, packed scales) of all E
    weights, uint8 device tensors, one weight after the other."""
    dev = _same_device(q=q, scales=scales, Bq=Bq, Sp=Sp)
    wb, sb = qgemm_packed_size(K, N, QGEMM_MXFP4)
    for t, name, size in ((q, "q", E * N * (K // 2)), (scales, "scales", E * N * (K // 32))):
        if not t.is_contiguous():          # (a copy would be made on the current stream)
            raise ValueError(f"{name}: must be contiguous")
        _exact(t.view(-1), name, (torch.uint8,), (size,))
    if Bq is None:
        Bq = _empty(E * wb, torch.uint8, dev, stream)
    if Sp is None:
        Sp = _empty(E * sb, torch.uint8, dev, stream)
    _exact(Bq, "Bq", (torch.uint8,), (E * wb,))
    _exact(Sp, "Sp", (torch.uint8,), (E * sb,))
    _call("qgemm_mx_pack_device", dev, stream, K, N, E, q.data_ptr(), scales.data_ptr(), Bq.data_ptr(), Sp.data_ptr())
    return Bq, Sp


@functools.lru_cache(maxsize=4096)
def qgemm_group_plan_size(T: int, topk: int, E: int) -> int:
    b = ctypes.c_size_t()
    _check(load().qgemm_group_plan_size(T, topk, E, ctypes.byref(b)), "qgemm_group_plan_size")
    return b.value


def _scratch(workspace, ws_bytes: int):
    """Address of a workspace tensor that claims ws_bytes."""
    have = workspace.numel() * workspace.element_size()
    if have < ws_bytes:
        raise ValueError(f"workspace: {have} bytes, ws_bytes={ws_bytes} claimed")
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace.data_ptr()


def _own_scratch(need: int, workspace, ws_bytes: int, dev, stream):
    """(tensor, address, bytes) of a call's scratch: the caller's, or one from
    torch's allocator, which hands its memory out and takes it back in the order
    of the current stream at next to no cost. The caller holds the tensor until
    the library has enqueued every launch of the call: given back before, its
    memory could go to another thread's work on the same stream between two of
    them. For a call on another stream that order says nothing, so the library
    allocates on that stream itself."""
    if workspace is not None:
        return workspace, _scratch(workspace, ws_bytes), ws_bytes
    if need == 0 or ws_bytes or stream is not None:
        return None, None, ws_bytes
    scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    return scratch, scratch.data_ptr(), need


def qgemm_group_plan(ids, E: int, offsets=None, rows=None, slots=None, workspace=None, ws_bytes: int = 0,
                     stream=None):
    """Expert ids [T][topk] (int32 or int64; an id outside [0, E) has no slot)
    -> (offsets [E + 1], rows [T * topk], slots [T][topk]), int32, allocated
    here unless given."""
    dev = _same_device(ids=ids, offsets=offsets, rows=rows, slots=slots, workspace=workspace)
    if ids.dim() != 2:
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected [T][topk]")
    T, topk = ids.shape
    _exact(ids, "ids", (torch.int32, torch.int64), (T, topk))
    need = qgemm_group_plan_size(T, topk, E)       # raises for a bad size
    if offsets is None:
        offsets = _empty(E + 1, torch.int32, dev, stream)
    else:
        _exact(offsets, "offsets", (torch.int32,), (E + 1,))
    if rows is None:
        rows = _empty(T * topk, torch.int32, dev, stream)
    else:
        _exact(rows, "rows", (torch.int32,), (T * topk,))
    if slots is None:
        slots = _empty((T, topk), torch.int32, dev, stream)
    else:
        _exact(slots, "slots", (torch.int32,), (T, topk))
    held, ws, ws_bytes = _own_scratch(need, workspace, ws_bytes, dev, stream)
    _call("qgemm_group_plan", dev, stream, T, topk, E, ids.data_ptr(), int(ids.dtype == torch.int64),
          offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), ws, ws_bytes)
    del held
    return offsets, rows, slots


@functools.lru_cache(maxsize=4096)
def qgemm_grouped_workspace_size(S: int, a_rows: int, K: int, N: int, E: int, fmt) -> int:
    b = ctypes.c_size_t()
    _check(load().qgemm_grouped_workspace_size(S, a_rows, K, N, E, _fmt(fmt), ctypes.byref(b)),
           "qgemm_grouped_workspace_size")
    return b.value


def qgemm_run_grouped(K: int, N: int, E: int, fmt, A, rows, offsets, Bq, scales, C, bias=None, residual=None,
                      activation="none", out_type="f32", workspace=None, ws_bytes: int = 0, stream=None) -> None:
    """C[s] = act(A[rows[s]] x deq(B_e) + bias[e] + residual[s]) for the slots s
    of every expert e, offsets[e] <= s < offsets[e + 1]; A fp16 [a_rows][K],
    rows int32 [S] or None (slot s reads row s), C [S][N] fp32 or fp16 per
    out_type, bias fp32 [E][N], residual as C. Rows of C that no expert owns
    are left as they were."""
    dev = _same_device(A=A, rows=rows, offsets=offsets, Bq=Bq, scales=scales, C=C, bias=bias, residual=residual,
                       workspace=workspace)
    f = _fmt(fmt)
    if C.dim() != 2 or A.dim() != 2:
        raise ValueError("A, C: expected [a_rows][K] and [S][N]")
    S, a_rows = C.shape[0], A.shape[0]
    c_dt = torch.float16 if out_type in (1, "f16") else torch.float32
    _exact(A, "A", (torch.float16,), (a_rows, K))
    _exact(C, "C", (c_dt,), (S, N))
    _exact(offsets, "offsets", (torch.int32,), (E + 1,))
    if rows is not None:
        _exact(rows, "rows", (torch.int32,), (S,))
    if bias is not None:
        _exact(bias, "bias", (torch.float32,), (E, N))
    if residual is not None:
        _exact(residual, "residual", (c_dt,), (S, N))
    if f in (QGEMM_MXFP4, QGEMM_MXFP4_A4):     # the library refuses any other
        wb, sb = qgemm_packed_size(K, N, f)
        _exact(Bq, "Bq", (torch.uint8,), (E * wb,))
        _exact(scales, "scales", (torch.uint8,), (E * sb,))
    epi = Epilogue(_dev_ptr(bias), _dev_ptr(residual),
                   ACTIVATIONS[activation] if isinstance(activation, str) else int(activation),
                   OUT_TYPES[out_type] if isinstance(out_type, str) else int(out_type))
    need = qgemm_grouped_workspace_size(S, a_rows, K, N, E, f)
    held, ws, ws_bytes = _own_scratch(need, workspace, ws_bytes, dev, stream)
    _call("qgemm_run_grouped", dev, stream, S, a_rows, K, N, E, f, A.data_ptr(), _dev_ptr(rows), offsets.data_ptr(),
          Bq.data_ptr(), scales.data_ptr(), C.data_ptr(), ctypes.byref(epi), ws, ws_bytes)
    del held


def qgemm_group_combine(Y, slots, weights, C, stream=None) -> None:
    """C[t] = sum over j of weights[t][j] * Y[slots[t][j]] (a slot outside Y adds
    nothing); Y [S][N] and C [T][N] fp32 or fp16, slots int32 and weights fp32
    [T][topk]."""
    dev = _same_device(Y=Y, slots=slots, weights=weights, C=C)
    if Y.dim() != 2 or slots.dim() != 2:
        raise ValueError("Y, slots: expected [S][N] and [T][topk]")
    (S, N), (T, topk) = Y.shape, slots.shape
    half = (torch.float32, torch.float16)
    _exact(Y, "Y", half, (S, N))
    _exact(slots, "slots", (torch.int32,), (T, topk))
    _exact(weights, "weights", (torch.float32,), (T, topk))
    _exact(C, "C", half, (T, N))
    _call("qgemm_group_combine", dev, stream, T, topk, N, S, Y.data_ptr(), _TYPE_IDS[Y.dtype], slots.data_ptr(),
          weights.data_ptr(), C.data_ptr(), _TYPE_IDS[C.dtype])


# ---------------------------------------------------------------------------
# Convenience: a packed weight resident on the GPU.
# ---------------------------------------------------------------------------
class PackedWeight:
    """Quantise (or take) a weight, pack it and upload it to the GPU. For the
    MXFP4 formats the pairs are the scale bytes [N][K/32]; "mxfp4" products take
    the weights in fp16 (exact for scales 2^-23 .. 2^13, infinite above 65504),
    "mxfp4a4" ones as they are."""

    def __init__(self, fmt, K: int, N: int, w_canonical: np.ndarray,
                 pairs_canonical: np.ndarray | None, device="cuda"):
        self.fmt = _fmt(fmt)
        self.K, self.N = K, N
        if self.fmt in (QGEMM_MXFP4, QGEMM_MXFP4_A4):
            wp, sp = qgemm_mx_pack(K, N, w_canonical, pairs_canonical)
        else:
            wp, sp = qgemm_pack_weights(K, N, self.fmt, w_canonical, pairs_canonical)
        self.Bq = torch.from_numpy(wp).to(device)
        self.scales = torch.from_numpy(sp).to(device) if sp.size else None

    @classmethod
    def from_float(cls, fmt, W: np.ndarray, device="cuda"):
        """W [N][K] float -> quantised by the library's host quantiser."""
        f = _fmt(fmt)
        N, K = W.shape
        if f == QGEMM_F32:
            return cls(f, K, N, np.ascontiguousarray(W.T, dtype=np.float32), None, device)
        q, pairs = qgemm_mx_quantize(W) if f in (QGEMM_MXFP4, QGEMM_MXFP4_A4) else qgemm_quantize_weights(W, f)
        return cls(f, K, N, q, pairs, device)

    def __call__(self, A: torch.Tensor, C: torch.Tensor | None = None, stream=None):
        if A.dim() != 2 or A.shape[1] != self.K:
            raise ValueError(f"A: shape {tuple(A.shape)}, expected [M][{self.K}]")
        M = A.shape[0]
        if C is None:
            C = torch.empty((M, self.N), dtype=torch.float32, device=A.device)
        qgemm_run(M, self.K, self.N, self.fmt, A, self.Bq, self.scales, C, stream)
        return C
