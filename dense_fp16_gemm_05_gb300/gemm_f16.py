"""ctypes binding over the C ABI of ``libgemm_f16.so`` (``include/gemm_f16.h``).

Argument marshalling only: tensors become device pointers and sizes, the
current torch stream becomes a ``cudaStream_t``, and status codes become
exceptions.  Every element of C is computed by the library's sm_103a kernel;
there is no fallback of any kind.  If the library has not been built, every
call raises :class:`LibraryNotBuilt`.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

import torch

from . import build as _build

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = -1
GEMM_ERR_ALIGNMENT = -2
GEMM_ERR_UNSUPPORTED_DEVICE = -3
GEMM_ERR_LAUNCH = -4
GEMM_ERR_TIMEOUT = -5
GEMM_ERR_CUDA = -6

# Config argument: id in the low byte, flag bits above (include/gemm_f16.h).
GEMM_F16_CONFIG_ID_MASK = 0xFF
GEMM_F16_NO_SPLIT = 0x100
GEMM_F16_NO_KSPLIT = 0x200
GEMM_F16_KSPLIT_AUTO = 0x400
GEMM_F16_KSPLIT_TAIL = 0x800
GEMM_F16_KSPLIT_SHIFT = 12
GEMM_F16_KSPLIT_MASK = 0x1F000


def ksplit(n: int) -> int:
    """Config flag: cut K into at most n slices (2 <= n <= 16), see gemm_f16.h."""
    return int(n) << GEMM_F16_KSPLIT_SHIFT

HEADER = os.path.join(_build.INCLUDE, "gemm_f16.h")


class LibraryNotBuilt(RuntimeError):
    pass


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status in (GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT):
            try:
                detail = lib().gemm_f16_last_error_detail().decode()
            except LibraryNotBuilt:
                pass
        self.detail = detail
        super().__init__(f"{what}: status {status} ({strerror(status)})" + (f": {detail}" if detail else ""))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises LibraryNotBuilt if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise LibraryNotBuilt(f"{_build.LIB} is missing; build it with __graft_entry__.build() "
                              "or python -m dense_fp16_gemm_05_gb300.build")
    L = ctypes.CDLL(_build.LIB)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.gemm_f16.argtypes = [vp, vp, vp, i64, i64, i64, ci, vp]
    L.gemm_f16.restype = ci
    L.gemm_f16_ex.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, vp]
    L.gemm_f16_ex.restype = ci
    L.gemm_f16_ex_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, vp]
    L.gemm_f16_ex_noalloc.restype = ci
    L.gemm_f16_from_host.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
    L.gemm_f16_from_host.restype = ci
    L.gemm_f16_check.argtypes = [vp]
    L.gemm_f16_check.restype = ci
    L.gemm_f16_last_timeout_record.argtypes = []
    L.gemm_f16_last_timeout_record.restype = ctypes.c_uint64
    L.gemm_f16_last_error_detail.argtypes = []
    L.gemm_f16_last_error_detail.restype = ctypes.c_char_p
    L.gemm_f16_strerror.argtypes = [ci]
    L.gemm_f16_strerror.restype = ctypes.c_char_p
    L.gemm_f16_version.argtypes = []
    L.gemm_f16_version.restype = ci
    L.gemm_f16_num_configs.argtypes = []
    L.gemm_f16_num_configs.restype = ci
    L.gemm_f16_config_name.argtypes = [ci]
    L.gemm_f16_config_name.restype = ctypes.c_char_p
    L.gemm_f16_auto_config.argtypes = [i64, i64, i64]
    L.gemm_f16_auto_config.restype = ci
    L.gemm_f16_tx.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, ci, ci, vp]
    L.gemm_f16_tx.restype = ci
    L.gemm_f16_relu_backward.argtypes = [vp, vp, vp, i64, vp]
    L.gemm_f16_relu_backward.restype = ci
    L.gemm_f16_config_layouts.argtypes = [ci]
    L.gemm_f16_config_layouts.restype = ci
    L.gemm_f16_selftest_timeout.argtypes = [vp, vp, vp, i64, i64, i64, ci, ctypes.c_uint64, vp]
    L.gemm_f16_selftest_timeout.restype = ci
    L.attention_fwd_f16.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float, ci, vp]
    L.attention_fwd_f16.restype = ci
    L.attention_fwd_f16_queue.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float, ci, vp, vp]
    L.attention_fwd_f16_queue.restype = ci
    L.gemm_fp8_block_scaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
    L.gemm_fp8_block_scaled.restype = ci
    L.gemm_mxfp8_block_scaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
    L.gemm_mxfp8_block_scaled.restype = ci
    L.mxfp4_quantize.argtypes = [vp, ci, vp, vp, vp, i64, i64, ci, vp]
    L.mxfp4_quantize.restype = ci
    L.gemm_mxfp4.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
    L.gemm_mxfp4.restype = ci
    L.gemm_mxfp4_selftest_timeout.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ctypes.c_uint64, vp]
    L.gemm_mxfp4_selftest_timeout.restype = ci
    cf = ctypes.c_float
    L.layer_norm_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, cf, ci, ci, vp]
    L.layer_norm_fwd.restype = ci
    L.layer_norm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, ci, ci, vp, i64, vp]
    L.layer_norm_bwd.restype = ci
    L.layer_norm_bwd_selftest_timeout.argtypes = [vp, vp, vp, vp, vp, i64, i64, ci, ctypes.c_uint64, vp]
    L.layer_norm_bwd_selftest_timeout.restype = ci
    L.layer_norm_bwd_workspace.argtypes = [i64, i64]
    L.layer_norm_bwd_workspace.restype = i64
    pi = ctypes.POINTER(ctypes.c_int)
    L.gemm_fp8_launch_info.argtypes = [i64, i64, i64, pi, pi]
    L.gemm_fp8_launch_info.restype = ci
    L.gemm_f16_launch_info.argtypes = [i64, i64, i64, ci, pi, pi, pi]
    L.gemm_f16_launch_info.restype = ci
    L.gemm_f16_config_cluster_k.argtypes = [ci]
    L.gemm_f16_config_cluster_k.restype = ci
    L.gemm_f16_tma_box_image.argtypes = [vp, i64, i64, i64, i64, i64, vp, vp]
    L.gemm_f16_tma_box_image.restype = ci
    _lib = L
    return L


def header_functions() -> list[str]:
    """Names of the functions declared in include/gemm_f16.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gemm_f16\w*)\s*\(", text)))


def strerror(status: int) -> str:
    try:
        return lib().gemm_f16_strerror(int(status)).decode()
    except LibraryNotBuilt:
        return "library not built"


def version() -> int:
    return int(lib().gemm_f16_version())


def num_configs() -> int:
    return int(lib().gemm_f16_num_configs())


def config_name(config: int) -> str | None:
    r = lib().gemm_f16_config_name(int(config))
    return None if r is None else r.decode()


def config_label(config: int) -> str | None:
    """config_name plus "+nosplit" / "+ksplitN" / "+ksplitauto" / "+noksplit" for the flag bits."""
    name = config_name(config)
    if name is None:
        return None
    c = int(config)
    n = (c & GEMM_F16_KSPLIT_MASK) >> GEMM_F16_KSPLIT_SHIFT
    return (name + ("+nosplit" if c & GEMM_F16_NO_SPLIT else "") + (f"+ksplit{n}" if n else "")
            + ("+ksplitauto" if c & GEMM_F16_KSPLIT_AUTO else "") + ("+ksplittail" if c & GEMM_F16_KSPLIT_TAIL else "")
            + ("+noksplit" if c & GEMM_F16_NO_KSPLIT else ""))


# Raw handle of torch's current stream on a device, without building a
# torch.cuda.Stream object (a few microseconds per call on small problems).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _NoSwitch:
    __slots__ = ()

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NO_SWITCH = _NoSwitch()


def _device_index(device) -> int:
    if isinstance(device, int):
        return device
    idx = (device if isinstance(device, torch.device) else torch.device(device)).index
    return idx if idx is not None else torch.cuda.current_device()


def _device_scope(device):
    """Makes ``device`` (a torch.device, index or name) current for the call;
    no switch when it already is."""
    if _device_index(device) == torch.cuda.current_device():
        return _NO_SWITCH
    return torch.cuda.device(device)


def _stream_handle(stream, device) -> int:
    if stream is None:
        if _current_raw_stream is not None:
            return int(_current_raw_stream(_device_index(device)))
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return int(stream.cuda_stream)
    return int(stream)


# Index of the current device without torch.cuda.current_device's lazy-init
# check (a CUDA tensor in hand means CUDA is up).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn, what: str, device: torch.device, stream, *args):
    """fn(*args, stream) on ``device``; GemmError for a status that is not GEMM_OK.

    A call on a small problem is bound by the host, so this does what
    _device_scope and _stream_handle do with as few steps as the common case
    (a CUDA tensor on the current device, torch's current stream) allows.
    """
    idx = device.index
    if stream is None and idx is not None and _current_raw_stream is not None and idx == _current_device():
        st = fn(*args, _current_raw_stream(idx))
    else:
        with _device_scope(device):
            st = fn(*args, _stream_handle(stream, device))
    if st != GEMM_OK:
        raise GemmError(st, what)


# torch's allocation of a strided CUDA tensor on the current device without the
# argument parser and dispatcher of torch.empty: 1.4 us instead of 3 us between
# launches, for calls that are bound by the host.  The same allocator, so stream
# order and graph pools are the same; dispatch modes and the deterministic fill of
# new memory do not see these tensors, which the launch that follows writes.  The
# name is not a public one: it is tried once before it is relied on.
def _find_empty_strided():
    """The function, or None where it is missing or does not do what _new needs."""
    try:
        f = torch._C._dynamo.guards._empty_strided_cuda
        t = f((2, 3), (3, 1), torch.float16)
        if (tuple(t.shape) == (2, 3) and t.stride() == (3, 1) and t.dtype == torch.float16
                and t.device == torch.device("cuda", _current_device())):
            return f
    except (AttributeError, TypeError, ValueError):
        pass
    return None


_empty_strided_cuda = False   # not looked for yet


def _new(shape, dtype, device, stream=None) -> torch.Tensor:
    """torch.empty(shape) for one to three sizes, an output of a launch on ``stream``."""
    if stream is not None:
        return _new_on(stream, shape, dtype, device)
    if device.index is None or device.index != _current_device():
        return torch.empty(shape, dtype=dtype, device=device)
    global _empty_strided_cuda
    if not _empty_strided_cuda:
        if _empty_strided_cuda is False:
            _empty_strided_cuda = _find_empty_strided()
            return _new(shape, dtype, device)
        return torch.empty(shape, dtype=dtype, device=device)
    n = len(shape)   # plain tuples below: the function takes no torch.Size
    if n == 2:
        r, c = shape
        return _empty_strided_cuda((r, c), (c, 1), dtype)
    if n == 1:
        return _empty_strided_cuda((shape[0],), (1,), dtype)
    if n == 3:
        b, r, c = shape
        return _empty_strided_cuda((b, r, c), (r * c, c, 1), dtype)
    return torch.empty(shape, dtype=dtype, device=device)


def _on_gpu(device) -> bool:
    return device.type == "cuda"


def _new_on(stream, shape, dtype, device) -> torch.Tensor:
    """torch.empty(shape) for a launch on ``stream`` (None: torch's current stream).

    Made on the stream that writes it: a block of the current stream's pool may
    still be in use by work queued there, which the launch does not wait for.
    The current stream, on which the caller gets the tensor, is recorded, so
    that the memory is not reused before what is queued there is done.
    """
    if stream is None or not _on_gpu(device):   # the library refuses host memory
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_launch_stream(stream, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _used_on(stream, device, *tensors):
    """Tells the allocator that a call's tensors, inputs too, are used on ``stream``:
    a caller may drop them at once and their memory is not reused before that
    stream is done."""
    if stream is not None:
        s = _launch_stream(stream, device)
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def _check_operand(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float16 or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D float16 tensor, got {t.dtype} {tuple(t.shape)}")


def gemm_f16(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None, relu: bool = True,
             stream=None, config: int = 0) -> torch.Tensor:
    """C = ReLU(A @ B) (relu=True) or A @ B, fp16 in and out, fp32 accumulation.

    A (M,K), B (K,N), C (M,N): contiguous float16 CUDA tensors on one device.
    C is allocated (torch.empty) when not given.  The call is asynchronous on
    ``stream`` (default: torch's current stream); errors in the arguments raise
    :class:`GemmError` immediately.
    """
    _check_operand(A, "A")
    _check_operand(B, "B")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner sizes differ: A {tuple(A.shape)}, B {tuple(B.shape)}")
    if C is None:
        C = _new_on(stream, (M, N), torch.float16, A.device)
    _check_operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    L = _lib if _lib is not None else lib()
    with _device_scope(A.device):
        st = L.gemm_f16_ex(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, int(bool(relu)), int(config),
                           _stream_handle(stream, A.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16")
    return C


def gemm_f16_noalloc(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, relu: bool = True, stream=None,
                     config: int = 0) -> torch.Tensor:
    """gemm_f16 through gemm_f16_ex_noalloc: K-slice partials in the library's
    fixed 16 MiB scratch instead of an allocation (see gemm_f16.h for the size
    limit and the rule that overlapping calls on one device race).  C must be
    given: nothing is allocated."""
    _check_operand(A, "A")
    _check_operand(B, "B")
    _check_operand(C, "C")
    M, K = A.shape
    K2, N = B.shape
    if K != K2 or tuple(C.shape) != (M, N):
        raise ValueError(f"shapes A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)} do not match")
    L = lib()
    with _device_scope(A.device):
        st = L.gemm_f16_ex_noalloc(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, int(bool(relu)), int(config),
                                   _stream_handle(stream, A.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16_ex_noalloc")
    return C


def gemm_f16_t(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None, transa: bool = False,
               transb: bool = False, relu: bool = True, stream=None, config: int = 0) -> torch.Tensor:
    """C = ReLU(op(A) @ op(B)) (relu=True) or op(A) @ op(B), fp16, fp32 accumulation.

    op(A) = A if not transa (A is (M,K)), else A.T (A stored (K,M));
    op(B) = B if not transb (B is (K,N)), else B.T (B stored (N,K)).
    All tensors contiguous float16 CUDA tensors; C (M,N) is allocated if not given.
    """
    _check_operand(A, "A")
    _check_operand(B, "B")
    M, K = (A.shape[1], A.shape[0]) if transa else (A.shape[0], A.shape[1])
    K2, N = (B.shape[1], B.shape[0]) if transb else (B.shape[0], B.shape[1])
    if K != K2:
        raise ValueError(f"inner sizes differ: op(A) {M}x{K}, op(B) {K2}x{N}")
    if C is None:
        C = _new_on(stream, (M, N), torch.float16, A.device)
    _check_operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    with _device_scope(A.device):
        st = lib().gemm_f16_tx(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, int(bool(transa)),
                               int(bool(transb)), int(bool(relu)), int(config), _stream_handle(stream, A.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16_tx")
    return C


def relu_backward(dC: torch.Tensor, C: torch.Tensor, dZ: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dZ = dC where C > 0 else +0 (gradient through the fused ReLU), on the GPU."""
    for t, n in ((dC, "dC"), (C, "C")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float16 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous float16 tensor")
    if dC.shape != C.shape:
        raise ValueError(f"dC {tuple(dC.shape)} and C {tuple(C.shape)} differ")
    if dZ is None:
        dZ = _new_on(stream, dC.shape, torch.float16, dC.device)
    with _device_scope(dC.device):
        st = lib().gemm_f16_relu_backward(dC.data_ptr(), C.data_ptr(), dZ.data_ptr(), dC.numel(),
                                          _stream_handle(stream, dC.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16_relu_backward")
    return dZ


def tma_box_image(X: torch.Tensor, box_rows: int, x: int, y: int, stream=None) -> torch.Tensor:
    """Raw shared-memory image (uint8, box_rows * 128 bytes) of one box of
    box_rows x 64 elements of the 2-D fp16 tensor X at column x, row y, loaded
    by TMA with the GEMM's operand encoding (gemm_f16_tma_box_image)."""
    _check_operand(X, "X")
    rows, cols = X.shape
    out = _new_on(stream, (int(box_rows) * 128,), torch.uint8, X.device)
    L = lib()
    with _device_scope(X.device):
        st = L.gemm_f16_tma_box_image(X.data_ptr(), rows, cols, int(box_rows), int(x), int(y), out.data_ptr(),
                                      _stream_handle(stream, X.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16_tma_box_image")
    return out


def config_cluster_k(config: int) -> bool:
    """True if the configuration splits K across a cluster (no workspace)."""
    r = lib().gemm_f16_config_cluster_k(int(config))
    if r < 0:
        raise GemmError(r, "gemm_f16_config_cluster_k")
    return r == 1


def workspace_split_configs() -> list[int]:
    """Fixed configuration ids whose K split uses a workspace."""
    return [c for c in range(1, num_configs() + 1) if not config_cluster_k(c)]


def config_layouts(config: int) -> int:
    return int(lib().gemm_f16_config_layouts(int(config)))


def gemm_f16_raw(A_ptr: int, B_ptr: int, C_ptr: int, M: int, N: int, K: int, relu: int, stream: int = 0,
                 config: int = 0) -> int:
    """The C call with raw pointers; returns the status code (no exception)."""
    return int(lib().gemm_f16_ex(A_ptr, B_ptr, C_ptr, M, N, K, relu, config, stream))


def gemm_f16_from_host(A_host: torch.Tensor, B_host: torch.Tensor, C_host: torch.Tensor,
                       A_dev: torch.Tensor, B_dev: torch.Tensor, C_dev: torch.Tensor,
                       relu: bool = True, stream=None) -> None:
    """End-to-end call: host A, B -> device, GEMM, device C -> host, ordered on ``stream``.

    A and C move in row panels so that copies and GEMMs overlap (see
    gemm_f16.h); the host tensors should be pinned (``pin_memory()``) for
    asynchronous copies.  Returns after enqueueing; synchronising the stream
    is enough before reading C_host.
    """
    for t, n in ((A_host, "A_host"), (B_host, "B_host"), (C_host, "C_host"),
                 (A_dev, "A_dev"), (B_dev, "B_dev"), (C_dev, "C_dev")):
        _check_operand(t, n)
    M, K = A_host.shape
    N = B_host.shape[1]
    L = lib()
    with _device_scope(A_dev.device):
        st = L.gemm_f16_from_host(A_host.data_ptr(), B_host.data_ptr(), C_host.data_ptr(), A_dev.data_ptr(),
                                  B_dev.data_ptr(), C_dev.data_ptr(), M, N, K, int(bool(relu)),
                                  _stream_handle(stream, A_dev.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16_from_host")


def check(stream=None, device=None) -> int:
    """Synchronises the stream and returns the device status (GEMM_OK or an error code)."""
    dev = device if device is not None else torch.cuda.current_device()
    with _device_scope(dev):
        return int(lib().gemm_f16_check(_stream_handle(stream, dev)))


def auto_config(M: int, N: int, K: int) -> int:
    return int(lib().gemm_f16_auto_config(M, N, K))


def launch_info(M: int, N: int, K: int, config: int = 0) -> dict:
    """Grid CTAs, cluster size and tile count that a call would launch with."""
    g, c, t = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = lib().gemm_f16_launch_info(M, N, K, int(config), ctypes.byref(g), ctypes.byref(c), ctypes.byref(t))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_f16_launch_info")
    return {"grid_ctas": g.value, "cluster_size": c.value, "tiles": t.value}


def selftest_timeout(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, config: int = 0,
                     timeout_cycles: int = 1 << 24, stream=None) -> int:
    """Launches the kernel with its producer switched off so that a bounded wait
    runs out (test hook); returns the launch status.  Read the outcome with check()."""
    M, K = A.shape
    N = B.shape[1]
    with _device_scope(A.device):
        return int(lib().gemm_f16_selftest_timeout(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, int(config),
                                                   int(timeout_cycles), _stream_handle(stream, A.device)))


def last_timeout_record() -> int:
    return int(lib().gemm_f16_last_timeout_record())


FP8_BLOCK = 128


def _check_fp8(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D uint8 / float8_e4m3fn tensor, got {t.dtype} {tuple(t.shape)}")


def _check_scales(t: torch.Tensor, name: str, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def gemm_fp8_block_scaled(A: torch.Tensor, SA: torch.Tensor, W: torch.Tensor, SW: torch.Tensor,
                          C: torch.Tensor | None = None, relu: bool = False, stream=None) -> torch.Tensor:
    """C = R(sum_b SA[:,b] SW[n/128,b] (A_b @ W_b^T)): the FP8 block-scaled linear layer.

    A (M,K) and W (N,K): E4M3 codes (uint8 or float8_e4m3fn) on one CUDA
    device; SA (M, ceil(K/128)) and SW (ceil(N/128), ceil(K/128)) float32;
    C (M,N) float16, allocated when not given.  Asynchronous on ``stream``.
    """
    _check_fp8(A, "A")
    _check_fp8(W, "W")
    M, K = A.shape
    N, K2 = W.shape
    if K != K2:
        raise ValueError(f"inner sizes differ: A {tuple(A.shape)}, W {tuple(W.shape)}")
    KB, NB = -(-K // FP8_BLOCK), -(-N // FP8_BLOCK)
    _check_scales(SA, "SA", (M, KB))
    _check_scales(SW, "SW", (NB, KB))
    if C is None:
        C = _new_on(stream, (M, N), torch.float16, A.device)
    _check_operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    L = lib()
    with _device_scope(A.device):
        st = L.gemm_fp8_block_scaled(A.data_ptr(), SA.data_ptr(), W.data_ptr(), SW.data_ptr(), C.data_ptr(),
                                     M, N, K, int(bool(relu)), _stream_handle(stream, A.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp8_block_scaled")
    return C


def gemm_mxfp8_block_scaled(A: torch.Tensor, SA: torch.Tensor, W: torch.Tensor, SW: torch.Tensor,
                            C: torch.Tensor | None = None, relu: bool = True, stream=None) -> torch.Tensor:
    """FP8 block-scaled GEMM with power-of-two scales: SA (M, ceil(K/128)) and
    SW (ceil(N/128), ceil(K/128)) uint8 E8M0 exponents; otherwise as
    gemm_fp8_block_scaled (see gemm_f16.h)."""
    _check_fp8(A, "A")
    _check_fp8(W, "W")
    M, K = A.shape
    N, K2 = W.shape
    if K != K2:
        raise ValueError(f"A {tuple(A.shape)} and W {tuple(W.shape)} disagree on K")
    KB, NB = -(-K // 128), -(-N // 128)
    for t, name, shape in ((SA, "SA", (M, KB)), (SW, "SW", (NB, KB))):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape}")
    if C is None:
        C = _new_on(stream, (M, N), torch.float16, A.device)
    _check_operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    L = lib()
    with _device_scope(A.device):
        st = L.gemm_mxfp8_block_scaled(A.data_ptr(), SA.data_ptr(), W.data_ptr(), SW.data_ptr(), C.data_ptr(),
                                       M, N, K, int(bool(relu)), _stream_handle(stream, A.device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_mxfp8_block_scaled")
    return C


TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}   # enum gemm_f16_type
MXFP4_BLOCK = 32


def mxfp4_shapes(rows: int, K: int) -> tuple[tuple[int, int], tuple[int, int, int]]:
    """Shapes of the codes and of the scale tiles of a (rows, K) MXFP4 matrix (see gemm_f16.h)."""
    return (rows, 16 * -(-K // MXFP4_BLOCK)), (-(-rows // 128), -(-K // 128), 512)


def mxfp4_tile_scales(E: torch.Tensor) -> torch.Tensor:
    """Scale bytes E (rows, blocks), one per row and block of 32, in the tile order of gemm_mxfp4.

    A layout change in torch, on E's device: for weights that come with
    row-major scales.  Fill bytes are zero.
    """
    if not isinstance(E, torch.Tensor) or E.dtype != torch.uint8 or E.dim() != 2:
        raise ValueError("E must be a 2-D uint8 tensor")
    rows, KB = E.shape
    RB, KT = -(-rows // 128), -(-KB // 4)
    full = torch.zeros((RB * 128, KT * 4), dtype=torch.uint8, device=E.device)
    full[:rows, :KB] = E
    return full.reshape(RB, 4, 32, KT, 4).permute(0, 3, 2, 1, 4).reshape(RB, KT, 512).contiguous()


def mxfp4_row_scales(S: torch.Tensor, rows: int, K: int) -> torch.Tensor:
    """The inverse of mxfp4_tile_scales: scale bytes (rows, ceil(K/32)) of tiles S."""
    if not isinstance(S, torch.Tensor) or S.dtype != torch.uint8 or tuple(S.shape) != mxfp4_shapes(rows, K)[1]:
        raise ValueError(f"S must be a uint8 tensor of shape {mxfp4_shapes(rows, K)[1]}")
    RB, KT, _ = S.shape
    full = S.reshape(RB, KT, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(RB * 128, KT * 4)
    return full[:rows, :-(-K // MXFP4_BLOCK)].contiguous()


def _check_like(t, name: str, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def mxfp4_quantize(X: torch.Tensor, transpose: bool = False, values: bool = False, Q: torch.Tensor | None = None,
                   S: torch.Tensor | None = None, V: torch.Tensor | None = None, stream=None):
    """MXFP4 codes and scale tiles (Q, S) of the (rows, K) matrix X, or (Q, S, V) with ``values``.

    X: contiguous 2-D float16, bfloat16 or float32 CUDA tensor; with
    ``transpose`` it is (K, rows) and its columns are quantised (a weight
    stored in-features x out-features becomes gemm_mxfp4's W).  V holds the
    values the codes stand for, (rows, K) of X's type.  Q, S and V are
    allocated when not given; formats and rounding as in gemm_f16.h.
    Asynchronous on ``stream``.
    """
    if not isinstance(X, torch.Tensor):
        raise TypeError("X must be a torch.Tensor")
    dtype, shape = X.dtype, X.shape
    code = TYPES.get(dtype)
    if code is None or len(shape) != 2 or not X.is_contiguous():
        raise ValueError(f"X must be a contiguous 2-D float16, bfloat16 or float32 tensor, got {dtype} {tuple(shape)}")
    K, rows = shape if transpose else (shape[1], shape[0])
    dev = X.device
    q_shape, s_shape = mxfp4_shapes(rows, K)
    if Q is None:
        Q = _new(q_shape, torch.uint8, dev, stream)
    else:
        _check_like(Q, "Q", torch.uint8, q_shape, dev)
    if S is None:
        S = _new(s_shape, torch.uint8, dev, stream)
    else:
        _check_like(S, "S", torch.uint8, s_shape, dev)
    if V is not None:
        _check_like(V, "V", dtype, (rows, K), dev)
    elif values:
        V = _new((rows, K), dtype, dev, stream)
    _call((_lib or lib()).mxfp4_quantize, "mxfp4_quantize", dev, stream, X.data_ptr(), code, Q.data_ptr(),
          S.data_ptr(), _ptr(V), rows, K, 1 if transpose else 0)
    _used_on(stream, dev, X, Q, S, V)
    return (Q, S) if V is None else (Q, S, V)


def gemm_mxfp4(A: torch.Tensor, SA: torch.Tensor, W: torch.Tensor, SW: torch.Tensor, C: torch.Tensor | None = None,
               relu: bool = False, K: int | None = None, stream=None) -> torch.Tensor:
    """C = R(A @ W^T) from MXFP4 operands (codes and scale tiles of mxfp4_quantize), C float16.

    A, SA: packed (M,K); W, SW: packed (N,K).  K defaults to the codes' width,
    2 A.shape[1] (give it when K is not a multiple of 32).  C (M,N) is
    allocated when not given.  Asynchronous on ``stream``.
    """
    for t, name in ((A, "A"), (W, "W")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D uint8 tensor, got {tuple(t.shape)}")
    M, a_bytes = A.shape
    N = W.shape[0]
    K = 2 * a_bytes if K is None else int(K)
    dev = A.device
    u8 = torch.uint8
    q_shape, s_shape = mxfp4_shapes(M, K)
    _check_like(A, "A", u8, q_shape, dev)
    _check_like(SA, "SA", u8, s_shape, dev)
    q_shape, s_shape = mxfp4_shapes(N, K)
    _check_like(W, "W", u8, q_shape, dev)
    _check_like(SW, "SW", u8, s_shape, dev)
    if C is None:
        C = _new((M, N), torch.float16, dev, stream)
    else:
        _check_like(C, "C", torch.float16, (M, N), dev)
    _call((_lib or lib()).gemm_mxfp4, "gemm_mxfp4", dev, stream, A.data_ptr(), SA.data_ptr(), W.data_ptr(),
          SW.data_ptr(), C.data_ptr(), M, N, K, 1 if relu else 0)
    _used_on(stream, dev, A, SA, W, SW, C)
    return C


def _norm_input(X, name: str = "X"):
    """(type code, dtype, shape, rows, dim) of a layer norm input."""
    if not isinstance(X, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype, shape = X.dtype, X.shape
    code = TYPES.get(dtype)
    if code is None or len(shape) < 1 or not X.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float16, bfloat16 or float32 tensor, got {dtype} {tuple(shape)}")
    dim = shape[-1]
    return code, dtype, shape, (shape[0] if len(shape) == 2 else math.prod(shape[:-1])), dim


def _norm_weight_type(dtype, dim: int, device, *weights) -> torch.dtype:
    wt = None
    for w in weights:
        if w is None:
            continue
        if wt is None:
            wt = w.dtype if isinstance(w, torch.Tensor) else dtype
            if wt != dtype and wt != torch.float32:
                raise ValueError(f"weights must be of X's type {dtype} or float32, got {wt}")
        _check_like(w, "a weight", wt, (dim,), device)
    return dtype if wt is None else wt


def layer_norm_fwd(X: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                   eps: float = 1e-5, Y: torch.Tensor | None = None, stats: bool = True, stream=None):
    """(Y, mean, rstd) of layer norm over X's last dimension (see gemm_f16.h).

    X: contiguous float16, bfloat16 or float32 CUDA tensor; gamma, beta: None
    (ones, zeros) or vectors of X's type or float32.  mean and rstd are float32
    of X's leading shape, or None without ``stats``.  Asynchronous on ``stream``.
    """
    code, dtype, shape, rows, dim = _norm_input(X)
    dev = X.device
    wt = _norm_weight_type(dtype, dim, dev, gamma, beta)
    if Y is None:
        Y = _new(shape, dtype, dev, stream)
    else:
        _check_like(Y, "Y", dtype, shape, dev)
    mean = rstd = None
    if stats:
        lead = shape[:-1]
        mean = _new(lead, torch.float32, dev, stream)
        rstd = _new(lead, torch.float32, dev, stream)
    _call((_lib or lib()).layer_norm_fwd, "layer_norm_fwd", dev, stream, X.data_ptr(), _ptr(gamma), _ptr(beta),
          Y.data_ptr(), _ptr(mean), _ptr(rstd), rows, dim, eps, code, TYPES[wt])
    _used_on(stream, dev, X, gamma, beta, Y, mean, rstd)
    return Y, mean, rstd


def layer_norm_bwd_workspace(rows: int, dim: int, device=None) -> int:
    """Bytes of workspace layer_norm_bwd needs."""
    with _device_scope(torch.cuda.current_device() if device is None else device):
        n = int(lib().layer_norm_bwd_workspace(rows, dim))
    if n < 0:
        raise GemmError(n, "layer_norm_bwd_workspace")
    return n


def layer_norm_bwd(dY: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   gamma: torch.Tensor | None = None, dX: torch.Tensor | None = None, weights: bool = True,
                   wtype: torch.dtype | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(dX, dgamma, dbeta) of layer_norm_fwd; dgamma and dbeta None without ``weights``.

    dY like X; mean, rstd and gamma as given to and returned by
    layer_norm_fwd.  dgamma and dbeta have gamma's type (``wtype`` without a
    gamma, X's type by default).  ``workspace``: a float32 vector of
    layer_norm_bwd_workspace bytes for callers that keep one; made on the
    launch stream when not given.  Asynchronous on ``stream``.
    """
    code, dtype, shape, rows, dim = _norm_input(X)
    dev = X.device
    _check_like(dY, "dY", dtype, shape, dev)
    lead = shape[:-1]
    _check_like(mean, "mean", torch.float32, lead, dev)
    _check_like(rstd, "rstd", torch.float32, lead, dev)
    wt = _norm_weight_type(dtype, dim, dev, gamma)
    if gamma is None and wtype is not None:
        wt = wtype
        if wt != dtype and wt != torch.float32:
            raise ValueError(f"wtype must be X's type {dtype} or float32, got {wt}")
    if dX is None:
        dX = _new(shape, dtype, dev, stream)
    else:
        _check_like(dX, "dX", dtype, shape, dev)
    L = _lib or lib()
    dgamma = dbeta = None
    ws_bytes = 0
    if weights:
        dgamma = _new((dim,), wt, dev, stream)
        dbeta = _new((dim,), wt, dev, stream)
        if workspace is None:
            if dev.index == _current_device():
                need = L.layer_norm_bwd_workspace(rows, dim)
                if need < 0:
                    raise GemmError(need, "layer_norm_bwd_workspace")
            else:
                need = layer_norm_bwd_workspace(rows, dim, dev)
            if stream is None:
                workspace = _new((need // 4,), torch.float32, dev)
            else:
                with torch.cuda.stream(_launch_stream(stream, dev)):
                    workspace = torch.empty((need // 4,), dtype=torch.float32, device=dev)
        elif (not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.float32
              or not workspace.is_contiguous() or workspace.device != dev):
            raise ValueError("workspace must be a contiguous float32 tensor on X's device")
        ws_bytes = 4 * workspace.numel()
    _call(L.layer_norm_bwd, "layer_norm_bwd", dev, stream, dY.data_ptr(), X.data_ptr(), _ptr(gamma), mean.data_ptr(),
          rstd.data_ptr(), dX.data_ptr(), _ptr(dgamma), _ptr(dbeta), rows, dim, code, TYPES[wt],
          _ptr(workspace) if weights else None, ws_bytes)
    _used_on(stream, dev, dY, X, mean, rstd, gamma, dX, dgamma, dbeta, workspace if weights else None)
    return dX, dgamma, dbeta


def fp8_launch_info(M: int, N: int, K: int) -> dict:
    g, t = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().gemm_fp8_launch_info(M, N, K, ctypes.byref(g), ctypes.byref(t))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp8_launch_info")
    return {"grid_ctas": g.value, "tiles": t.value}


def _launch_stream(stream, device) -> torch.cuda.Stream:
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if int(stream) == 0:   # the default stream; of a null handle ExternalStream makes a new one
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(int(stream), device=device)


def attention_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None = None,
                  sm_scale: float | None = None, causal: bool = False, stream=None,
                  queue: torch.Tensor | bool | None = None) -> torch.Tensor:
    """O = softmax(sm_scale Q K^T [causal]) V per (batch, head).

    Q, K, V (and O): contiguous float16 CUDA tensors of one shape
    (batch, heads, seq, dim), dim 64 or 128; sm_scale defaults to
    1/sqrt(dim).  O is allocated when not given.  Asynchronous on ``stream``.

    ``queue`` (causal only): the work queue of attention_fwd_f16_queue, a
    2-element int32 CUDA tensor that is zero when the launch starts and that
    the kernel leaves zero; one queue serves launches that run one after
    another, launches that may overlap need one each.  None: a fresh zeroed
    queue is made on the launch stream for this call.  False: no queue (the
    fixed shares of attention_fwd_f16).  Results are the same bits either way.
    """
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous 4-D float16 tensor")
    if Q.shape != K.shape or Q.shape != V.shape:
        raise ValueError(f"Q, K, V shapes differ: {tuple(Q.shape)} {tuple(K.shape)} {tuple(V.shape)}")
    B, H, S, D = Q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if O is None:
        O = _new_on(stream, Q.shape, torch.float16, Q.device)
    if O.dtype != torch.float16 or O.shape != Q.shape or not O.is_contiguous():
        raise ValueError("O must be a contiguous float16 tensor shaped like Q")
    q_ptr = None
    if causal and queue is not False and Q.numel() > 0:
        if queue is None or queue is True:
            with torch.cuda.stream(_launch_stream(stream, Q.device)):
                queue = torch.zeros(2, dtype=torch.int32, device=Q.device)
        if (not isinstance(queue, torch.Tensor) or queue.dtype != torch.int32 or queue.numel() < 2
                or not queue.is_contiguous() or queue.device != Q.device):
            raise ValueError("queue must be a contiguous int32 tensor of >= 2 elements on Q's device")
        q_ptr = queue.data_ptr()
    L = lib()
    with _device_scope(Q.device):
        st = L.attention_fwd_f16_queue(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), B, H, S, D,
                                       float(sm_scale), int(bool(causal)), q_ptr, _stream_handle(stream, Q.device))
    if st != GEMM_OK:
        raise GemmError(st, "attention_fwd_f16_queue")
    return O
