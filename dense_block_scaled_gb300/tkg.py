"""ctypes binding of libtkg.so (C ABI in include/tkg_gemm.h).

Argument marshalling only: every entry point forwards device pointers, sizes
and a CUDA stream handle to the library; all arithmetic runs in the library's
CUDA kernels.  The library is built in-tree (``python -m
dense_block_scaled_gb300.build``); if it is missing or fails to load, every
call raises -- there is no fallback path.

Helpers accept torch tensors only as carriers of device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
# TKG_LIBRARY selects another build of the library, e.g. libtkg_check.so
LIB_PATH = os.environ.get("TKG_LIBRARY") or os.path.join(PKG, "libtkg.so")

OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_CHECK = range(7)
OPT_CTA_GROUP, OPT_SINGLE_STAGE, OPT_TIMEOUT_MS, OPT_INJECT_STALL, OPT_MAX_CLUSTERS, OPT_ACC_STAGES = 1, 2, 3, 4, 5, 6
OPT_SCHEDULER = 7
OPT_SPLIT_K = 8
OPT_RASTER_GROUP = 9
OPT_BF16_TILE_N = 10
OPT_TAIL_SPLIT = 11
OPT_EPILOGUE_STORE = 12

EXPORTS = [
    "tkg_gemm_bf16", "tkg_gemm_mxfp8", "tkg_gemm_nvfp4", "tkg_get_device_status", "tkg_status_string",
    "tkg_scale_bytes", "tkg_scales_to_tiled", "tkg_quantize_mxfp8", "tkg_quantize_nvfp4",
    "tkg_set_option", "tkg_get_option", "tkg_gemm_bf16_noalloc",
    "tkg_gemm_grouped_bf16", "tkg_gemm_grouped_mxfp8", "tkg_gemm_grouped_nvfp4", "tkg_grouped_scale_bytes",
    "tkg_gemm_bf16_from_host", "tkg_gemm_grouped_dev_bf16", "tkg_gemm_grouped_dev_mxfp8",
    "tkg_gemm_grouped_dev_nvfp4", "tkg_grouped_dev_scale_bytes", "tkg_quantize_nvfp4_scaled",
    "tkg_gemm_list_bf16", "tkg_gemm_list_mxfp8", "tkg_gemm_list_nvfp4",
    "tkg_gemm_bf16_strided", "tkg_gemm_mxfp8_strided", "tkg_gemm_nvfp4_strided",
    "tkg_linear_ce_loss", "tkg_linear_ce_loss_workspace_bytes", "tkg_linear_ce_grad",
    "tkg_linear_ce_grad_workspace_bytes", "tkg_gemm_grouped_dev_bf16_dgrad", "tkg_gemm_grouped_dev_bf16_wgrad",
]

MAX_LIST = 16

GRAD_BF16, GRAD_F32, GRAD_F32_ADD = 0, 1, 2


class GemmDesc(ctypes.Structure):
    """tkg_gemm_desc: one GEMM of a list (device pointers, sizes, alpha)."""
    _fields_ = [("m", ctypes.c_int), ("n", ctypes.c_int), ("k", ctypes.c_int),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("sfa", ctypes.c_void_p), ("sfb", ctypes.c_void_p),
                ("tensor_scale_a", ctypes.c_void_p), ("tensor_scale_b", ctypes.c_void_p),
                ("D", ctypes.c_void_p), ("alpha", ctypes.c_float)]

_lock = threading.Lock()
_lib = None


class TkgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def load() -> ctypes.CDLL:
    """Load libtkg.so (raises if it has not been built)."""
    global _lib
    lib = _lib
    if lib is not None:   # loaded: no lock on the per-call path
        return lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m dense_block_scaled_gb300.build`")
            lib = ctypes.CDLL(LIB_PATH)
            i, vp, f, st = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_int
            lib.tkg_gemm_bf16.argtypes = [i, i, i, vp, vp, vp, f, vp]
            lib.tkg_gemm_bf16_noalloc.argtypes = [i, i, i, vp, vp, vp, f, vp]
            lib.tkg_gemm_mxfp8.argtypes = [i, i, i, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_gemm_nvfp4.argtypes = [i, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_bf16.argtypes = [i, vp, i, i, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_mxfp8.argtypes = [i, vp, i, i, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_nvfp4.argtypes = [i, vp, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_grouped_scale_bytes.argtypes = [i, vp, i, i]
            lib.tkg_grouped_scale_bytes.restype = ctypes.c_size_t
            lib.tkg_gemm_bf16_from_host.argtypes = [i, i, i, vp, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_dev_bf16.argtypes = [i, vp, i, i, i, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_dev_mxfp8.argtypes = [i, vp, i, i, i, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_dev_nvfp4.argtypes = [i, vp, i, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp]
            lib.tkg_grouped_dev_scale_bytes.argtypes = [i, i, i, i]
            lib.tkg_grouped_dev_scale_bytes.restype = ctypes.c_size_t
            for name in ("tkg_gemm_list_bf16", "tkg_gemm_list_mxfp8", "tkg_gemm_list_nvfp4"):
                getattr(lib, name).argtypes = [i, ctypes.POINTER(GemmDesc), vp]
                getattr(lib, name).restype = ctypes.c_int
            lib.tkg_gemm_bf16_strided.argtypes = [i, i, i, vp, i, vp, i, vp, i, f, vp]
            lib.tkg_gemm_mxfp8_strided.argtypes = [i, i, i, vp, i, vp, i, vp, vp, vp, i, f, vp]
            lib.tkg_gemm_nvfp4_strided.argtypes = [i, i, i, vp, i, vp, i, vp, vp, vp, vp, vp, i, f, vp]
            for name in ("tkg_gemm_bf16_strided", "tkg_gemm_mxfp8_strided", "tkg_gemm_nvfp4_strided"):
                getattr(lib, name).restype = ctypes.c_int
            sz = ctypes.c_size_t
            lib.tkg_linear_ce_loss.argtypes = [i, i, i, vp, i, vp, i, vp, f, vp, vp, vp, sz, vp]
            lib.tkg_linear_ce_loss_workspace_bytes.argtypes = [i, i]
            lib.tkg_linear_ce_grad.argtypes = [i, i, i, vp, i, vp, i, vp, f, vp, vp, vp, i, vp, i, i, i, vp, sz, vp]
            lib.tkg_linear_ce_grad_workspace_bytes.argtypes = [i, i, i, i]
            lib.tkg_gemm_grouped_dev_bf16_dgrad.argtypes = [i, vp, i, i, i, vp, vp, vp, f, vp]
            lib.tkg_gemm_grouped_dev_bf16_wgrad.argtypes = [i, vp, i, i, i, vp, vp, vp, i, f, vp]
            for name in ("tkg_linear_ce_loss", "tkg_linear_ce_grad", "tkg_gemm_grouped_dev_bf16_dgrad",
                         "tkg_gemm_grouped_dev_bf16_wgrad"):
                getattr(lib, name).restype = ctypes.c_int
            for name in ("tkg_linear_ce_loss_workspace_bytes", "tkg_linear_ce_grad_workspace_bytes"):
                getattr(lib, name).restype = sz
            lib.tkg_get_device_status.argtypes = [vp]
            lib.tkg_status_string.argtypes = [st]
            lib.tkg_status_string.restype = ctypes.c_char_p
            lib.tkg_scale_bytes.argtypes = [i, i, i]
            lib.tkg_scale_bytes.restype = ctypes.c_size_t
            lib.tkg_scales_to_tiled.argtypes = [i, i, vp, i, vp, vp]
            lib.tkg_quantize_mxfp8.argtypes = [i, i, vp, vp, vp, vp]
            lib.tkg_quantize_nvfp4.argtypes = [i, i, vp, vp, vp, vp, vp]
            lib.tkg_quantize_nvfp4_scaled.argtypes = [i, i, vp, vp, vp, vp, vp]
            lib.tkg_set_option.argtypes = [i, i]
            lib.tkg_get_option.argtypes = [i]
            for name in ("tkg_gemm_bf16", "tkg_gemm_bf16_noalloc", "tkg_gemm_mxfp8", "tkg_gemm_nvfp4", "tkg_get_device_status",
                         "tkg_scales_to_tiled", "tkg_quantize_mxfp8", "tkg_quantize_nvfp4",
                         "tkg_quantize_nvfp4_scaled", "tkg_set_option",
                         "tkg_get_option"):
                getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().tkg_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise TkgError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, dev=None):
    """The handle of `stream`, or of the current stream (of GPU `dev`, where the caller knows the current one)."""
    if stream is None:
        import torch
        # the current stream's handle without a Stream object (2.7 us less per call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------- raw C calls (pointers)

def gemm_bf16_raw(m, n, k, A, B, D, alpha, stream) -> int:
    return load().tkg_gemm_bf16(m, n, k, A, B, D, ctypes.c_float(alpha), stream)


def gemm_bf16_noalloc_raw(m, n, k, A, B, D, alpha, stream) -> int:
    return load().tkg_gemm_bf16_noalloc(m, n, k, A, B, D, ctypes.c_float(alpha), stream)


def gemm_mxfp8_raw(m, n, k, A, B, sfa, sfb, D, alpha, stream) -> int:
    return load().tkg_gemm_mxfp8(m, n, k, A, B, sfa, sfb, D, ctypes.c_float(alpha), stream)


def gemm_nvfp4_raw(m, n, k, A, B, sfa, sfb, ta, tb, D, alpha, stream) -> int:
    return load().tkg_gemm_nvfp4(m, n, k, A, B, sfa, sfb, ta, tb, D, ctypes.c_float(alpha), stream)


def _sizes(m_sizes):
    """Host int32 array of group sizes (kept alive by the caller's reference)."""
    arr = (ctypes.c_int * len(m_sizes))(*[int(x) for x in m_sizes])
    return arr, len(m_sizes)


def gemm_grouped_bf16_raw(groups, m_sizes, n, k, A, B, D, alpha, stream) -> int:
    return load().tkg_gemm_grouped_bf16(groups, m_sizes, n, k, A, B, D, ctypes.c_float(alpha), stream)


def gemm_grouped_mxfp8_raw(groups, m_sizes, n, k, A, B, sfa, sfb, D, alpha, stream) -> int:
    return load().tkg_gemm_grouped_mxfp8(groups, m_sizes, n, k, A, B, sfa, sfb, D, ctypes.c_float(alpha), stream)


def gemm_grouped_nvfp4_raw(groups, m_sizes, n, k, A, B, sfa, sfb, ta, tb, D, alpha, stream) -> int:
    return load().tkg_gemm_grouped_nvfp4(groups, m_sizes, n, k, A, B, sfa, sfb, ta, tb, D, ctypes.c_float(alpha),
                                         stream)


# ---------------------------------------------------------------- tensor helpers

def gemm_bf16(A, B, D, alpha: float = 1.0, stream=None) -> None:
    """D (m x n bf16) = alpha * A (m x k bf16) @ B (n x k bf16)^T."""
    m, k = A.shape
    n = B.shape[0]
    _check(gemm_bf16_raw(m, n, k, _ptr(A), _ptr(B), _ptr(D), alpha, _stream(stream)), "tkg_gemm_bf16")


def gemm_bf16_noalloc(A, B, D, alpha: float = 1.0, stream=None) -> None:
    """As gemm_bf16, through the entry point that allocates no device memory."""
    m, k = A.shape
    n = B.shape[0]
    _check(gemm_bf16_noalloc_raw(m, n, k, _ptr(A), _ptr(B), _ptr(D), alpha, _stream(stream)),
           "tkg_gemm_bf16_noalloc")


def gemm_mxfp8(A, B, sfa, sfb, D, alpha: float = 1.0, stream=None) -> None:
    """A (m x k uint8 E4M3), B (n x k), tiled E8M0 scales sfa / sfb (uint8)."""
    m, k = A.shape
    n = B.shape[0]
    _check(gemm_mxfp8_raw(m, n, k, _ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(D), alpha, _stream(stream)),
           "tkg_gemm_mxfp8")


def gemm_nvfp4(A, B, sfa, sfb, D, alpha: float = 1.0, ta=None, tb=None, stream=None) -> None:
    """A (m x k/2 uint8, packed E2M1), B (n x k/2), tiled UE4M3 scales, FP32 per-tensor scales ta / tb (device)."""
    m, kh = A.shape
    n = B.shape[0]
    _check(gemm_nvfp4_raw(m, n, 2 * kh, _ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(ta), _ptr(tb), _ptr(D),
                          alpha, _stream(stream)), "tkg_gemm_nvfp4")


def gemm_strided(fmt: str, m: int, n: int, k: int, A, lda: int, B, ldb: int, D, ldd: int, alpha: float = 1.0,
                 sfa=None, sfb=None, ta=None, tb=None, stream=None) -> None:
    """The GEMM on row-pitched views: lda / ldb in storage units (bf16 elements, or bytes of E4M3 / packed E2M1
    codes), ldd in bf16 elements; A, B, D are the first elements of the views."""
    lib = load()
    s = _stream(stream)
    if fmt == "bf16":
        st = lib.tkg_gemm_bf16_strided(m, n, k, _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldd, ctypes.c_float(alpha), s)
    elif fmt == "mxfp8":
        st = lib.tkg_gemm_mxfp8_strided(m, n, k, _ptr(A), lda, _ptr(B), ldb, _ptr(sfa), _ptr(sfb), _ptr(D), ldd,
                                        ctypes.c_float(alpha), s)
    else:
        st = lib.tkg_gemm_nvfp4_strided(m, n, k, _ptr(A), lda, _ptr(B), ldb, _ptr(sfa), _ptr(sfb), _ptr(ta), _ptr(tb),
                                        _ptr(D), ldd, ctypes.c_float(alpha), s)
    _check(st, f"tkg_gemm_{fmt}_strided")


def gemm_grouped_bf16(m_sizes, A, B, D, alpha: float = 1.0, stream=None) -> None:
    """Grouped: rows of A (sum(m_sizes) x k bf16) in consecutive groups, B (groups x n x k), D (sum x n)."""
    arr, g = _sizes(m_sizes)
    k = A.shape[-1]
    n = B.shape[-2]
    _check(gemm_grouped_bf16_raw(g, arr, n, k, _ptr(A), _ptr(B), _ptr(D), alpha, _stream(stream)),
           "tkg_gemm_grouped_bf16")


def gemm_grouped_mxfp8(m_sizes, A, B, sfa, sfb, D, alpha: float = 1.0, stream=None) -> None:
    """Grouped MXFP8: per-group tiled SFA buffers back to back, SFB one tiled buffer per group."""
    arr, g = _sizes(m_sizes)
    k = A.shape[-1]
    n = B.shape[-2]
    _check(gemm_grouped_mxfp8_raw(g, arr, n, k, _ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(D), alpha,
                                  _stream(stream)), "tkg_gemm_grouped_mxfp8")


def gemm_grouped_nvfp4(m_sizes, A, B, sfa, sfb, D, alpha: float = 1.0, ta=None, tb=None, stream=None) -> None:
    """Grouped NVFP4: ta one FP32 (device) for A, tb one FP32 per group (device)."""
    arr, g = _sizes(m_sizes)
    k = 2 * A.shape[-1]
    n = B.shape[-2]
    _check(gemm_grouped_nvfp4_raw(g, arr, n, k, _ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(ta), _ptr(tb),
                                  _ptr(D), alpha, _stream(stream)), "tkg_gemm_grouped_nvfp4")


def gemm_bf16_from_host(A_host, B_host, D_host, A_dev, B_dev, D_dev, alpha: float = 1.0, stream=None) -> None:
    """D_host = alpha * A_host @ B_host^T with host (pinned) operands; *_dev are device staging buffers."""
    m, k = A_host.shape
    n = B_host.shape[0]
    _check(load().tkg_gemm_bf16_from_host(m, n, k, _ptr(A_host), _ptr(B_host), _ptr(D_host), _ptr(A_dev),
                                          _ptr(B_dev), _ptr(D_dev), ctypes.c_float(alpha), _stream(stream)),
           "tkg_gemm_bf16_from_host")


def gemm_grouped_dev_bf16(sizes_dev, A, B, D, alpha: float = 1.0, stream=None) -> None:
    """Grouped BF16 GEMM with the group sizes in a device int32 tensor; A, D hold up to A.shape[0] rows."""
    g = sizes_dev.numel()
    _check(load().tkg_gemm_grouped_dev_bf16(g, _ptr(sizes_dev), A.shape[0], B.shape[-2], A.shape[-1], _ptr(A),
                                            _ptr(B), _ptr(D), ctypes.c_float(alpha), _stream(stream)),
           "tkg_gemm_grouped_dev_bf16")


def gemm_grouped_dev_mxfp8(sizes_dev, A, B, sfa, sfb, D, alpha: float = 1.0, stream=None) -> None:
    g = sizes_dev.numel()
    _check(load().tkg_gemm_grouped_dev_mxfp8(g, _ptr(sizes_dev), A.shape[0], B.shape[-2], A.shape[-1], _ptr(A),
                                             _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(D), ctypes.c_float(alpha),
                                             _stream(stream)), "tkg_gemm_grouped_dev_mxfp8")


def gemm_grouped_dev_nvfp4(sizes_dev, A, B, sfa, sfb, D, alpha: float = 1.0, ta=None, tb=None, stream=None) -> None:
    g = sizes_dev.numel()
    _check(load().tkg_gemm_grouped_dev_nvfp4(g, _ptr(sizes_dev), A.shape[0], B.shape[-2], 2 * A.shape[-1], _ptr(A),
                                             _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(ta), _ptr(tb), _ptr(D),
                                             ctypes.c_float(alpha), _stream(stream)), "tkg_gemm_grouped_dev_nvfp4")


def gemm_list_raw(fmt: str, descs, stream) -> int:
    """tkg_gemm_list_<fmt> on a sequence of GemmDesc."""
    arr = (GemmDesc * max(len(descs), 1))(*descs)
    return getattr(load(), f"tkg_gemm_list_{fmt}")(len(descs), arr, stream)


def gemm_desc(fmt: str, A, B, D, alpha: float = 1.0, sfa=None, sfb=None, ta=None, tb=None) -> GemmDesc:
    """Descriptor of one GEMM from its device tensors (A: m x k, or m x k/2 bytes for NVFP4)."""
    m = A.shape[0]
    k = 2 * A.shape[1] if fmt == "nvfp4" else A.shape[1]
    return GemmDesc(m, B.shape[0], k, _ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(ta), _ptr(tb), _ptr(D),
                    float(alpha))


def gemm_list(fmt: str, descs, stream=None) -> None:
    """Several independent GEMMs (GemmDesc each, at most MAX_LIST) in one launch."""
    _check(gemm_list_raw(fmt, descs, _stream(stream)), f"tkg_gemm_list_{fmt}")


# ---------------------------------------------------------------- training-side operators
# These check the tensors they are given (one combined test on the way through,
# the reason looked for only when it fails) and may take their workspace from
# torch's allocator.  A small call is bound by this host work, so it is kept short.

def _wrong(name, t, dtype, shape, pitched):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        return f"{name}: {dtype} of shape {tuple(shape)} is wanted, got {t.dtype} {tuple(t.shape)}"
    if max(shape) >> 31 or (len(shape) == 2 and shape[0] > 1 and t.stride(0) >> 31):
        return f"{name}: sizes and row pitches below 2^31 are wanted, got {tuple(shape)} in strides {t.stride()}"
    if pitched and len(shape) == 2 and (shape[1] <= 1 or t.stride(1) == 1):
        return None
    if not t.is_contiguous():
        return f"{name}: a {'matrix with contiguous rows' if pitched else 'contiguous tensor'} is wanted"
    return None


def _refuse(wanted):
    """Raises ValueError for the first of (name, tensor, dtype, shape, rows may be pitched) that does not hold, or that
    is not on the current GPU: an address of the host's, or of another GPU, would reach the kernel as one of this."""
    for w in wanted:
        msg = _wrong(*w)
        if msg:
            raise ValueError(msg)
    _off_gpu([(w[0], w[1]) for w in wanted])


def _off_gpu(named):
    for name, t in named:
        if t.get_device() < 0:
            raise ValueError(f"{name}: a tensor on the GPU is wanted, got one on {t.device}")
    import torch
    for name, t in named:
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name}: on {t.device}, but the current GPU is cuda:{torch.cuda.current_device()}")


_kept = threading.local()    # per thread: {device: workspace} for the default stream
_KEEP_BYTES = 16 << 20


def _workspace(workspace, nbytes, like, stream, handle):
    """(address, bytes, tensor to keep until the call is made) of the caller's workspace, or of one of torch's.

    On the default stream small ones are kept per thread and device (asking torch's allocator costs 6 us while work is
    queued): calls of one thread follow one another there, and that stream is never captured into a graph.  Elsewhere
    each call takes its own; on another stream than the current one it is tied to the work queued there."""
    import torch
    if workspace is not None:
        if workspace.get_device() != like.get_device():
            _off_gpu([("workspace", workspace)])
        if not workspace.is_contiguous():
            raise ValueError("workspace: a contiguous tensor is wanted")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    small = stream is None and nbytes <= _KEEP_BYTES and handle == 0
    if small:
        kept = _kept.__dict__.get(like.get_device())
        if kept is not None and kept[1] >= nbytes:
            return kept
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    if small:
        kept = _kept.__dict__[like.get_device()] = (workspace.data_ptr(), nbytes, workspace)
        return kept
    if stream is not None:
        s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
        if s != torch.cuda.current_stream():
            # the memory may have been used by work of the current stream, and must outlive that of `stream`
            s.wait_stream(torch.cuda.current_stream())
            workspace.record_stream(s)
    return workspace.data_ptr(), nbytes, workspace


def _pitch(t, width):
    """Row pitch in elements of a checked matrix (a single row's stride says nothing)."""
    return t.stride(0) if t.size(0) > 1 else width


@functools.lru_cache(maxsize=256)   # (a ctypes call costs 0.6 us)
def linear_ce_loss_workspace_bytes(tokens: int, vocab: int) -> int:
    return int(load().tkg_linear_ce_loss_workspace_bytes(tokens, vocab))


def linear_ce_loss(X, W, labels, loss, lse, alpha: float = 1.0, workspace=None, stream=None) -> None:
    """Softmax cross entropy of the head alpha * X @ W^T: loss and log-sum-exp per token (FP32), logits never kept.

    X (tokens x hidden bf16), W (vocab x hidden bf16), rows may be pitched; labels int64, outside [0, vocab): ignored."""
    import torch
    (tokens, hidden), vocab, row, dev = X.shape, W.shape[0], labels.shape, X.get_device()
    if not (-1 < dev == torch.cuda.current_device() == W.get_device() == labels.get_device() == loss.get_device()
            == lse.get_device() and not (tokens | vocab | hidden) >> 31
            and X.dtype is W.dtype is torch.bfloat16 and labels.dtype is torch.int64
            and loss.dtype is lse.dtype is torch.float32 and W.shape[1] == hidden and row == loss.shape == lse.shape
            and row == (tokens,) and X.is_contiguous() and W.is_contiguous() and labels.is_contiguous()
            and loss.is_contiguous() and lse.is_contiguous()):
        _refuse((("X", X, torch.bfloat16, (tokens, hidden), True), ("W", W, torch.bfloat16, (vocab, hidden), True),
                 ("labels", labels, torch.int64, (tokens,), False), ("loss", loss, torch.float32, (tokens,), False),
                 ("lse", lse, torch.float32, (tokens,), False)))
    lib, handle = load(), _stream(stream, dev)
    at, nbytes, _keep = _workspace(workspace, linear_ce_loss_workspace_bytes(tokens, vocab), X, stream, handle)
    _check(lib.tkg_linear_ce_loss(tokens, vocab, hidden, X.data_ptr(), _pitch(X, hidden), W.data_ptr(),
                                  _pitch(W, hidden), labels.data_ptr(), alpha, loss.data_ptr(), lse.data_ptr(), at,
                                  nbytes, handle), "tkg_linear_ce_loss")


def linear_ce_grad_workspace_bytes(tokens: int, vocab: int, hidden: int, piece: int = 0) -> int:
    return int(load().tkg_linear_ce_grad_workspace_bytes(tokens, vocab, hidden, piece))


def _grad_type(t, name, accumulate):
    import torch
    if t.dtype is torch.bfloat16 and not accumulate:
        return GRAD_BF16
    if t.dtype is not torch.float32:
        raise ValueError(f"{name}: bfloat16, or float32 (the type that can accumulate) is wanted, got {t.dtype}")
    return GRAD_F32_ADD if accumulate else GRAD_F32


def linear_ce_grad(X, W, labels, lse, dloss, dX, dW, alpha: float = 1.0, accumulate: bool = False, piece: int = 0,
                   workspace=None, stream=None) -> None:
    """Gradient of sum(dloss * loss): dX (tokens x hidden bf16) and dW (vocab x hidden, bf16 or float32); either may
    be None.  accumulate: add to the float32 dW.  piece: vocabulary entries worked on at a time (0: chosen)."""
    import torch
    (tokens, hidden), vocab, row, dev = X.shape, W.shape[0], labels.shape, X.get_device()
    gtype = GRAD_BF16 if dW is None else _grad_type(dW, "dW", accumulate)
    if not (-1 < dev == torch.cuda.current_device() == W.get_device() == labels.get_device() == lse.get_device()
            == dloss.get_device() and not (tokens | vocab | hidden) >> 31
            and X.dtype is W.dtype is torch.bfloat16 and labels.dtype is torch.int64
            and lse.dtype is dloss.dtype is torch.float32 and W.shape[1] == hidden and row == lse.shape == dloss.shape
            and row == (tokens,) and X.is_contiguous() and W.is_contiguous() and labels.is_contiguous()
            and lse.is_contiguous() and dloss.is_contiguous()
            and (dX is None or (dX.dtype is torch.bfloat16 and dX.shape == X.shape and dX.is_contiguous()
                                and dX.get_device() == dev))
            and (dW is None or (dW.shape == W.shape and dW.is_contiguous() and dW.get_device() == dev))):
        wanted = [("X", X, torch.bfloat16, (tokens, hidden), True), ("W", W, torch.bfloat16, (vocab, hidden), True),
                  ("labels", labels, torch.int64, (tokens,), False), ("lse", lse, torch.float32, (tokens,), False),
                  ("dloss", dloss, torch.float32, (tokens,), False)]
        if dX is not None:
            wanted.append(("dX", dX, torch.bfloat16, (tokens, hidden), True))
        if dW is not None:
            wanted.append(("dW", dW, dW.dtype, (vocab, hidden), True))
        _refuse(wanted)
    lib, handle = load(), _stream(stream, dev)
    at, nbytes, _keep = _workspace(workspace, lib.tkg_linear_ce_grad_workspace_bytes(tokens, vocab, hidden, piece), X,
                                   stream, handle)
    _check(lib.tkg_linear_ce_grad(tokens, vocab, hidden, X.data_ptr(), _pitch(X, hidden), W.data_ptr(),
                                  _pitch(W, hidden), labels.data_ptr(), alpha, lse.data_ptr(), dloss.data_ptr(),
                                  _ptr(dX), 0 if dX is None else _pitch(dX, hidden), _ptr(dW),
                                  0 if dW is None else _pitch(dW, hidden), gtype, piece, at, nbytes,
                                  handle), "tkg_linear_ce_grad")


def gemm_grouped_dev_bf16_dgrad(sizes_dev, dD, B, dA, alpha: float = 1.0, stream=None) -> None:
    """Gradient of gemm_grouped_dev_bf16 to its rows: dA (capacity x k) = alpha * dD (capacity x n) @ B_g (n x k)."""
    import torch
    groups, (cap, n), k, dev = sizes_dev.shape[0], dD.shape, B.shape[-1], dD.get_device()
    if not (-1 < dev == torch.cuda.current_device() == sizes_dev.get_device() == B.get_device() == dA.get_device()
            and not (cap | n | k) >> 31
            and dD.dtype is B.dtype is dA.dtype is torch.bfloat16 and sizes_dev.dtype is torch.int32
            and sizes_dev.dim() == 1 and B.shape == (groups, n, k) and dA.shape == (cap, k) and dD.is_contiguous()
            and B.is_contiguous() and dA.is_contiguous() and sizes_dev.is_contiguous()):
        _refuse((("sizes_dev", sizes_dev, torch.int32, (groups,), False), ("dD", dD, torch.bfloat16, (cap, n), False),
                 ("B", B, torch.bfloat16, (groups, n, k), False), ("dA", dA, torch.bfloat16, (cap, k), False)))
    _check(load().tkg_gemm_grouped_dev_bf16_dgrad(groups, sizes_dev.data_ptr(), cap, n, k, dD.data_ptr(),
                                                  B.data_ptr(), dA.data_ptr(), alpha, _stream(stream, dev)),
           "tkg_gemm_grouped_dev_bf16_dgrad")


def gemm_grouped_dev_bf16_wgrad(sizes_dev, dD, A, dB, alpha: float = 1.0, accumulate: bool = False, stream=None) -> None:
    """Gradient of gemm_grouped_dev_bf16 to the experts: dB_g (n x k, bf16 or float32) = alpha * dD_g^T @ A_g.
    accumulate: add to the float32 dB."""
    import torch
    groups, (cap, n), k, dev = sizes_dev.shape[0], dD.shape, A.shape[-1], dD.get_device()
    gtype = _grad_type(dB, "dB", accumulate)
    if not (-1 < dev == torch.cuda.current_device() == sizes_dev.get_device() == A.get_device() == dB.get_device()
            and not (cap | n | k) >> 31
            and dD.dtype is A.dtype is torch.bfloat16 and sizes_dev.dtype is torch.int32 and sizes_dev.dim() == 1
            and A.shape == (cap, k) and dB.shape == (groups, n, k) and dD.is_contiguous() and A.is_contiguous()
            and dB.is_contiguous() and sizes_dev.is_contiguous()):
        _refuse((("sizes_dev", sizes_dev, torch.int32, (groups,), False), ("dD", dD, torch.bfloat16, (cap, n), False),
                 ("A", A, torch.bfloat16, (cap, k), False), ("dB", dB, dB.dtype, (groups, n, k), False)))
    _check(load().tkg_gemm_grouped_dev_bf16_wgrad(groups, sizes_dev.data_ptr(), cap, n, k, dD.data_ptr(),
                                                  A.data_ptr(), dB.data_ptr(), gtype, alpha, _stream(stream, dev)),
           "tkg_gemm_grouped_dev_bf16_wgrad")


def grouped_dev_scale_bytes(groups: int, m_capacity: int, k: int, block: int) -> int:
    return int(load().tkg_grouped_dev_scale_bytes(groups, m_capacity, k, block))


def grouped_scale_bytes(m_sizes, k: int, block: int) -> int:
    arr, g = _sizes(m_sizes)
    return int(load().tkg_grouped_scale_bytes(g, arr, k, block))


def scale_bytes(rows: int, k: int, block: int) -> int:
    return int(load().tkg_scale_bytes(rows, k, block))


def scales_to_tiled(src, dst, kblocks: int | None = None, stream=None) -> None:
    rows, ld = src.shape
    kb = ld if kblocks is None else kblocks
    _check(load().tkg_scales_to_tiled(rows, kb, _ptr(src), ld, _ptr(dst), _stream(stream)), "tkg_scales_to_tiled")


def quantize_mxfp8(X, Q, sf, stream=None) -> None:
    rows, k = X.shape
    _check(load().tkg_quantize_mxfp8(rows, k, _ptr(X), _ptr(Q), _ptr(sf), _stream(stream)), "tkg_quantize_mxfp8")


def quantize_nvfp4(X, Q, sf, tensor_scale, stream=None) -> None:
    rows, k = X.shape
    _check(load().tkg_quantize_nvfp4(rows, k, _ptr(X), _ptr(Q), _ptr(sf), _ptr(tensor_scale), _stream(stream)),
           "tkg_quantize_nvfp4")


def quantize_nvfp4_scaled(X, Q, sf, tensor_scale, stream=None) -> None:
    """NVFP4 codes and tiled scales of X with the given FP32 tensor scale (device, one element, read only)."""
    rows, k = X.shape
    _check(load().tkg_quantize_nvfp4_scaled(rows, k, _ptr(X), _ptr(Q), _ptr(sf), _ptr(tensor_scale),
                                            _stream(stream)), "tkg_quantize_nvfp4_scaled")


def device_status(stream=None) -> int:
    return int(load().tkg_get_device_status(_stream(stream)))


def set_option(option: int, value: int) -> None:
    _check(load().tkg_set_option(option, value), "tkg_set_option")


def get_option(option: int) -> int:
    return int(load().tkg_get_option(option))
