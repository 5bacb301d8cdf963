"""libkmassign: the k-means assignment step on one NVIDIA GB300 (sm_103a).

For points X[N, D] and centroids C[K, D] (bf16), returns

    idx[i] = argmin_j (||c_j||^2 - 2 x_i . c_j)      (lowest j on ties)

(flashlib PR #22 "Optimize Blackwell k-means assignment reduction",
Summary).  Every step runs in the CUDA kernels of ``libkmassign.so``; this
module only marshals torch tensors into the C ABI declared in
``include/kmassign.h`` and raises on error codes.  There is no CPU path: if
the shared library is missing, every call raises.
"""

from __future__ import annotations

import array
import ctypes
import os
import threading

import torch

from . import _build

__all__ = [
    "KmassignError", "library", "library_path", "kmassign", "kmassign_ex", "kmassign_norms",
    "kmassign_noalloc", "kmassign_set_wait_timeout", "shard_rows", "kmassign_update",
    "kmassign_centroids", "kmassign_lloyd",
    "kmassign_plan", "kmassign_plan_for", "kmassign_check", "kmassign_strerror", "assign", "norms", "assign_host",
    "kmassign_route", "kmassign_route_grad", "kmassign_lists", "kmassign_lookup",
    "kmassign_lookup_grad", "kmassign_grad_norm", "kmassign_clip",
    "kmassign_experts", "kmassign_experts_grad", "kmassign_rmsnorm", "kmassign_rmsnorm_grad",
    "STATUS",
]

STATUS = {
    "KMASSIGN_OK": 0,
    "KMASSIGN_ERR_NULL": -1,
    "KMASSIGN_ERR_ALIGN": -2,
    "KMASSIGN_ERR_SHAPE": -3,
    "KMASSIGN_ERR_UNSUPPORTED_D": -4,
    "KMASSIGN_ERR_CUDA": -5,
    "KMASSIGN_ERR_TIMEOUT": -6,
    "KMASSIGN_ERR_NOT_DEVICE": -7,
    "KMASSIGN_ERR_ARG": -8,
    "KMASSIGN_ERR_SCRATCH": -9,
    "KMASSIGN_ERR_NOT_HOST": -10,
    "KMASSIGN_ERR_DEBUG_CHECK": -11,
}
_NAMES = {v: k for k, v in STATUS.items()}

_lock = threading.Lock()
_lib = None


class KmassignError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {_NAMES.get(code, code)} ({kmassign_strerror(code)})")


def library_path() -> str:
    return _build.LIB_PATH


def _declare(lib):
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.kmassign_norms.argtypes = [vp, i64, i64, vp, vp]
    lib.kmassign_norms.restype = i32
    lib.kmassign.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.kmassign.restype = i32
    lib.kmassign_ex.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, i32, i32, i32, i32, vp]
    lib.kmassign_ex.restype = i32
    lib.kmassign_host.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.kmassign_host.restype = i32
    lib.kmassign_host_ex.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, i64, vp]
    lib.kmassign_host_ex.restype = i32
    lib.kmassign_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.kmassign_noalloc.restype = i32
    lib.kmassign_plan.argtypes = [i64, i64, i64, vp]
    lib.kmassign_plan.restype = i32
    lib.kmassign_plan_ex.argtypes = [i64, i64, i64, i32, i32, i32, i32, vp]
    lib.kmassign_plan_ex.restype = i32
    lib.kmassign_plan_for.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32, i32, vp]
    lib.kmassign_plan_for.restype = i32
    lib.kmassign_update.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp]
    lib.kmassign_update.restype = i32
    lib.kmassign_update_ex.argtypes = [vp, vp, i64, i64, i64, vp, vp, i32, vp]
    lib.kmassign_update_ex.restype = i32
    lib.kmassign_centroids.argtypes = [vp, vp, vp, i64, i64, vp, vp, vp]
    lib.kmassign_centroids.restype = i32
    lib.kmassign_lloyd.argtypes = [vp, vp, i64, i64, i64, i32, vp, vp]
    lib.kmassign_lloyd.restype = i32
    lib.kmassign_topk.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, i32, vp]
    lib.kmassign_topk.restype = i32
    lib.kmassign_topk_ex.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, i32, i32, vp]
    lib.kmassign_topk_ex.restype = i32
    f32 = ctypes.c_float
    lib.kmassign_route.argtypes = [vp, i32, i64, i64, i32, i32, vp, i32, i32, i32, i32, f32, vp,
                                   vp, vp]
    lib.kmassign_route.restype = i32
    lib.kmassign_route_grad.argtypes = [vp, i32, i64, i64, i32, i32, i32, f32, vp, vp, vp, vp]
    lib.kmassign_route_grad.restype = i32
    lib.kmassign_lists.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.kmassign_lists.restype = i32
    lib.kmassign_lookup.argtypes = [vp, i32, i64, i64, vp, vp, i64, i32, f32, vp, vp]
    lib.kmassign_lookup.restype = i32
    lib.kmassign_lookup_grad.argtypes = [vp, i32, vp, vp, vp, i64, i32, i64, i64, f32, i32, i32,
                                         vp, i32, vp, vp]
    lib.kmassign_lookup_grad.restype = i32
    lib.kmassign_grad_norm.argtypes = [vp, vp, vp, i32, vp, vp]
    lib.kmassign_grad_norm.restype = i32
    lib.kmassign_clip.argtypes = [vp, vp, vp, vp, i32, f32, vp, vp]
    lib.kmassign_clip.restype = i32
    lib.kmassign_experts.argtypes = [vp, i32, i64, i64, vp, i64, i64, vp, vp, vp, i64, vp, i32, vp,
                                     vp, i32, i64, vp]
    lib.kmassign_experts.restype = i32
    lib.kmassign_experts_grad.argtypes = [vp, i32, i64, i64, vp, i64, i64, vp, i64, vp, i64, vp,
                                          i32, vp, vp, vp, i32, vp]
    lib.kmassign_experts_grad.restype = i32
    lib.kmassign_rmsnorm.argtypes = [vp, i32, i64, i64, vp, vp, i32, f32, vp, vp, i32, vp, vp, vp]
    lib.kmassign_rmsnorm.restype = i32
    lib.kmassign_rmsnorm_grad.argtypes = [vp, i32, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp]
    lib.kmassign_rmsnorm_grad.restype = i32
    lib.kmassign_set_wait_timeout.argtypes = [ctypes.c_uint64]
    lib.kmassign_set_wait_timeout.restype = i32
    lib.kmassign_check.argtypes = [vp]
    lib.kmassign_check.restype = i32
    lib.kmassign_strerror.argtypes = [i32]
    lib.kmassign_strerror.restype = ctypes.c_char_p
    return lib


def library(path: str | None = None):
    """The loaded libkmassign (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or library_path()
            if not os.path.exists(p):
                raise RuntimeError(
                    f"libkmassign.so not found at {p}; build it with "
                    "`python -m means_nearest_centroid_gb300._build` (there is no CPU fallback)")
            _lib = _declare(ctypes.CDLL(p))
        return _lib


def kmassign_strerror(code: int) -> str:
    return library().kmassign_strerror(int(code)).decode()


def _check(code: int, where: str):
    if code != 0:
        raise KmassignError(code, where)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, device=None) -> int:
    """The cudaStream_t to launch on: ``stream``, else the current stream of
    ``device`` (the tensors' device), else of the current device."""
    if stream is None:
        if _raw_stream is not None:
            idx = torch.cuda.current_device() if device is None else device.index
            return _raw_stream(idx)
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _new(shape, dtype, device, stream, make=torch.empty):
    """An output of a call on ``stream`` (None: the current one), whose memory that stream owns.

    The caching allocator hands out again at once what was freed on the current
    stream, while work enqueued there may still read it; another stream must not
    write there before that work is done (nor start before ``make`` has).
    """
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(t, name, dtype):
    # the common case in one expression; the detail only on failure
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def kmassign_norms(C: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """cnorm[j] = ||c_j||^2 (fp32) on the GPU."""
    _need_cuda(C, "C", torch.bfloat16)
    K, D = C.shape
    if out is None:
        out = _new(K, torch.float32, C.device, stream)
    _need_cuda(out, "out", torch.float32)
    _check(library().kmassign_norms(_ptr(C), K, D, _ptr(out), _stream_ptr(stream, C.device)),
           "kmassign_norms")
    return out


def kmassign_ex(X, C, cnorm=None, idx=None, minscore=None, ksplit: int = 0,
                rows_per_cta: int = 0, centroids_per_tile: int = 0, consumer_warps: int = 0,
                stream=None):
    """Assignment with an explicit plan (0 = automatic).  Returns idx (int32)."""
    _need_cuda(X, "X", torch.bfloat16)
    _need_cuda(C, "C", torch.bfloat16)
    N, D = X.shape
    K, D2 = C.shape
    if D != D2:
        raise ValueError("X and C disagree on D")
    if cnorm is not None:
        _need_cuda(cnorm, "cnorm", torch.float32)
    if idx is None:
        idx = _new(N, torch.int32, X.device, stream)
    _need_cuda(idx, "idx", torch.int32)
    if minscore is not None:
        _need_cuda(minscore, "minscore", torch.float32)
    rc = library().kmassign_ex(_ptr(X), _ptr(C), _ptr(cnorm), N, K, D, _ptr(idx), _ptr(minscore),
                               int(ksplit), int(rows_per_cta), int(centroids_per_tile),
                               int(consumer_warps), _stream_ptr(stream, X.device))
    _check(rc, "kmassign_ex")
    return idx


def kmassign(X, C, cnorm=None, idx=None, minscore=None, stream=None):
    """idx[i] = argmin_j (||c_j||^2 - 2 x_i . c_j) on the GPU; returns idx."""
    _need_cuda(X, "X", torch.bfloat16)
    _need_cuda(C, "C", torch.bfloat16)
    N, D = X.shape
    K, D2 = C.shape
    if D != D2:
        raise ValueError("X and C disagree on D")
    if cnorm is not None:
        _need_cuda(cnorm, "cnorm", torch.float32)
    if idx is None:
        idx = _new(N, torch.int32, X.device, stream)
    _need_cuda(idx, "idx", torch.int32)
    if minscore is not None:
        _need_cuda(minscore, "minscore", torch.float32)
    rc = library().kmassign(_ptr(X), _ptr(C), _ptr(cnorm), N, K, D, _ptr(idx), _ptr(minscore),
                            _stream_ptr(stream, X.device))
    _check(rc, "kmassign")
    return idx


def kmassign_noalloc(X, C, cnorm=None, idx=None, minscore=None, stream=None):
    """kmassign for callers that cannot let the library allocate device memory.

    The library's temporaries come from its static device array instead of
    the stream allocator (see ``include/kmassign.h``).  ``idx`` should be
    passed preallocated by such callers; it is allocated here only for
    convenience.  Calls that overlap on the GPU share that array and race.
    """
    _need_cuda(X, "X", torch.bfloat16)
    _need_cuda(C, "C", torch.bfloat16)
    N, D = X.shape
    K, D2 = C.shape
    if D != D2:
        raise ValueError("X and C disagree on D")
    if cnorm is not None:
        _need_cuda(cnorm, "cnorm", torch.float32)
    if idx is None:
        idx = _new(N, torch.int32, X.device, stream)
    _need_cuda(idx, "idx", torch.int32)
    if minscore is not None:
        _need_cuda(minscore, "minscore", torch.float32)
    rc = library().kmassign_noalloc(_ptr(X), _ptr(C), _ptr(cnorm), N, K, D, _ptr(idx),
                                    _ptr(minscore), _stream_ptr(stream, X.device))
    _check(rc, "kmassign_noalloc")
    return idx


def kmassign_topk(X, C, k: int, cnorm=None, idx=None, score=None, distances: bool = False,
                  with_score: bool = True, ksplit: int = 0, stream=None):
    """The k nearest centroids of every point: (idx int32 [N, k], score fp32 [N, k]).

    Row i lists centroids in ascending score s_ij = ||c_j||^2 - 2 x_i . c_j
    (lowest index first on ties); ``distances`` returns ||x_i||^2 + s_ij
    instead.  ``score`` is None when ``with_score`` is false and no output
    tensor is given.  ``ksplit`` forces a split of the centroid axis (0 =
    automatic; see ``kmassign_topk_ex`` in ``include/kmassign.h``).
    """
    _need_cuda(X, "X", torch.bfloat16)
    _need_cuda(C, "C", torch.bfloat16)
    N, D = X.shape
    K, D2 = C.shape
    if D != D2:
        raise ValueError("X and C disagree on D")
    if cnorm is not None:
        _need_cuda(cnorm, "cnorm", torch.float32)
    k = int(k)
    if idx is None:
        idx = _new((N, max(k, 0)), torch.int32, X.device, stream)
    _need_cuda(idx, "idx", torch.int32)
    if score is None and (with_score or distances):
        score = _new((N, max(k, 0)), torch.float32, X.device, stream)
    if score is not None:
        _need_cuda(score, "score", torch.float32)
    lib = library()
    if ksplit:
        rc = lib.kmassign_topk_ex(_ptr(X), _ptr(C), _ptr(cnorm), N, K, D, k, _ptr(idx),
                                  _ptr(score), int(bool(distances)), int(ksplit),
                                  _stream_ptr(stream, X.device))
    else:
        rc = lib.kmassign_topk(_ptr(X), _ptr(C), _ptr(cnorm), N, K, D, k, _ptr(idx), _ptr(score),
                               int(bool(distances)), _stream_ptr(stream, X.device))
    _check(rc, "kmassign_topk")
    return idx, score


def kmassign_plan(N: int, K: int, D: int, ksplit: int = 0, rows_per_cta: int = 0,
                  centroids_per_tile: int = 0, consumer_warps: int = 0) -> dict:
    """The plan kmassign (or, with forcing arguments, kmassign_ex) would run."""
    out = (ctypes.c_int32 * 9)()
    _check(library().kmassign_plan_ex(int(N), int(K), int(D), int(ksplit), int(rows_per_cta),
                                      int(centroids_per_tile), int(consumer_warps),
                                      ctypes.cast(out, ctypes.c_void_p)),
           "kmassign_plan")
    keys = ["ksplit", "rows_per_cta", "centroids_per_tile", "grid", "stages", "xbufs",
            "whole_row_tiles", "split_row_tiles", "consumer_warps"]
    return dict(zip(keys, list(out)))


def kmassign_plan_for(N: int, K: int, D: int, sms: int = 152, smem_per_block: int = 232448,
                      pair_clusters: int = 76, ksplit: int = 0, rows_per_cta: int = 0,
                      centroids_per_tile: int = 0, consumer_warps: int = 0) -> dict:
    """The plan for a described device (default: a GB300); needs no GPU."""
    out = (ctypes.c_int32 * 9)()
    _check(library().kmassign_plan_for(int(N), int(K), int(D), int(sms), int(smem_per_block),
                                       int(pair_clusters), int(ksplit), int(rows_per_cta),
                                       int(centroids_per_tile), int(consumer_warps),
                                       ctypes.cast(out, ctypes.c_void_p)),
           "kmassign_plan_for")
    keys = ["ksplit", "rows_per_cta", "centroids_per_tile", "grid", "stages", "xbufs",
            "whole_row_tiles", "split_row_tiles", "consumer_warps"]
    return dict(zip(keys, list(out)))


def kmassign_update(X, idx, K: int, sums=None, counts=None, method: int = 0, stream=None):
    """Per-centroid fp32 sums [K, D] and int32 counts [K] of X's rows by idx.

    When sums/counts are given they are accumulated into; otherwise zeroed
    tensors are created.  ``method``: 0 automatic, 1 atomic, 2 sorted (see
    ``kmassign_update_ex`` in ``include/kmassign.h``).  Returns (sums, counts).
    """
    _need_cuda(X, "X", torch.bfloat16)
    _need_cuda(idx, "idx", torch.int32)
    N, D = X.shape
    if idx.shape != (N,):
        raise ValueError("idx must hold one id per point")
    if sums is None:
        sums = _new((K, D), torch.float32, X.device, stream, torch.zeros)
    if counts is None:
        counts = _new(K, torch.int32, X.device, stream, torch.zeros)
    _need_cuda(sums, "sums", torch.float32)
    _need_cuda(counts, "counts", torch.int32)
    _check(library().kmassign_update_ex(_ptr(X), _ptr(idx), N, int(K), D, _ptr(sums),
                                        _ptr(counts), int(method),
                                        _stream_ptr(stream, X.device)),
           "kmassign_update")
    return sums, counts


def kmassign_centroids(sums, counts, C_old, C_new=None, means=None, stream=None):
    """bf16 means of the assigned points (C_old where a centroid has none)."""
    _need_cuda(sums, "sums", torch.float32)
    _need_cuda(counts, "counts", torch.int32)
    _need_cuda(C_old, "C_old", torch.bfloat16)
    K, D = C_old.shape
    if C_new is None:
        C_new = _new((K, D), torch.bfloat16, C_old.device, stream)
    _need_cuda(C_new, "C_new", torch.bfloat16)
    if means is not None:
        _need_cuda(means, "means", torch.float32)
    _check(library().kmassign_centroids(_ptr(sums), _ptr(counts), _ptr(C_old), K, D, _ptr(C_new),
                                        _ptr(means), _stream_ptr(stream, sums.device)),
           "kmassign_centroids")
    return C_new


def kmassign_lloyd(X, C, iters: int, idx=None, stream=None):
    """``iters`` Lloyd iterations on the GPU, updating C (bf16) in place.

    Returns idx, the last assignment (made before the last update).
    """
    _need_cuda(X, "X", torch.bfloat16)
    _need_cuda(C, "C", torch.bfloat16)
    N, D = X.shape
    K = C.shape[0]
    if idx is None:
        idx = _new(N, torch.int32, X.device, stream)
    _need_cuda(idx, "idx", torch.int32)
    _check(library().kmassign_lloyd(_ptr(X), _ptr(C), N, K, D, int(iters), _ptr(idx),
                                    _stream_ptr(stream, X.device)), "kmassign_lloyd")
    return idx


# ---- learned assignments: routing, lookup, inverted lists, clipping ----------
#
# These calls are not recorded by autograd.  In grad mode they refuse inputs that
# require grad (but for the bias, which the weights do not depend on), and in any
# mode inputs with a forward-mode tangent.

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}


def _need_float(t, name) -> int:
    """The kmassign_dtype of a contiguous CUDA tensor of a supported type."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous():
        code = _DTYPES.get(t.dtype)
        if code is not None:
            return code
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _need_detached(where, name):
    """In grad mode, raises for an input that requires grad: no result is part of autograd's graph."""
    if torch.is_grad_enabled():
        raise RuntimeError(
            f"{where}: {name} requires grad, and autograd would not see the result; call it "
            "under torch.no_grad() or in a torch.autograd.Function (gradients: "
            "kmassign_route_grad, kmassign_lookup_grad, kmassign_experts_grad, "
            "kmassign_rmsnorm_grad)")


_forward_ad = torch.autograd.forward_ad


def _need_no_tangent(where, *tensors):
    """Raises for an input with a forward-mode tangent (also under no_grad, where torch keeps them)."""
    if getattr(_forward_ad, "_current_level", 0) < 0:   # the common case: no forward mode
        return
    for t in tensors:
        if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(
                f"{where}: an input carries a forward-mode tangent, and the result would carry "
                "none; call it with the primal or in a torch.autograd.Function with a jvp")


# Tells autograd that a call wrote to these tensors of the caller, as torch's in-place operations
# do: a backward pass that has saved one raises.
_written = torch.autograd.graph.increment_version


def _need_shape(t, name, shape):
    if t.shape != shape:   # a torch.Size is a tuple
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _stream_of(stream, t) -> int:
    """The cudaStream_t to launch on: ``stream``, else the current one of t's device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _stream_ptr(stream, t.device)


def _score_code(score) -> int:
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return code


def _need_matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    return t.shape


def _need_ids(idx):
    """N and k of ids [N] (one a point) or [N, k]."""
    _need_cuda(idx, "idx", torch.int32)
    if idx.dim() == 1:
        return idx.shape[0], 1
    if idx.dim() == 2:
        return idx.shape
    raise ValueError(f"idx must have one or two dimensions, got {idx.dim()}")


def kmassign_route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1,
                   topk_groups: int | None = None, group_top: int = 2, renorm: bool = True,
                   scale: float = 1.0, idx=None, weights=None, stream=None):
    """The k experts (rows) of every point: (idx int32 [N, k], weights fp32 [N, k]).

    ``logits`` is fp32, bf16 or fp16 [N, E] (E <= 1024); an expert whose logit
    is -inf or NaN is masked.  ``score`` is "softmax" or "sigmoid"; ``bias``
    (fp32 [E]) is added to the scores for the choice only.  With
    ``topk_groups`` < ``groups`` the choice is made within the best groups, by
    the sum of each group's ``group_top`` (1 or 2) best keys.  Row i lists its
    experts by descending key, lower index first on ties, and -1 (weight 0)
    where fewer than k can be selected.  The weights are the scores, divided
    by their sum over the selection with ``renorm``, times ``scale``.  See
    ``kmassign_route`` in ``include/kmassign.h``.
    """
    dtype = _need_float(logits, "logits")
    N, E = _need_matrix(logits, "logits")
    if logits.requires_grad:
        _need_detached("kmassign_route", "logits")
    _need_no_tangent("kmassign_route", logits)
    k, groups = int(k), int(groups)
    if bias is not None:
        _need_cuda(bias, "bias", torch.float32)
        _need_shape(bias, "bias", (E,))
    given = idx, weights
    if idx is None:
        idx = _new((N, max(k, 0)), torch.int32, logits.device, stream)
    else:
        _need_cuda(idx, "idx", torch.int32)
        _need_shape(idx, "idx", (N, k))
    if weights is None:
        weights = _new((N, max(k, 0)), torch.float32, logits.device, stream)
    else:
        _need_cuda(weights, "weights", torch.float32)
        _need_shape(weights, "weights", (N, k))
    rc = library().kmassign_route(
        logits.data_ptr(), dtype, N, E, k, _score_code(score), _ptr(bias), groups,
        groups if topk_groups is None else int(topk_groups), int(group_top), int(bool(renorm)),
        float(scale), idx.data_ptr(), weights.data_ptr(), _stream_of(stream, logits))
    if rc:
        _check(rc, "kmassign_route")
    if given != (None, None):
        _written([t for t in given if t is not None])
    return idx, weights


def kmassign_route_grad(logits, idx, dweights, score: str = "softmax", renorm: bool = True,
                        scale: float = 1.0, dlogits=None, stream=None):
    """The gradient of the logits [N, E] (their type) from that of the weights.

    ``idx`` (int32 [N, k]; ids outside [0, E) are skipped, an expert named more
    than once in a row takes the sum over its places) is the choice that
    ``kmassign_route`` made with the same ``score``, ``renorm`` and ``scale``;
    ``dweights`` is fp32 [N, k].
    """
    dtype = _need_float(logits, "logits")
    N, E = _need_matrix(logits, "logits")
    _need_cuda(idx, "idx", torch.int32)
    k = _need_matrix(idx, "idx")[1]
    _need_shape(idx, "idx", (N, k))
    _need_cuda(dweights, "dweights", torch.float32)
    _need_shape(dweights, "dweights", (N, k))
    if logits.requires_grad or dweights.requires_grad:
        _need_detached("kmassign_route_grad", "logits or dweights")
    _need_no_tangent("kmassign_route_grad", logits, dweights)
    given = dlogits is not None
    if not given:
        dlogits = _new((N, E), logits.dtype, logits.device, stream)
    else:
        _need_cuda(dlogits, "dlogits", logits.dtype)
        _need_shape(dlogits, "dlogits", (N, E))
    rc = library().kmassign_route_grad(
        logits.data_ptr(), dtype, N, E, k, _score_code(score), int(bool(renorm)), float(scale),
        idx.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(),
        _stream_of(stream, logits))
    if rc:
        _check(rc, "kmassign_route_grad")
    if given:
        _written([dlogits])
    return dlogits


def kmassign_lists(idx, K: int, order=None, offsets=None, stream=None):
    """Inverted lists of ids: (order int32 [M], offsets int32 [K + 1]).

    ``idx`` is int32 of any shape, M ids in all; row r's (flat) positions are
    ``order[offsets[r]:offsets[r + 1]]``, ascending.  Ids outside [0, K) are
    left out, and as many places at the end of ``order`` hold -1.
    """
    _need_cuda(idx, "idx", torch.int32)
    M, K = idx.numel(), int(K)
    given = order, offsets
    if order is None:
        order = _new(M, torch.int32, idx.device, stream)
    else:
        _need_cuda(order, "order", torch.int32)
        _need_shape(order, "order", (M,))
    if offsets is None:
        offsets = _new(max(K, 0) + 1, torch.int32, idx.device, stream)
    else:
        _need_cuda(offsets, "offsets", torch.int32)
        _need_shape(offsets, "offsets", (K + 1,))
    rc = library().kmassign_lists(idx.data_ptr(), M, K, order.data_ptr(), offsets.data_ptr(),
                                  _stream_of(stream, idx))
    if rc:
        _check(rc, "kmassign_lists")
    if given != (None, None):
        _written([t for t in given if t is not None])
    return order, offsets


def kmassign_lookup(table, idx, weights=None, scale: float = 1.0, out=None, stream=None):
    """out[i] = scale * sum_j weights[i, j] * table[idx[i, j]], in the table's type.

    ``table`` is fp32, bf16 or fp16 [K, D]; ``idx`` int32 [N] (one row a
    point) or [N, k]; ``weights`` fp32 of idx's shape, or None for all 1.  Ids
    outside [0, K) add nothing.  Returns out [N, D].
    """
    dtype = _need_float(table, "table")
    K, D = _need_matrix(table, "table")
    N, k = _need_ids(idx)
    if weights is not None:
        _need_cuda(weights, "weights", torch.float32)
        _need_shape(weights, "weights", idx.shape)
    if table.requires_grad or (weights is not None and weights.requires_grad):
        _need_detached("kmassign_lookup", "table or weights")
    _need_no_tangent("kmassign_lookup", table, weights)
    given = out is not None
    if not given:
        out = _new((N, D), table.dtype, table.device, stream)
    else:
        _need_cuda(out, "out", table.dtype)
        _need_shape(out, "out", (N, D))
    rc = library().kmassign_lookup(table.data_ptr(), dtype, K, D, idx.data_ptr(), _ptr(weights),
                                   N, k, float(scale), out.data_ptr(),
                                   _stream_of(stream, table))
    if rc:
        _check(rc, "kmassign_lookup")
    if given:
        _written([out])
    return out


def kmassign_lookup_grad(dout, idx, K: int, weights=None, table=None, scale: float = 1.0,
                         padding: int = -1, dtable=None, accumulate: bool = False, dtype=None,
                         dweights=None, stream=None):
    """Gradients of ``kmassign_lookup``: (dtable [K, D], dweights or None).

    ``dout`` is fp32, bf16 or fp16 [N, D].  ``dtable`` is allocated in
    ``dtype`` (fp32, the default, or dout's type) unless given; with
    ``accumulate`` the gradient is added to a given one.  The row ``padding``
    takes no gradient.  The gradient of the weights (fp32, idx's shape) is
    formed when ``weights`` are given, and needs ``table`` (dout's type).
    """
    code = _need_float(dout, "dout")
    N, D = _need_matrix(dout, "dout")
    rows, k = _need_ids(idx)
    if rows != N:
        raise ValueError("idx must hold one row of ids per row of dout")
    K = int(K)
    given = dtable, dweights
    if weights is not None:
        _need_cuda(weights, "weights", torch.float32)
        _need_shape(weights, "weights", idx.shape)
        if table is None:
            raise ValueError("the gradient of the weights needs the table")
        _need_cuda(table, "table", dout.dtype)
        _need_shape(table, "table", (K, D))
        if dweights is None:
            dweights = _new(idx.shape, torch.float32, dout.device, stream)
        else:
            _need_cuda(dweights, "dweights", torch.float32)
            _need_shape(dweights, "dweights", idx.shape)
    elif dweights is not None:
        raise ValueError("dweights needs weights")
    if dout.requires_grad or (weights is not None and
                              (weights.requires_grad or table.requires_grad)):
        _need_detached("kmassign_lookup_grad", "dout, weights or table")
    _need_no_tangent("kmassign_lookup_grad", dout, weights, None if weights is None else table)
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs a given dtable")
        dtable = _new((max(K, 0), D), dtype or torch.float32, dout.device, stream)
    elif dtype is not None and dtable.dtype != dtype:
        raise TypeError(f"dtable must be {dtype}, got {dtable.dtype}")
    grad = _need_float(dtable, "dtable")
    _need_shape(dtable, "dtable", (K, D))
    rc = library().kmassign_lookup_grad(
        dout.data_ptr(), code, idx.data_ptr(), _ptr(weights),
        table.data_ptr() if weights is not None else None, N, k, K, D, float(scale), int(padding),
        int(bool(accumulate)), dtable.data_ptr(), grad, _ptr(dweights),
        _stream_of(stream, dout))
    if rc:
        _check(rc, "kmassign_lookup_grad")
    if given != (None, None):
        _written([t for t in given if t is not None])
    return dtable, dweights


_contiguous, _pointer, _size = (torch.Tensor.is_contiguous, torch.Tensor.data_ptr,
                                torch.Tensor.numel)


def _need_floats(tensors, where, name):
    """The kmassign_dtypes of a list of tensors; raises for one that cannot be taken."""
    codes = [_need_float(t, name) for t in tensors]
    if any(t.requires_grad for t in tensors):
        _need_detached(where, f"one of {name}")
    return codes


def _tensor_arrays(tensors, where, name):
    """Pointers, sizes and type codes of a list of tensors, as C arrays.

    Past the first tensor, which memory they are in is left to the library's own
    check (``_check_tensors`` tells the detail).
    """
    try:   # the common case in few steps a tensor; the detail only on failure
        codes = [_DTYPES[t.dtype] for t in tensors if _contiguous(t) and not t.requires_grad]
        plain = len(codes) == len(tensors) and (not tensors or tensors[0].is_cuda)
    except (TypeError, KeyError):
        plain = False
    if not plain:
        codes = _need_floats(tensors, where, name)
    if getattr(_forward_ad, "_current_level", 0) >= 0:
        _need_no_tangent(where, *tensors)
    return (array.array("Q", list(map(_pointer, tensors))),
            array.array("q", list(map(_size, tensors))), array.array("i", codes))


def _check_tensors(code, where, **lists):
    for name, tensors in lists.items():
        _need_floats(tensors or (), where, name)
    _check(code, where)


def _address(a):
    return a.buffer_info()[0]


def _norm_out(tensors, norm, stream):
    if norm is None:
        return _new((), torch.float32, tensors[0].device if tensors else torch.device("cuda"),
                    stream)
    _need_cuda(norm, "norm", torch.float32)
    if norm.numel() != 1:
        raise ValueError("norm must hold one element")
    return norm


def kmassign_grad_norm(tensors, norm=None, stream=None):
    """The 2-norm over all elements of a list of tensors, an fp32 scalar on the GPU."""
    tensors = list(tensors)
    ptrs, sizes, codes = _tensor_arrays(tensors, "kmassign_grad_norm", "tensors")
    given = norm is not None
    norm = _norm_out(tensors, norm, stream)
    rc = library().kmassign_grad_norm(_address(ptrs), _address(sizes), _address(codes),
                                      len(tensors), norm.data_ptr(),
                                      _stream_of(stream, norm))
    if rc:
        _check_tensors(rc, "kmassign_grad_norm", tensors=tensors)
    if given:
        _written([norm])
    return norm


def kmassign_clip(grads, max_norm: float, out=None, norm=None, stream=None):
    """Clip a list of gradients by their global norm; returns the norm (fp32 scalar).

    Each gradient (fp32, bf16 or fp16) is multiplied by min(1, max_norm /
    (norm + 1e-6)): in place, or into ``out``, a list of tensors of the same
    sizes and types.
    """
    grads = list(grads)
    ptrs, sizes, codes = _tensor_arrays(grads, "kmassign_clip", "grads")
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out must hold one tensor per gradient")
        outs, out_sizes, out_codes = _tensor_arrays(out, "kmassign_clip", "out")
        if out_codes != codes:
            raise TypeError("out must have the gradients' types")
        if out_sizes != sizes:
            raise ValueError("out must have the gradients' sizes")
    given = norm is not None
    norm = _norm_out(grads, norm, stream)
    rc = library().kmassign_clip(_address(ptrs), None if outs is None else _address(outs),
                                 _address(sizes), _address(codes), len(grads), float(max_norm),
                                 norm.data_ptr(), _stream_of(stream, norm))
    if rc:
        _check_tensors(rc, "kmassign_clip", grads=grads, out=out)
    _written(grads if out is None else out)
    if given:
        _written([norm])
    return norm


# ---- experts behind a router: grouped products, their gradients, the norm ------

_E4M3 = torch.float8_e4m3fn


def _blocks(n) -> int:
    """Blocks of 128 columns (or rows) that share a scale."""
    return -(-n // 128)


def _need_product_types(X, W, xscale, wscale):
    """The kmassign_dtype of the operands; their scales' shapes are checked."""
    if isinstance(X, torch.Tensor) and X.dtype == _E4M3:
        _need_cuda(X, "X", _E4M3)
        if xscale is None or wscale is None:
            raise ValueError("8-bit operands need xscale and wscale")
        _need_cuda(xscale, "xscale", torch.float32)
        _need_cuda(wscale, "wscale", torch.float32)
        code = 3
    else:
        code = _need_float(X, "X")
        if code == 0:
            raise TypeError("X must be bfloat16, float16 or float8_e4m3fn, got torch.float32")
        if xscale is not None or wscale is not None:
            raise ValueError("xscale and wscale belong to 8-bit operands")
    _need_cuda(W, "W", X.dtype)
    return code


def _need_lists(X, W, offsets, rows, slots, places):
    """R, D, E, F, M of a grouped product; the ids' types and sizes are checked."""
    R, D = _need_matrix(X, "X")
    if W.dim() != (2 if offsets is None else 3):
        raise ValueError("W must have shape [E, F, D] with offsets and [F, D] without, got "
                         f"{tuple(W.shape)}")
    E, F = (1, W.shape[0]) if offsets is None else W.shape[:2]
    if W.shape[-1] != D:
        raise ValueError("X and W disagree on D")
    if offsets is not None:
        _need_cuda(offsets, "offsets", torch.int32)
        _need_shape(offsets, "offsets", (E + 1,))
    M = R
    if rows is not None:
        _need_cuda(rows, "rows", torch.int32)
        M = rows.numel()
    elif slots != 1:
        raise ValueError("slots needs rows")
    if not 1 <= slots < 2 ** 31:
        raise ValueError(f"slots must be positive, got {slots}")
    if places is not None:
        _need_cuda(places, "places", torch.int32)
        if rows is not None and places.numel() != M:
            raise ValueError("rows and places must hold one id per position each")
        M = places.numel()
    return R, D, E, F, M


def kmassign_experts(X, W, offsets=None, rows=None, slots: int = 1, places=None, xscale=None,
                     wscale=None, dtype=None, out=None, stream=None):
    """Products grouped by expert: out[places[p]] = W[e] X[rows[p] // slots] for p in list e.

    ``X`` is [R, D] and ``W`` [E, F, D], bf16 or fp16, or float8_e4m3fn with
    ``xscale`` (fp32 [R, ceil(D / 128)]) and ``wscale`` (fp32 [E, ceil(F /
    128), ceil(D / 128)]).  ``offsets`` (int32 [E + 1], ``kmassign_lists``')
    says which positions belong to which expert; without it ``W`` is [F, D]
    and all positions take it.  ``rows`` and ``places`` are int32 [M] (of any
    shape): ``rows=order, slots=k`` takes the points' rows in the lists' order,
    ``places=order`` puts rows of the lists' order back to their slots.  Returns
    out [M, F] in ``dtype``: X's type or fp32, in 8 bits bf16 (the default),
    fp16 or fp32.  Rows of no list are zeros; with ``places`` rows that no
    position names are zeros, or stay as they were in a given ``out``, which
    may then have any number of rows.
    """
    code = _need_product_types(X, W, xscale, wscale)
    slots = int(slots)
    R, D, E, F, M = _need_lists(X, W, offsets, rows, slots, places)
    if code == 3:
        _need_shape(xscale, "xscale", (R, _blocks(D)))
        _need_shape(wscale, "wscale", (*W.shape[:-2], _blocks(F), _blocks(D)))
    if X.requires_grad or W.requires_grad or (
            code == 3 and (xscale.requires_grad or wscale.requires_grad)):
        _need_detached("kmassign_experts", "X, W or a scale")
    _need_no_tangent("kmassign_experts", X, W, xscale, wscale)
    given = out is not None
    if not given:
        out = _new((M, F), dtype or (torch.bfloat16 if code == 3 else X.dtype), X.device, stream,
                   torch.empty if places is None else torch.zeros)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, got {out.dtype}")
    out_code = _need_float(out, "out")
    if code != 3 and out_code not in (0, code):
        raise TypeError(f"out must be {X.dtype} or float32, got {out.dtype}")
    out_rows = M
    if given:
        out_rows, out_cols = _need_matrix(out, "out")
        if out_cols != F or (places is None and out_rows != M):
            raise ValueError(f"out must have shape {(M, F)}, got {tuple(out.shape)}")
    rc = library().kmassign_experts(
        X.data_ptr(), code, R, D, W.data_ptr(), E, F, _ptr(xscale), _ptr(wscale), _ptr(offsets), M,
        _ptr(rows), slots, _ptr(places), out.data_ptr(), out_code, out_rows,
        _stream_of(stream, X))
    if rc:
        _check(rc, "kmassign_experts")
    if given:
        _written([out])
    return out


def kmassign_experts_grad(dout, X, W, offsets=None, rows=None, slots: int = 1, places=None,
                          dtype=None, dX=None, dW=None, need_x: bool = True, need_w: bool = True,
                          stream=None):
    """Gradients of ``kmassign_experts`` in 16 bits: (dX [R, D], dW of W's shape).

    ``dout`` is [M, F] ([out's rows, F] with ``places``) in X's type, the other
    arguments are the forward call's.  ``dX`` has X's type, ``dW`` is fp32 (the
    default ``dtype``) or X's type; one that is not needed is None.
    """
    if isinstance(X, torch.Tensor) and X.dtype == _E4M3:
        raise TypeError("X must be bfloat16 or float16, got torch.float8_e4m3fn")
    code = _need_product_types(X, W, None, None)
    slots = int(slots)
    R, D, E, F, M = _need_lists(X, W, offsets, rows, slots, places)
    _need_cuda(dout, "dout", X.dtype)
    out_rows, out_cols = _need_matrix(dout, "dout")
    if out_cols != F or (places is None and out_rows != M):
        raise ValueError(f"dout must have shape {(M, F)}, got {tuple(dout.shape)}")
    if not (need_x or need_w):
        raise ValueError("neither gradient is needed")
    if (dX is not None and not need_x) or (dW is not None and not need_w):
        raise ValueError("a gradient is given but not needed")
    if dout.requires_grad or X.requires_grad or W.requires_grad:
        _need_detached("kmassign_experts_grad", "dout, X or W")
    _need_no_tangent("kmassign_experts_grad", dout, X, W)
    given = dX, dW
    if dX is not None:
        _need_cuda(dX, "dX", X.dtype)
        _need_shape(dX, "dX", (R, D))
    elif need_x:
        dX = _new((R, D), X.dtype, X.device, stream)
    if dW is None:
        if need_w:
            dW = _new(W.shape, dtype or torch.float32, X.device, stream)
    else:
        if dtype is not None and dW.dtype != dtype:
            raise TypeError(f"dW must be {dtype}, got {dW.dtype}")
        _need_shape(dW, "dW", W.shape)
    dw_code = 0 if dW is None else _need_float(dW, "dW")
    if dw_code not in (0, code):
        raise TypeError(f"dW must be {X.dtype} or float32, got {dW.dtype}")
    rc = library().kmassign_experts_grad(
        dout.data_ptr(), code, out_rows, F, X.data_ptr(), R, D, W.data_ptr(), E, _ptr(offsets), M,
        _ptr(rows), slots, _ptr(places), _ptr(dX), _ptr(dW), dw_code, _stream_of(stream, X))
    if rc:
        _check(rc, "kmassign_experts_grad")
    if given != (None, None):
        _written([t for t in given if t is not None])
    return dX, dW


def _need_norm_weight(weight, dtype, D) -> int:
    """The kmassign_dtype of a norm's weight: fp32 or the rows' type."""
    if weight is None:
        return 0
    code = _need_float(weight, "weight")
    if code not in (0, _DTYPES[dtype]):
        raise TypeError(f"weight must be {dtype} or float32, got {weight.dtype}")
    _need_shape(weight, "weight", (D,))
    return code


def kmassign_rmsnorm(X, weight=None, residual=None, eps: float = 1e-6, dtype=None, out=None,
                     scales=None, total=None, rstd=None, stream=None):
    """Root-mean-square norm of rows: (out, scales, total, rstd).

    ``X`` is fp32, bf16 or fp16 [N, D]; with ``residual`` (the same) the rows
    are total = X + residual, rounded to that type, else total is ``X`` itself.
    out = total * rstd * weight, rstd = 1 / sqrt(mean(total^2) + eps) (fp32
    [N]); ``weight`` [D] is fp32 or of X's type, None for all 1.  ``dtype`` is
    X's type (the default; scales is None) or float8_e4m3fn: out's values are
    then code * scale with scales fp32 [N, ceil(D / 128)], as
    ``kmassign_experts`` takes them.
    """
    code = _need_float(X, "X")
    N, D = _need_matrix(X, "X")
    wcode = _need_norm_weight(weight, X.dtype, D)
    if residual is not None:
        _need_cuda(residual, "residual", X.dtype)
        _need_shape(residual, "residual", (N, D))
    elif total is not None:
        raise ValueError("total needs a residual")
    if X.requires_grad or (weight is not None and weight.requires_grad) or (
            residual is not None and residual.requires_grad):
        _need_detached("kmassign_rmsnorm", "X, weight or residual")
    _need_no_tangent("kmassign_rmsnorm", X, weight, residual)
    given = [t for t in (out, scales, total, rstd) if t is not None]
    if dtype is None:
        dtype = X.dtype if out is None else out.dtype
    if dtype not in (X.dtype, _E4M3):
        raise TypeError(f"dtype must be {X.dtype} or float8_e4m3fn, got {dtype}")
    if out is None:
        out = _new((N, D), dtype, X.device, stream)
    else:
        _need_cuda(out, "out", dtype)
        _need_shape(out, "out", (N, D))
    if dtype == _E4M3:
        if scales is None:
            scales = _new((N, _blocks(D)), torch.float32, X.device, stream)
        else:
            _need_cuda(scales, "scales", torch.float32)
            _need_shape(scales, "scales", (N, _blocks(D)))
    elif scales is not None:
        raise ValueError("scales belong to an 8-bit output")
    if residual is not None:
        if total is None:
            total = _new((N, D), X.dtype, X.device, stream)
        else:
            _need_cuda(total, "total", X.dtype)
            _need_shape(total, "total", (N, D))
    if rstd is None:
        rstd = _new((N,), torch.float32, X.device, stream)
    else:
        _need_cuda(rstd, "rstd", torch.float32)
        _need_shape(rstd, "rstd", (N,))
    rc = library().kmassign_rmsnorm(
        X.data_ptr(), code, N, D, _ptr(residual), _ptr(weight), wcode, float(eps), _ptr(total),
        out.data_ptr(), 3 if dtype == _E4M3 else code, _ptr(scales), rstd.data_ptr(),
        _stream_of(stream, X))
    if rc:
        _check(rc, "kmassign_rmsnorm")
    if given:
        _written(given)
    return out, scales, X if total is None else total, rstd


def kmassign_rmsnorm_grad(dout, total, weight, rstd, dtotal=None, dX=None, dweight=None,
                          stream=None):
    """Gradients of ``kmassign_rmsnorm``: (dX [N, D], dweight fp32 [D] or None without a weight).

    ``dout`` is the gradient of out in the rows' type, ``total`` and ``rstd``
    what the forward call returned; ``dtotal`` (the rows' type), the gradient
    that reaches total otherwise, is added.  dX is the gradient of X and of the
    residual alike.
    """
    code = _need_float(total, "total")
    N, D = _need_matrix(total, "total")
    _need_cuda(dout, "dout", total.dtype)
    _need_shape(dout, "dout", (N, D))
    wcode = _need_norm_weight(weight, total.dtype, D)
    _need_cuda(rstd, "rstd", torch.float32)
    _need_shape(rstd, "rstd", (N,))
    if dtotal is not None:
        _need_cuda(dtotal, "dtotal", total.dtype)
        _need_shape(dtotal, "dtotal", (N, D))
    if dout.requires_grad or total.requires_grad or rstd.requires_grad or (
            weight is not None and weight.requires_grad) or (
            dtotal is not None and dtotal.requires_grad):
        _need_detached("kmassign_rmsnorm_grad", "an input")
    _need_no_tangent("kmassign_rmsnorm_grad", dout, total, weight, rstd, dtotal)
    given = [t for t in (dX, dweight) if t is not None]
    if dX is None:
        dX = _new((N, D), total.dtype, total.device, stream)
    else:
        _need_cuda(dX, "dX", total.dtype)
        _need_shape(dX, "dX", (N, D))
    if weight is None:
        if dweight is not None:
            raise ValueError("dweight needs a weight")
    elif dweight is None:
        dweight = _new((D,), torch.float32, total.device, stream)
    else:
        _need_cuda(dweight, "dweight", torch.float32)
        _need_shape(dweight, "dweight", (D,))
    rc = library().kmassign_rmsnorm_grad(
        dout.data_ptr(), code, N, D, total.data_ptr(), _ptr(weight), wcode, rstd.data_ptr(),
        _ptr(dtotal), dX.data_ptr(), _ptr(dweight), _stream_of(stream, total))
    if rc:
        _check(rc, "kmassign_rmsnorm_grad")
    if given:
        _written(given)
    return dX, dweight


def kmassign_set_wait_timeout(ns: int) -> None:
    """Bound on every kernel pipeline wait, in ns (0 = default 2 s)."""
    _check(library().kmassign_set_wait_timeout(int(ns)), "kmassign_set_wait_timeout")


def shard_rows(N: int, rank: int, world: int) -> tuple:
    """Contiguous, balanced share [begin, end) of N points for one of `world` GPUs.

    The assignment needs no exchange between GPUs: each holds all centroids
    and assigns its own rows; the answers concatenate in rank order.
    """
    if world < 1 or not 0 <= rank < world or N < 0:
        raise ValueError("need N >= 0 and 0 <= rank < world")
    base, extra = divmod(int(N), int(world))
    begin = rank * base + min(rank, extra)
    return begin, begin + base + (1 if rank < extra else 0)


def kmassign_check(stream=None) -> int:
    """Synchronise the stream and return the device status code (0 = OK)."""
    return int(library().kmassign_check(_stream_ptr(stream)))


def norms(C, stream=None):
    return kmassign_norms(C, stream=stream)


def assign(X, C, cnorm=None, with_minscore: bool = False, stream=None):
    """Convenience: returns idx, or (idx, minscore) when ``with_minscore``."""
    ms = None
    if with_minscore:
        ms = _new(X.shape[0], torch.float32, X.device, stream)
    idx = kmassign(X, C, cnorm=cnorm, minscore=ms, stream=stream)
    return (idx, ms) if with_minscore else idx


def _need_host(t, name, dtype):
    if isinstance(t, torch.Tensor) and not t.is_cuda and t.dtype == dtype and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name} must be a CPU tensor (ideally pinned)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def assign_host(X_host, C_host, idx_host=None, cnorm_host=None, minscore_host=None,
                device=None, stream=None, rows_per_slice: int = 0):
    """End-to-end assignment of host tensors through ``kmassign_host``.

    X (bf16 [N, D]), C (bf16 [K, D]) and the optional cnorm (fp32 [K]) are
    CPU tensors, ideally pinned so that the copies overlap the kernels.  The
    library copies C in, then X in row slices of whole kernel waves while the
    previous slice is assigned, and copies each slice's idx (and minscore)
    back as soon as it is ready; the call returns when the answers are in
    ``idx_host`` (int32 [N], pinned, allocated if None) and ``minscore_host``
    (fp32 [N] or None).  ``device`` is the GPU to run on (default: current),
    ``stream`` a stream of it (default: its current stream),
    ``rows_per_slice`` forces the slice size (0: automatic).  Returns idx_host.
    """
    _need_host(X_host, "X_host", torch.bfloat16)
    _need_host(C_host, "C_host", torch.bfloat16)
    N, D = X_host.shape
    K, D2 = C_host.shape
    if D != D2:
        raise ValueError("X and C disagree on D")
    if cnorm_host is not None:
        _need_host(cnorm_host, "cnorm_host", torch.float32)
    if idx_host is None:
        idx_host = torch.empty(N, dtype=torch.int32, pin_memory=True)
    _need_host(idx_host, "idx_host", torch.int32)
    if minscore_host is not None:
        _need_host(minscore_host, "minscore_host", torch.float32)
    device = torch.device("cuda") if device is None else torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        rc = library().kmassign_host_ex(_ptr(X_host), _ptr(C_host), _ptr(cnorm_host), N, K, D,
                                        _ptr(idx_host), _ptr(minscore_host), int(rows_per_slice),
                                        _stream_ptr(stream, device))
    _check(rc, "kmassign_host")
    return idx_host
