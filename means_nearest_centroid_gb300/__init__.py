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
# require grad (but for the bias, which the weights do not depend on).

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
            "kmassign_route_grad, kmassign_lookup_grad)")


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
