"""Argument checks of the learned-assignment entry points, without a GPU: every
error comes back before anything touches CUDA."""

import ctypes

import pytest
import torch

import means_nearest_centroid_gb300 as km
from means_nearest_centroid_gb300 import _build

P = ctypes.c_void_p
NULL = P(0)
A, B, C, D_, ODD = P(0x10000), P(0x20000), P(0x30000), P(0x40000), P(0x10001)
S = km.STATUS
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return km.library()


def route(lib, logits=A, dtype=0, N=10, E=16, k=2, score=0, bias=NULL, groups=1, topk=1, top=2,
          renorm=1, scale=1.0, idx=B, w=C):
    return lib.kmassign_route(logits, dtype, N, E, k, score, bias, groups, topk, top, renorm, scale,
                              idx, w, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), "SHAPE"), (dict(N=2**31), "SHAPE"), (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"),
    (dict(N=2**27, k=16), "SHAPE"), (dict(k=0), "ARG"), (dict(k=17), "ARG"),
    (dict(E=100, k=33), "ARG"), (dict(dtype=3), "ARG"), (dict(dtype=-1), "ARG"),
    (dict(score=2), "ARG"), (dict(renorm=2), "ARG"), (dict(scale=NAN), "ARG"),
    (dict(scale=INF), "ARG"), (dict(groups=0), "ARG"), (dict(groups=3), "ARG"),
    (dict(E=66, groups=33, topk=33), "ARG"), (dict(groups=4, topk=5), "ARG"),
    (dict(groups=4, topk=0), "ARG"), (dict(groups=8, topk=1, k=3), "ARG"), (dict(top=3), "ARG"),
    (dict(top=0), "ARG"), (dict(logits=NULL), "NULL"), (dict(idx=NULL), "NULL"),
    (dict(w=NULL), "NULL"), (dict(logits=ODD), "ALIGN"), (dict(bias=P(0x10002)), "ALIGN"),
    (dict(idx=P(0x10002)), "ALIGN"), (dict(w=P(0x10002)), "ALIGN"),
    (dict(logits=P(0x10002)), "ALIGN"),
], ids=str)
def test_route_refuses(lib, bad, code):
    assert route(lib, **bad) == S["KMASSIGN_ERR_" + code]


def test_empty_calls_do_nothing(lib):
    assert route(lib, N=0, logits=NULL, idx=NULL, w=NULL) == 0
    assert lib.kmassign_route_grad(NULL, 0, 0, 16, 2, 0, 1, 1.0, NULL, NULL, NULL, NULL) == 0
    assert lib.kmassign_lookup(NULL, 0, 4, 8, NULL, NULL, 0, 1, 1.0, NULL, NULL) == 0


def test_half_precision_logits_need_two_byte_alignment_only(lib):
    assert route(lib, dtype=1, logits=P(0x10002)) != S["KMASSIGN_ERR_ALIGN"]


def grad(lib, logits=A, dtype=0, N=10, E=16, k=2, score=0, renorm=1, scale=1.0, idx=B, dw=C, dl=D_):
    return lib.kmassign_route_grad(logits, dtype, N, E, k, score, renorm, scale, idx, dw, dl, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(E=2000), "SHAPE"), (dict(k=40), "ARG"), (dict(score=-1), "ARG"), (dict(renorm=-1), "ARG"),
    (dict(idx=NULL), "NULL"), (dict(dw=NULL), "NULL"), (dict(dl=NULL), "NULL"),
    (dict(dl=ODD), "ALIGN"), (dict(logits=P(0x10002)), "ALIGN"),
], ids=str)
def test_route_grad_refuses(lib, bad, code):
    assert grad(lib, **bad) == S["KMASSIGN_ERR_" + code]


def lookup(lib, table=A, dtype=1, K=4, D=8, idx=B, w=NULL, N=3, k=1, scale=1.0, out=C):
    return lib.kmassign_lookup(table, dtype, K, D, idx, w, N, k, scale, out, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=2**31), "SHAPE"), (dict(k=0), "SHAPE"),
    (dict(N=2**20, k=2**11), "SHAPE"), (dict(D=0), "UNSUPPORTED_D"),
    (dict(D=65537), "UNSUPPORTED_D"), (dict(dtype=7), "ARG"), (dict(scale=NAN), "ARG"),
    (dict(table=NULL), "NULL"), (dict(idx=NULL), "NULL"), (dict(out=NULL), "NULL"),
    (dict(table=ODD), "ALIGN"), (dict(out=ODD), "ALIGN"), (dict(w=P(0x10002)), "ALIGN"),
], ids=str)
def test_lookup_refuses(lib, bad, code):
    assert lookup(lib, **bad) == S["KMASSIGN_ERR_" + code]


def lookup_grad(lib, dout=A, dtype=1, idx=B, w=NULL, table=NULL, N=3, k=1, K=4, D=8, scale=1.0,
                padding=-1, acc=0, dt=C, gt=0, dw=NULL):
    return lib.kmassign_lookup_grad(dout, dtype, idx, w, table, N, k, K, D, scale, padding, acc, dt,
                                    gt, dw, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(acc=2), "ARG"), (dict(gt=2), "ARG"), (dict(gt=5), "ARG"), (dict(dout=NULL), "NULL"),
    (dict(idx=NULL), "NULL"), (dict(dt=NULL), "NULL"), (dict(dw=D_), "NULL"),
    (dict(dt=P(0x10002)), "ALIGN"), (dict(D=0), "UNSUPPORTED_D"), (dict(N=2**31), "SHAPE"),
], ids=str)
def test_lookup_grad_refuses(lib, bad, code):
    assert lookup_grad(lib, **bad) == S["KMASSIGN_ERR_" + code]


@pytest.mark.parametrize("args,code", [
    ((B, -1, 4, C, A), "SHAPE"), ((B, 2**31, 4, C, A), "SHAPE"), ((B, 3, 0, C, A), "SHAPE"),
    ((NULL, 3, 4, C, A), "NULL"), ((B, 3, 4, NULL, A), "NULL"), ((B, 3, 4, C, NULL), "NULL"),
    ((P(0x10002), 3, 4, C, A), "ALIGN"),
], ids=str)
def test_lists_refuses(lib, args, code):
    assert lib.kmassign_lists(*args, NULL) == S["KMASSIGN_ERR_" + code]


def clip(lib, ptrs=(0x10000,), sizes=(4,), types=(0,), n=None, max_norm=1.0, norm=B, out=None):
    c = len(ptrs)
    arr = (P * c)(*ptrs)
    outs = None if out is None else (P * c)(*out)
    return lib.kmassign_clip(arr, outs, (ctypes.c_int64 * c)(*sizes), (ctypes.c_int32 * c)(*types),
                             c if n is None else n, max_norm, norm, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), "SHAPE"), (dict(sizes=(-1,)), "SHAPE"), (dict(types=(9,)), "ARG"),
    (dict(max_norm=-1.0), "ARG"), (dict(max_norm=NAN), "ARG"), (dict(norm=NULL), "NULL"),
    (dict(ptrs=(0,)), "NULL"), (dict(out=(0,)), "NULL"), (dict(ptrs=(0x10002,)), "ALIGN"),
    (dict(norm=P(0x10002)), "ALIGN"),
], ids=str)
def test_clip_refuses(lib, bad, code):
    assert clip(lib, **bad) == S["KMASSIGN_ERR_" + code]


def test_clip_refuses_null_arrays(lib):
    assert lib.kmassign_grad_norm(None, None, None, 2, B, NULL) == S["KMASSIGN_ERR_NULL"]


def test_python_refuses_host_tensors_types_and_shapes():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: km.kmassign_route(x, 2), lambda: km.kmassign_lookup(x, i),
                 lambda: km.kmassign_lists(i, 4), lambda: km.kmassign_clip([x], 1.0),
                 lambda: km.kmassign_lookup_grad(x, i, 4), lambda: km.kmassign_grad_norm([x]),
                 lambda: km.kmassign_route_grad(x, i, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        km.kmassign_route([1.0], 2)
    with pytest.raises(ValueError, match="softmax"):
        km._score_code("tanh")
