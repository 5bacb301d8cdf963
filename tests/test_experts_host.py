"""Argument checks of the experts' products and the root-mean-square norm, without a GPU: every error
comes back before anything touches CUDA."""

import ctypes
import os
import re

import pytest
import torch

import means_nearest_centroid_gb300 as km
from means_nearest_centroid_gb300 import _build

P = ctypes.c_void_p
NULL = P(0)
A, B, C, D_, E_ = P(0x10000), P(0x20000), P(0x30000), P(0x40000), P(0x50000)
ODD, EIGHT = P(0x10001), P(0x10008)
S = km.STATUS
BF16, FP16, E4M3 = 1, 2, 3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return km.library()


def experts(lib, X=A, dtype=BF16, R=40, D=64, W=B, E=4, F=64, xs=NULL, ws=NULL, offsets=C, M=40,
            rows=NULL, slots=1, places=NULL, out=D_, out_dtype=BF16, out_rows=40):
    return lib.kmassign_experts(X, dtype, R, D, W, E, F, xs, ws, offsets, M, rows, slots, places, out,
                                out_dtype, out_rows, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), "ARG"), (dict(dtype=4), "ARG"), (dict(dtype=-1), "ARG"), (dict(out_dtype=3), "ARG"),
    (dict(out_dtype=FP16), "ARG"), (dict(dtype=E4M3, out_dtype=E4M3, xs=E_, ws=E_), "ARG"),
    (dict(xs=E_), "ARG"), (dict(ws=E_), "ARG"),
    (dict(R=-1), "SHAPE"), (dict(R=2**31), "SHAPE"), (dict(M=-1), "SHAPE"), (dict(M=2**31), "SHAPE"), (dict(M=2**30, R=2**31 - 1, out_rows=2**31 - 1), "SHAPE"),
    (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"), (dict(slots=0), "SHAPE"), (dict(slots=2), "SHAPE"),
    (dict(M=41), "SHAPE"), (dict(M=41, rows=E_), "SHAPE"), (dict(M=41, places=E_), "SHAPE"),
    (dict(out_rows=39), "SHAPE"), (dict(offsets=NULL), "SHAPE"), (dict(out_rows=2**31), "SHAPE"),
    (dict(D=60), "UNSUPPORTED_D"), (dict(D=0), "UNSUPPORTED_D"), (dict(F=4), "UNSUPPORTED_D"),
    (dict(F=65), "UNSUPPORTED_D"), (dict(D=65544), "UNSUPPORTED_D"), (dict(F=65544), "UNSUPPORTED_D"),
    (dict(dtype=E4M3, D=72, xs=E_, ws=E_), "UNSUPPORTED_D"),
    (dict(X=NULL), "NULL"), (dict(W=NULL), "NULL"), (dict(out=NULL), "NULL"),
    (dict(dtype=E4M3, ws=E_), "NULL"), (dict(dtype=E4M3, xs=E_), "NULL"),
    (dict(X=EIGHT), "ALIGN"), (dict(W=EIGHT), "ALIGN"), (dict(out=EIGHT), "ALIGN"),
    (dict(offsets=ODD), "ALIGN"), (dict(rows=ODD), "ALIGN"), (dict(places=ODD), "ALIGN"),
    (dict(dtype=E4M3, xs=ODD, ws=E_), "ALIGN"), (dict(R=0, M=3, rows=E_, places=E_), "SHAPE"),
], ids=str)
def test_experts_refuses(lib, bad, code):
    assert experts(lib, **bad) == S["KMASSIGN_ERR_" + code]


def test_products_of_nothing_do_nothing(lib):
    assert experts(lib, M=0, X=NULL, W=NULL, out=NULL, offsets=NULL, E=1) == 0
    assert experts(lib, M=0, R=0, X=NULL, out=NULL, out_rows=0) == 0
    assert experts(lib, places=E_, out=NULL, out_rows=0) == 0


def grad(lib, dout=A, dtype=BF16, out_rows=40, F=64, X=B, R=40, D=64, W=C, E=4, offsets=D_, M=40,
         rows=NULL, slots=1, places=NULL, dX=E_, dW=P(0x60000), dw=0):
    return lib.kmassign_experts_grad(dout, dtype, out_rows, F, X, R, D, W, E, offsets, M, rows, slots,
                                     places, dX, dW, dw, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), "ARG"), (dict(dtype=E4M3), "ARG"), (dict(dw=FP16), "ARG"), (dict(dw=3), "ARG"),
    (dict(M=41), "SHAPE"), (dict(out_rows=39), "SHAPE"), (dict(E=1025), "SHAPE"),
    (dict(slots=3), "SHAPE"), (dict(offsets=NULL), "SHAPE"), (dict(D=12), "UNSUPPORTED_D"),
    (dict(F=12), "UNSUPPORTED_D"), (dict(dX=NULL, dW=NULL), "NULL"), (dict(dout=NULL), "NULL"),
    (dict(W=NULL), "NULL"), (dict(X=NULL), "NULL"), (dict(dX=EIGHT), "ALIGN"), (dict(dW=EIGHT), "ALIGN"),
    (dict(dout=EIGHT), "ALIGN"), (dict(rows=ODD), "ALIGN"), (dict(places=ODD), "ALIGN"),
], ids=str)
def test_experts_grad_refuses(lib, bad, code):
    assert grad(lib, **bad) == S["KMASSIGN_ERR_" + code]


def norm(lib, X=A, dtype=BF16, N=10, D=64, residual=NULL, weight=B, wdtype=BF16, eps=1e-6, total=NULL,
         out=C, out_dtype=BF16, scales=NULL, rstd=NULL):
    return lib.kmassign_rmsnorm(X, dtype, N, D, residual, weight, wdtype, eps, total, out, out_dtype,
                                scales, rstd, NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), "SHAPE"), (dict(N=2**31), "SHAPE"), (dict(D=0), "UNSUPPORTED_D"),
    (dict(D=32769), "UNSUPPORTED_D"), (dict(dtype=3), "ARG"), (dict(out_dtype=FP16), "ARG"),
    (dict(out_dtype=0), "ARG"), (dict(wdtype=FP16), "ARG"), (dict(wdtype=3), "ARG"),
    (dict(eps=-1e-6), "ARG"), (dict(eps=NAN), "ARG"), (dict(eps=INF), "ARG"), (dict(X=NULL), "NULL"),
    (dict(out=NULL), "NULL"), (dict(residual=A), "NULL"), (dict(out_dtype=E4M3), "NULL"),
    (dict(X=ODD), "ALIGN"), (dict(residual=ODD, total=D_), "ALIGN"), (dict(residual=A, total=ODD), "ALIGN"),
    (dict(weight=ODD), "ALIGN"), (dict(weight=P(0x10002), wdtype=0), "ALIGN"), (dict(out=ODD), "ALIGN"),
    (dict(rstd=P(0x10002)), "ALIGN"), (dict(out_dtype=E4M3, scales=P(0x10002)), "ALIGN"),
], ids=str)
def test_norm_refuses(lib, bad, code):
    assert norm(lib, **bad) == S["KMASSIGN_ERR_" + code]


def norm_grad(lib, dout=A, dtype=BF16, N=10, D=64, total=B, weight=C, wdtype=BF16, rstd=D_, dtotal=NULL,
              dX=E_, dweight=NULL):
    return lib.kmassign_rmsnorm_grad(dout, dtype, N, D, total, weight, wdtype, rstd, dtotal, dX, dweight,
                                     NULL)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), "SHAPE"), (dict(D=0), "UNSUPPORTED_D"), (dict(D=32769), "UNSUPPORTED_D"),
    (dict(dtype=3), "ARG"), (dict(wdtype=FP16), "ARG"), (dict(dout=NULL), "NULL"), (dict(total=NULL), "NULL"),
    (dict(rstd=NULL), "NULL"), (dict(dX=NULL), "NULL"), (dict(dX=ODD), "ALIGN"), (dict(dtotal=ODD), "ALIGN"),
    (dict(rstd=P(0x10002)), "ALIGN"), (dict(dweight=P(0x10002)), "ALIGN"),
], ids=str)
def test_norm_grad_refuses(lib, bad, code):
    assert norm_grad(lib, **bad) == S["KMASSIGN_ERR_" + code]


def test_norms_of_nothing_do_nothing(lib):
    assert norm(lib, N=0, X=NULL, out=NULL) == 0
    assert norm_grad(lib, N=0, dout=NULL, total=NULL, rstd=NULL, dX=NULL) == 0


def test_a_batch_without_points_may_have_slots(lib):
    """An empty tensor's pointer is NULL: no positions, whatever the slots of a point."""
    for e8 in (dict(), dict(dtype=E4M3, xs=E_, ws=E_)):
        assert experts(lib, M=0, slots=8, **e8) == 0
        assert experts(lib, M=0, R=0, X=NULL, slots=8, out=NULL, out_rows=0, **e8) == 0
        assert experts(lib, M=0, slots=0, **e8) == S["KMASSIGN_ERR_SHAPE"]
    assert grad(lib, M=0, slots=8, dX=NULL, dW=NULL) == S["KMASSIGN_ERR_NULL"]   # the next check


@pytest.mark.parametrize("call", [
    lambda x: km.kmassign_experts(x, x), lambda x: km.kmassign_experts_grad(x, x, x),
    lambda x: km.kmassign_rmsnorm(x), lambda x: km.kmassign_rmsnorm_grad(x, x, None, x[:, 0]),
])
def test_host_tensors_are_refused(call):
    for x in (torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.float8_e4m3fn)):
        with pytest.raises((TypeError, ValueError)):
            call(x)
    with pytest.raises(TypeError):
        call([[1.0]])


def test_forward_mode_tangents_are_refused():
    """Also under no_grad, which keeps them; not where a Function's own jvp takes over."""
    forward = torch.autograd.forward_ad
    x = torch.ones(3)
    km._need_no_tangent("here", x, None)
    with forward.dual_level():
        dual = forward.make_dual(x, x)
        km._need_no_tangent("here", x, None, forward.unpack_dual(dual).primal)
        for mode in (torch.no_grad, torch.enable_grad):
            with mode(), pytest.raises(RuntimeError, match="here.*tangent"):
                km._need_no_tangent("here", x, None, dual)

        class Own(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x):
                km._need_no_tangent("here", x)
                return 2 * x

            @staticmethod
            def jvp(ctx, t):
                return 2 * t
        assert torch.equal(forward.unpack_dual(Own.apply(dual)).tangent, 2 * x)
    km._need_no_tangent("here", dual)


def test_kernels_that_start_early_use_plain_loads():
    """A kernel that may start before the one in front of it ends runs while its inputs are written: loads that
    promise constant memory for as long as it runs (__ldg, const __restrict__) are not for it."""
    csrc = os.path.join(os.path.dirname(km.__file__), "csrc")
    early = 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            helpers, *kernels = f.read().split("__global__")
        starts = ["wait_for_previous()" in k for k in kernels]
        early += sum(starts)
        if kernels and all(starts):
            assert "__ldg" not in helpers, name
        for kernel, is_early in zip(kernels, starts):
            if is_early:
                assert not re.search(r"__ldg|ld\.global\.nc|const \w+ \*__restrict__", kernel), (name, kernel[:120])
    assert early >= 16
