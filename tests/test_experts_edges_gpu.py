"""Experts' products and the norm on the GPU at the edges of what the entry points accept.

Tolerances and helpers are those of test_experts_gpu; whole numbers are compared bit for bit."""

import pytest
import torch

import means_nearest_centroid_gb300 as km
from test_experts_gpu import (  # noqa: F401
    BF16, E4M3, FP32, dev, no_kernel_gave_up)

pytestmark = pytest.mark.gpu


# ---- batches without points -----------------------------------------------------

@pytest.mark.parametrize("k", [1, 8])
def test_a_batch_without_points(dev, k):  # noqa: F811
    """Lists of no ids, as a step without points makes them, with the slots of any other step."""
    E, D, F = 16, 64, 72
    order, off = km.kmassign_lists(torch.zeros(0, k, device=dev, dtype=torch.int32), E)
    W = torch.ones(E, F, D, device=dev, dtype=BF16)
    X, dout = torch.zeros(0, D, device=dev, dtype=BF16), torch.zeros(0, F, device=dev, dtype=BF16)
    for kw in (dict(rows=order, slots=k), dict(rows=order, slots=k, places=order), dict(places=order)):
        assert km.kmassign_experts(X, W, off, **kw).shape == (0, F)
        s, t = torch.zeros(0, 1, device=dev), torch.ones(E, 1, 1, device=dev)
        out = km.kmassign_experts(X.to(E4M3), W.to(E4M3), off, xscale=s, wscale=t, **kw)
        assert out.shape == (0, F) and out.dtype == BF16
        for dtype in (FP32, BF16):
            dX, dW = km.kmassign_experts_grad(dout, X, W, off, dtype=dtype, **kw)
            assert dX.shape == (0, D) and dW.shape == W.shape and dW.dtype == dtype and not dW.any()
    # points that no list names, and an output that stays as it was
    given = torch.full((5, F), 7.0, device=dev, dtype=BF16)
    some = torch.ones(5, D, device=dev, dtype=BF16)
    assert km.kmassign_experts(some, W, off, rows=order, slots=k, places=order, out=given) is given
    assert (given == 7).all()
    dX, dW = km.kmassign_experts_grad(dout, some, W, off, rows=order, slots=k)
    assert dX.shape == some.shape and not dX.any() and not dW.any()
