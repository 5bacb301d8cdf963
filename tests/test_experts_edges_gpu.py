"""Experts' products and the norm on the GPU at the edges of what the entry points accept.

Tolerances and helpers are those of test_experts_gpu; whole numbers are compared bit for bit."""

import os
import subprocess
import sys

import pytest
import torch

import means_nearest_centroid_gb300 as km
from test_experts_gpu import (  # noqa: F401
    BF16, E4M3, FP16, FP32, OUT, ROOT, U, dev, gen_of, ints, no_kernel_gave_up, offsets_of)

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


# ---- rows' gradients by ids --------------------------------------------------------

def exact_rows_gradient(dout, W, off, rows, slots, R):
    """In 64 bits, nothing rounded; and the sum of magnitudes."""
    dX = torch.zeros(R, W.shape[2], dtype=torch.float64, device=W.device)
    size = dX.clone()
    for e in range(W.shape[0]):
        p = torch.arange(int(off[e]), int(off[e + 1]), device=W.device)
        r, d, w = rows.view(-1)[p].long() // slots, dout[p].double(), W[e].double()
        dX.index_add_(0, r, d @ w)
        size.index_add_(0, r, d.abs() @ w.abs())
    return dX, size


@pytest.mark.parametrize("E,N,k,D,F", [(4, 30, 2, 40, 64), (8, 700, 4, 520, 136), (64, 500, 8, 264, 72),
                                       (2, 9, 2, 2048, 1000), (6, 3000, 3, 72, 2056)])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
def test_a_point_s_gradient_is_rounded_once(dev, E, N, k, D, F, dtype):  # noqa: F811
    """The products of a point's positions cancel for the most part: what is left of them is as near as
    fp32 sums of F and k terms and one rounding allow."""
    g = gen_of(dev, N + D)
    order, off = km.kmassign_lists(torch.randint(0, E, (N, k), generator=g, device=dev).int(), E)
    W = torch.randn(E, F, D, generator=g, device=dev).to(dtype)
    dout = torch.randn(N * k, F, generator=g, device=dev).to(dtype)
    X = torch.zeros(N, D, device=dev, dtype=dtype)
    ref, size = exact_rows_gradient(dout, W, off, order, k, N)
    for need_w in (False, True):
        dX, _ = km.kmassign_experts_grad(dout, X, W, off, rows=order, slots=k, need_w=need_w)
        assert ((dX.double() - ref).abs() <= OUT[dtype] * ref.abs() * 1.01 + (2 * F + k) * U * size + 2.0 ** -25).all()
    # an error that is even over half a step either way has a root mean square of 1 / sqrt(3) of that at most
    # (one rounding gives 0.42, one more of each product 0.60)
    assert (dX.double() - ref).norm() <= 0.578 * OUT[dtype] * ref.norm()


@pytest.mark.parametrize("N", [5, 600])
def test_products_past_fp16_that_cancel(dev, N):  # noqa: F811
    """Each position's product is beyond fp16's largest number, a point's sum is not."""
    E, D, F = 2, 48, 128
    g = gen_of(dev, N)
    idx = torch.tensor([[0, 1]], device=dev).int().repeat(N, 1)
    order, off = km.kmassign_lists(idx, E)
    W = torch.empty(E, F, D, device=dev, dtype=FP16)
    W[0], W[1] = 8, -8
    W[1, 0] += ints(g, (D,), 5, FP16)
    dout = torch.full((2 * N, F), 128.0, device=dev, dtype=FP16)
    dX, dW = km.kmassign_experts_grad(dout, torch.ones(N, D, device=dev, dtype=FP16), W, off, rows=order, slots=2)
    ref, size = exact_rows_gradient(dout, W, off, order, 2, N)
    assert size.min() > 2 * 65504 and ref.abs().max() <= 640
    assert torch.equal(dX, ref.to(FP16)) and (dW == 128 * N).all()


@pytest.mark.parametrize("D", [1000, 776])
def test_rows_gradients_of_many_positions(dev, D):  # noqa: F811
    """Whole numbers, more columns and positions than are held at once."""
    g = gen_of(dev, D)
    E, N, k, F = 5, 40_000, 4, 16
    order, off = km.kmassign_lists(torch.randint(-1, E, (N, k), generator=g, device=dev).int(), E)
    W, dout = ints(g, (E, F, D), 4, BF16), ints(g, (N * k, F), 4, BF16)
    ref, _ = exact_rows_gradient(dout, W, off, order, k, N)
    X = torch.zeros(N, D, device=dev, dtype=BF16)
    for need_w in (False, True):
        dX, _ = km.kmassign_experts_grad(dout, X, W, off, rows=order, slots=k, need_w=need_w)
        assert torch.equal(dX, ref.to(BF16))


@pytest.mark.parametrize("M,D", [(1, 8), (77, 8), (3000, 24), (160_000, 1000)])
def test_rows_gradients_of_rows_named_by_many(dev, M, D):  # noqa: F811
    """Three of a hundred rows take every position: sums that span the chunks of both halves of the columns."""
    g = gen_of(dev, M + D)
    E, F, R = 3, 16, 100
    rows = torch.tensor([0, 57, 99], device=dev).int()[torch.randint(0, 3, (M,), generator=g, device=dev)]
    off = offsets_of([M // 3, 0, M - M // 3], dev)
    W, dout = ints(g, (E, F, D), 2, BF16), ints(g, (M, F), 2, BF16)
    ref, size = exact_rows_gradient(dout, W, off, rows, 1, R)
    assert size.max() < 2 ** 24
    dX, _ = km.kmassign_experts_grad(dout, torch.zeros(R, D, device=dev, dtype=BF16), W, off, rows=rows, need_w=False)
    assert torch.equal(dX, ref.to(BF16))


# ---- the norm's gradients -------------------------------------------------------------

@pytest.mark.parametrize("dtype", [FP32, BF16, FP16], ids=str)
@pytest.mark.parametrize("N,D", [(1, 40), (12000, 40), (12000, 33), (3000, 500), (4000, 129), (11000, 256), (5000, 2048),
                                 (700, 8200), (2000, 777)])
def test_weights_gradient_of_whole_numbers_comes_out_exactly(dev, N, D, dtype):  # noqa: F811
    """rstd are powers of two and the sums fit 24 bits, so that a row that is left out or counted twice shows."""
    g = gen_of(dev, N + D)
    x, dout = ints(g, (N, D), 3, dtype), ints(g, (N, D), 3, dtype)
    rstd = 2.0 ** ints(g, (N,), 1, FP32)
    w = torch.ones(D, device=dev)
    ref = (dout.double() * x.double() * rstd.double()[:, None]).sum(0)
    _, dw = km.kmassign_rmsnorm_grad(dout, x, w, rstd)
    assert torch.equal(dw.double(), ref)


ROOM = """
import sys
import torch
import means_nearest_centroid_gb300 as km
for N, D, dtype in ((6000, 32768, torch.bfloat16), (6000, 16384, torch.float32), (6000, 7168, torch.bfloat16)):
    x = torch.ones(N, D, device="cuda", dtype=dtype)
    dx, w, dw = torch.empty_like(x), torch.ones(D, device="cuda"), torch.empty(D, device="cuda")
    rstd = torch.ones(N, device="cuda")
    small = torch.ones(8, 8, device="cuda", dtype=dtype)
    km.kmassign_rmsnorm_grad(x, x, None, rstd, dX=dx)
    km.kmassign_rmsnorm_grad(small, small, w[:8], rstd[:8])
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    km.kmassign_rmsnorm_grad(x, x, w, rstd, dX=dx, dweight=dw)
    torch.cuda.synchronize()
    print(free - torch.cuda.mem_get_info()[0])
"""


def test_the_weight_s_partial_sums_take_little_room(dev):  # noqa: F811
    """A row of partial sums for each group of rows in flight: of these long rows up to four groups an SM,
    150 rows to 610 of 28 to 128 KB, 20 MB at most."""
    out = subprocess.run([sys.executable, "-c", ROOM], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    used = [int(line) for line in out.stdout.split()]
    assert len(used) == 3 and max(used) <= 72 << 20, used


# ---- 8 bits -----------------------------------------------------------------------------

@pytest.mark.parametrize("N,D", [(300, 128), (4001, 1000), (64, 16384), (2000, 777), (3, 20000)])
@pytest.mark.parametrize("bits", [3, 8, 24])
def test_codes_are_the_quotients_rounded_to_nearest(dev, N, D, bits):  # noqa: F811
    """Values of few bits, whose quotients are often between two codes; blocks of every size."""
    g = gen_of(dev, N + D + bits)
    x = torch.randn(N, D, generator=g, device=dev) if bits == 24 else ints(g, (N, D), 2 ** bits, FP32)
    for w in (torch.ones(D, device=dev), 2.0 ** torch.randint(-110, 100, (D,), generator=g, device=dev).float(),
              2.0 ** -100 * torch.rand(D, generator=g, device=dev), torch.randn(D, generator=g, device=dev)):
        y, _, _, rstd = km.kmassign_rmsnorm(x, w)
        codes, scales, _, same = km.kmassign_rmsnorm(x, w, dtype=E4M3)
        nb = -(-D // 128)
        tops = torch.nn.functional.pad(y, (0, nb * 128 - D)).view(N, nb, 128).abs().amax(-1).clamp(min=2.0 ** -100)
        assert torch.equal(rstd, same) and torch.equal(scales, tops / torch.full_like(tops, 448))
        want = (y / scales.repeat_interleave(128, 1)[:, :D]).to(E4M3)
        assert torch.equal(codes.float(), want.float())


@pytest.mark.parametrize("D", [144, 1040, 2048])
def test_in_8_bits_a_row_s_bits_depend_on_nothing_else(dev, D):  # noqa: F811
    """Alone, among few and among many: other kernels, the same sums."""
    g = gen_of(dev, D)
    F, nb = 136, -(-D // 128)
    X = torch.randn(600, D, generator=g, device=dev).to(E4M3)
    W = torch.randn(3, F, D, generator=g, device=dev).to(E4M3)
    xs, ws = torch.rand(600, nb, generator=g, device=dev), torch.rand(3, 2, nb, generator=g, device=dev)
    kw = dict(wscale=ws, dtype=FP32)
    many = km.kmassign_experts(X, W, offsets_of([0, 600, 0], dev), xscale=xs, **kw)
    few = km.kmassign_experts(X[:50], W, offsets_of([0, 50, 0], dev), xscale=xs[:50], **kw)
    one = km.kmassign_experts(X[49:50], W[1], xscale=xs[49:50], wscale=ws[1], dtype=FP32)
    rows = torch.arange(600, device=dev).flip(0).int()
    back = km.kmassign_experts(X, W, offsets_of([0, 600, 0], dev), rows=rows, xscale=xs, **kw)
    assert torch.equal(many[:50], few) and torch.equal(many[49:50], one) and torch.equal(back.flip(0), many)


# ---- how calls are made -----------------------------------------------------------------

def test_calls_refuse_forward_mode_tangents(dev):  # noqa: F811
    """Any input that a result depends on, also under no_grad; a primal beside a dual level is taken."""
    X, W = torch.ones(6, 16, device=dev, dtype=BF16), torch.ones(2, 8, 16, device=dev, dtype=BF16)
    q, v, s, t = X.to(E4M3), W.to(E4M3), torch.ones(6, 1, device=dev), torch.ones(2, 1, 1, device=dev)
    off, d = torch.tensor([0, 3, 6], device=dev).int(), torch.ones(6, 8, device=dev, dtype=BF16)
    idx, w, rstd = torch.zeros(6, 1, device=dev).int(), torch.ones(6, 1, device=dev), torch.ones(6, device=dev)
    calls = [
        (lambda a, b: km.kmassign_experts(a, b, off), X, W),
        (lambda a, b: km.kmassign_experts(q, v, off, xscale=a, wscale=b), s, t),
        (lambda a, b, c: km.kmassign_experts_grad(a, b, c, off), d, X, W),
        (lambda a, b, c: km.kmassign_rmsnorm(a, b, residual=c), X, W[0, 0], X),
        (lambda a, b, c, e, f: km.kmassign_rmsnorm_grad(a, b, c, e, dtotal=f), X, X, W[0, 0], rstd, X),
        (lambda a: km.kmassign_route(a, 2), X),
        (lambda a, b: km.kmassign_route_grad(a, idx, b), X, w),
        (lambda a, b: km.kmassign_lookup(a, idx, weights=b), X, w),
        (lambda a, b, c: km.kmassign_lookup_grad(a, idx, 6, weights=b, table=c), X, w, X),
        (lambda a: km.kmassign_grad_norm([rstd, a]), X),
        (lambda a: km.kmassign_clip([rstd.clone(), a], 1.0), X.clone()),
    ]
    forward = torch.autograd.forward_ad
    with forward.dual_level():
        for call, *args in calls:
            call(*args)
            for i, x in enumerate(args):
                dual = args[:i] + [forward.make_dual(x, torch.ones_like(x))] + args[i + 1:]
                for mode in (torch.no_grad, torch.enable_grad):
                    with mode(), pytest.raises(RuntimeError, match="tangent"):
                        call(*dual)


def test_weights_gradient_with_a_short_wait_bound(dev):  # noqa: F811
    """A wait of its that runs out is reported, whole and cut k-blocks alike, and the next call is right. (Segments
    of 32 k-blocks: see the test of the other products.)"""
    g = gen_of(dev, 7)
    E, per, D, F = 8, 8200, 2048, 1024
    M = E * per
    X, W, d = ints(g, (M, D), 1, BF16), torch.zeros(E, F, D, device=dev, dtype=BF16), ints(g, (M, F), 1, BF16)
    off = offsets_of([per] * E, dev)
    rows = torch.arange(M, device=dev).int()
    rows[::97] = -1
    for kw in (dict(), dict(rows=rows)):
        def call():
            return km.kmassign_experts_grad(d, X, W, off, need_x=False, dtype=BF16, **kw)[1]
        want = call()
        try:
            km.kmassign_set_wait_timeout(100)
            call()
            rc = km.kmassign_check()
        finally:
            km.kmassign_set_wait_timeout(0)
        assert rc == km.STATUS["KMASSIGN_ERR_TIMEOUT"], km.kmassign_strerror(rc)
        assert km.kmassign_check() == 0
        assert torch.equal(call(), want) and km.kmassign_check() == 0
