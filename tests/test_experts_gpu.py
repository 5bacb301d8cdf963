"""Products grouped by expert in 16 and 8 bits, their gradients, and the root-mean-square norm on the
GPU, against plain 64-bit implementations.

Tolerances.  U = 2^-24 is half an fp32 ulp, OUT[type] half an ulp of an output type, relative.  Operands
that are small whole numbers (scales powers of two) have sums that fp32 holds exactly, in whatever order
they are formed, so those results are the correctly rounded ones, bit for bit.  For others the tensor cores
may cut off instead of rounding: a sum of K terms is allowed K whole ulps (2 U each) of the sum of
magnitudes.  Sums of n fp32 terms elsewhere are allowed n roundings of the sum of magnitudes."""

import importlib.util
import os

import pytest
import torch

import means_nearest_centroid_gb300 as km

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from means_nearest_centroid_gb300 import _build
    _build.build()
    km.library()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def no_kernel_gave_up(dev):
    yield
    assert km.kmassign_check() == 0


def gen_of(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def ints(g, shape, top, dtype):
    return torch.randint(-top, top + 1, shape, generator=g, device=g.device).to(dtype)


def offsets_of(lengths, dev, start=0):
    return torch.tensor([start] + lengths, device=dev).cumsum(0).int()


def spread(total, E, g):
    """E list lengths that add up to total, a third of the lists empty."""
    w = torch.rand(E, generator=g, device=g.device) ** 3
    w[torch.rand(E, generator=g, device=g.device) < 0.33] = 0
    if not w.sum():
        w[E // 2] = 1
    n = (w / w.sum() * total).long()
    n[int(w.argmax())] += total - int(n.sum())
    return n.tolist()


def pairs(off, M, rows=None, slots=1, places=None, R=None, out_rows=None):
    """(expert, position, row of X or -1, row of out or -1) of every position of a list."""
    off = off.clamp(0, M).tolist()
    rows = None if rows is None else rows.view(-1).tolist()
    places = None if places is None else places.view(-1).tolist()
    for e in range(len(off) - 1):
        for p in range(off[e], off[e + 1]):
            r = p if rows is None else (rows[p] // slots if rows[p] >= 0 else -1)
            o = p if places is None else places[p]
            yield e, p, r if R is None or 0 <= r < R else -1, o if out_rows is None or 0 <= o < out_rows else -1


def ref_forward(X, W, off, M, out, **kw):
    """In 64 bits; out: [rows, F] with what unnamed rows hold."""
    kw.update(R=X.shape[0], out_rows=out.shape[0])
    x, w = X.double(), W.double()
    for e in range(W.shape[0]):
        es = [(r, o) for f, _, r, o in pairs(off, M, **kw) if f == e and o >= 0]
        if es:
            r = torch.tensor([a for a, _ in es], device=x.device)
            o = torch.tensor([b for _, b in es], device=x.device)
            y = x[r.clamp(min=0)] @ w[e].t()
            out[o] = torch.where(r[:, None] < 0, 0.0, y)
    return out


# ---- forward -------------------------------------------------------------------

SHAPES = [  # E, D, F, positions
    (1, 8, 8, 1), (1, 64, 128, 1), (3, 8, 264, 5), (2, 72, 40, 33), (5, 128, 256, 64), (4, 200, 136, 257),
    (7, 136, 72, 700), (2, 512, 520, 513), (40, 64, 64, 300), (300, 24, 16, 1000), (1024, 16, 8, 900),
    (3, 64, 1032, 1100), (1, 256, 384, 2049),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("E,D,F,M", SHAPES)
def test_whole_numbers_come_out_exactly(dev, E, D, F, M, dtype):
    g = gen_of(dev, E + D + F + M)
    X, W = ints(g, (M, D), 3, dtype), ints(g, (E, F, D), 3, dtype)
    off = offsets_of(spread(M, E, g), dev)
    ref = ref_forward(X, W, off, M, torch.zeros(M, F, dtype=torch.float64, device=dev))
    for out_type in (dtype, FP32):
        out = km.kmassign_experts(X, W, off, dtype=out_type)
        assert out.dtype == out_type and torch.equal(out, ref.to(out_type))


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("D", [64, 2048, 2056, 6000])
def test_random_values(dev, D, few):
    """Also contractions longer than what the tensor cores add up without a break."""
    g = gen_of(dev, D)
    E, F, M = (16, 136, 90) if few else (2, 136, 600)
    X = torch.randn(M, D, generator=g, device=dev).to(BF16)
    W = torch.randn(E, F, D, generator=g, device=dev).to(BF16)
    off = offsets_of(spread(M, E, g), dev)
    zero = torch.zeros(M, F, dtype=torch.float64, device=dev)
    ref = ref_forward(X, W, off, M, zero.clone())
    size = ref_forward(X.abs(), W.abs(), off, M, zero.clone())
    for out_type in (FP32, BF16):
        out = km.kmassign_experts(X, W, off, dtype=out_type).double()
        assert ((out - ref).abs() <= OUT[out_type] * ref.abs() * 1.01 + 2 * U * D * size).all()
    # the actual error is that of sums of 2,048, not of D terms
    out = km.kmassign_experts(X, W, off, dtype=FP32).double()
    assert (out - ref).norm() <= 2 * U * 200 * ref.norm()


@pytest.mark.parametrize("E,M", [(4, 60), (4, 700), (64, 700)])
@pytest.mark.parametrize("slots", [1, 3])
def test_rows_and_places(dev, E, M, slots):
    """Ids that name no row give zeros, places outside are not written, rows not named stay."""
    g = gen_of(dev, E + M + slots)
    R, D, F, out_rows = 50, 40, 72, 2 * M
    X, W = ints(g, (R, D), 3, BF16), ints(g, (E, F, D), 3, BF16)
    rows = torch.randint(-2, (R + 3) * slots, (M,), generator=g, device=dev).int()
    places = torch.randperm(out_rows + 40, generator=g, device=dev)[:M].int() - 20
    lengths = spread(M - 9, E, g)
    off = offsets_of(lengths, dev, start=4)   # positions before and behind the lists
    for kw in (dict(rows=rows, slots=slots), dict(places=places), dict(rows=rows, slots=slots, places=places)):
        x = X if "rows" in kw else ints(g, (M, D), 3, BF16)
        x = x.clone()
        x[-1] = 0 if "rows" in kw else x[-1]
        if "places" in kw:
            given = torch.full((out_rows, F), 7.0, device=dev, dtype=BF16)
            ref = ref_forward(x, W, off, M, given.double(), **kw)
            out = km.kmassign_experts(x, W, off, out=given, **kw)
            assert out is given
            if M <= out_rows:
                inside = {**kw, "places": kw["places"].clamp(0, M - 1)}
                inside["places"] = torch.randperm(M, generator=g, device=dev).int()
                fresh = km.kmassign_experts(x, W, off, **inside)
                zero = torch.zeros(M, F, dtype=torch.float64, device=dev)
                assert torch.equal(fresh, ref_forward(x, W, off, M, zero, **inside).to(BF16))
        else:
            ref = ref_forward(x, W, off, M, torch.zeros(M, F, dtype=torch.float64, device=dev), **kw)
            given = torch.full((M, F), NAN, device=dev, dtype=BF16)
            out = km.kmassign_experts(x, W, off, out=given, **kw)
        assert torch.equal(out, ref.to(BF16))


def test_rows_that_are_not_there_stay_zero_beside_infinities(dev):
    """A missing row's product is zeros even where row 0 or the weights are not finite."""
    for M in (20, 400):
        X = torch.full((3, 64), INF, device=dev, dtype=BF16)
        X[1] = 1
        W = torch.ones(2, 72, 64, device=dev, dtype=BF16)
        W[1] = NAN
        rows = torch.tensor([1, -1, 5, 1] * (M // 4), device=dev).int()
        off = offsets_of([M // 2, M // 2], dev)
        out = km.kmassign_experts(X, W, off, rows=rows)
        there, first = rows == 1, torch.arange(M, device=dev) < M // 2
        assert (out[~there] == 0).all()
        assert (out[there & first] == 64).all() and out[there & ~first].isnan().all()


def test_what_is_not_finite_stays_in_its_row_and_column(dev):
    g = gen_of(dev, 0)
    M, E, D, F = 300, 3, 136, 264
    X, W = ints(g, (M, D), 2, BF16), ints(g, (E, F, D), 2, BF16)
    off = offsets_of([100, 77, 123], dev)
    ref = km.kmassign_experts(X, W, off)
    X2, W2 = X.clone(), W.clone()
    X2[100, 7], X2[99, 5], W2[1, 3, 9], W2[2, 263, 0] = NAN, INF, NAN, NAN
    out = km.kmassign_experts(X2, W2, off)
    same = torch.ones(M, F, dtype=torch.bool, device=dev)
    same[100] = same[99] = False
    same[100:177, 3] = False
    same[177:, 263] = False
    assert torch.equal(out[same], ref[same])
    assert out[100].isnan().all() and out[100:177, 3].isnan().all() and out[177:, 263].isnan().all()
    assert not out[99].isfinite()[W[0][:, 5] != 0].any()


@pytest.mark.parametrize("bad", [[-5, 3, 1000], [4, 2, 9], [10, 10, 10], [0, 0, 0], [9, 1, 0], [2**31 - 1, 0, 5]])
def test_offsets_that_are_none_stay_in_bounds(dev, bad):
    """Offsets are clamped to [0, M]; what guard rows around out hold is not touched."""
    M, D, F = 10, 16, 24
    X, W = torch.ones(M, D, device=dev, dtype=BF16), torch.ones(2, F, D, device=dev, dtype=BF16)
    guard = torch.full((M + 200, F), 7.0, device=dev, dtype=BF16)
    km.kmassign_experts(X, W, torch.tensor(bad, device=dev).int(), out=guard[100:100 + M])
    assert (guard[:100] == 7).all() and (guard[100 + M:] == 7).all()
    big = torch.full((2, F, D), 7.0, device=dev)
    dX, dW = km.kmassign_experts_grad(torch.ones(M, F, device=dev, dtype=BF16), X, W,
                                      torch.tensor(bad, device=dev).int(), dW=big)
    assert dX.isfinite().all() and dW.isfinite().all()


@pytest.mark.parametrize("M,E", [(10, 40), (3000, 40), (3000, 7)])
def test_lists_that_overlap_stay_in_bounds(dev, M, E):
    """Every other list would be all positions: the first has them, and nothing else is touched."""
    D, F = 16, 264
    X = torch.ones(M, D, device=dev, dtype=BF16)
    W = torch.arange(1, E + 1, device=dev).view(E, 1, 1).expand(E, F, D).to(BF16).contiguous()
    offsets = torch.tensor([0, M] * (E // 2 + 1), device=dev)[:E + 1].int()
    guard = torch.full((M + 200, F), 7.0, device=dev, dtype=BF16)
    km.kmassign_experts(X, W, offsets, out=guard[100:100 + M])
    assert (guard[:100] == 7).all() and (guard[100 + M:] == 7).all() and (guard[100:100 + M] == D).all()
    dW = km.kmassign_experts_grad(torch.ones(M, F, device=dev, dtype=BF16), X, W, offsets, need_x=False)[1]
    assert (dW[0] == M).all() and not dW[1:].any()
    assert km.kmassign_check() == 0


def test_a_plain_product(dev):
    g = gen_of(dev, 3)
    for M, D, F in ((1, 8, 8), (37, 264, 392), (1000, 72, 200)):
        X, W = ints(g, (M, D), 3, FP16), ints(g, (F, D), 3, FP16)
        assert torch.equal(km.kmassign_experts(X, W), (X.double() @ W.double().t()).half())
        dout = ints(g, (M, F), 2, FP16)
        dX, dW = km.kmassign_experts_grad(dout, X, W)
        assert torch.equal(dX, (dout.double() @ W.double()).half())
        assert dW.shape == W.shape and torch.equal(dW, (dout.double().t() @ X.double()).float())


def test_a_row_s_bits_depend_on_nothing_else(dev):
    """Alone, among few and among many: other tiles, the same sums."""
    g = gen_of(dev, 4)
    D, F = 1000, 136
    X = torch.randn(600, D, generator=g, device=dev).to(BF16)
    W = torch.randn(3, F, D, generator=g, device=dev).to(BF16)
    many = km.kmassign_experts(X, W, offsets_of([0, 600, 0], dev), dtype=FP32)
    few = km.kmassign_experts(X[:50], W, offsets_of([0, 50, 0], dev), dtype=FP32)
    one = km.kmassign_experts(X[49:50], W[1], dtype=FP32)
    rows = torch.arange(600, device=dev).flip(0).int()
    back = km.kmassign_experts(X, W, offsets_of([0, 600, 0], dev), rows=rows, dtype=FP32)
    assert torch.equal(many[:50], few) and torch.equal(many[49:50], one) and torch.equal(back.flip(0), many)


# ---- 8 bits ----------------------------------------------------------------------

def whole_8_bits(g, R, D, E, F):
    """Whole numbers that e4m3 holds, scales powers of two."""
    nb, fb = -(-D // 128), -(-F // 128)
    X, W = ints(g, (R, D), 8, FP32).to(E4M3), ints(g, (E, F, D), 8, FP32).to(E4M3)
    xs = 2.0 ** ints(g, (R, nb), 1, FP32)
    ws = 2.0 ** ints(g, (E, fb, nb), 1, FP32)
    return X, W, xs, ws


def values(X, W, xs, ws):
    D, F = X.shape[-1], W.shape[-2]
    x = X.double() * xs.double().repeat_interleave(128, -1)[:, :D]
    w = W.double() * ws.double().repeat_interleave(128, -1)[..., :D].repeat_interleave(128, -2)[..., :F, :]
    return x, w


@pytest.mark.parametrize("E,D,F,M", [
    (1, 16, 8, 1), (3, 128, 136, 7), (2, 144, 264, 40), (4, 512, 128, 300), (4, 1040, 72, 513),
    (40, 272, 392, 200), (3, 2048, 40, 1000), (1, 640, 1032, 260),
])
def test_8_bits_whole_numbers_come_out_exactly(dev, E, D, F, M):
    g = gen_of(dev, D + F + M)
    X, W, xs, ws = whole_8_bits(g, M, D, E, F)
    x, w = values(X, W, xs, ws)
    off = offsets_of(spread(M, E, g), dev)
    ref = ref_forward(x, w, off, M, torch.zeros(M, F, dtype=torch.float64, device=dev))
    for out_type in (BF16, FP32, FP16):
        if out_type == FP16 and ref.abs().max() > 60000:
            continue
        out = km.kmassign_experts(X, W, off, xscale=xs, wscale=ws, dtype=out_type)
        assert torch.equal(out, ref.to(out_type))
    assert km.kmassign_experts(X, W, off, xscale=xs, wscale=ws).dtype == BF16


@pytest.mark.parametrize("M", [30, 900])
def test_8_bits_random_scales_rows_and_places(dev, M):
    g = gen_of(dev, M)
    E, D, F, R, slots = 5, 912, 200, 70, 4
    X, W, xs, ws = whole_8_bits(g, R, D, E, F)
    xs, ws = torch.rand(xs.shape, generator=g, device=dev) + 0.5, torch.rand(ws.shape, generator=g, device=dev) + 0.5
    rows = torch.randint(-4, (R + 2) * slots, (M,), generator=g, device=dev).int()
    places = torch.randperm(M, generator=g, device=dev).int()
    off = offsets_of(spread(M - 3, E, g), dev, start=2)
    x, w = values(X, W, xs, ws)
    kw = dict(rows=rows, slots=slots, places=places)
    zero = torch.zeros(M, F, dtype=torch.float64, device=dev)
    ref, size = ref_forward(x, w, off, M, zero.clone(), **kw), ref_forward(x.abs(), w.abs(), off, M, zero.clone(), **kw)
    out = km.kmassign_experts(X, W, off, xscale=xs, wscale=ws, dtype=FP32, **kw).double()
    # a block's sum is exact; its scale and each addition are rounded
    assert ((out - ref).abs() <= U * (-(-D // 128) + 3) * size).all()


def test_8_bits_a_plain_product_and_misaligned_scales(dev):
    g = gen_of(dev, 9)
    X, W, xs, ws = whole_8_bits(g, 77, 1024, 1, 136)
    x, w = values(X, W, xs, ws)
    ref = (x @ w[0].t()).float()
    assert torch.equal(km.kmassign_experts(X, W[0], xscale=xs, wscale=ws[0], dtype=FP32), ref)
    moved = torch.empty(77 * 8 + 1, device=dev)[1:].view(77, 8).copy_(xs)
    assert torch.equal(km.kmassign_experts(X, W[0], xscale=moved, wscale=ws[0], dtype=FP32), ref)


# ---- gradients ---------------------------------------------------------------------

def ref_grad(dout, X, W, off, M, dtype, **kw):
    """dX (each position's product rounded to the type first, where rows are named) and dW, in 64 bits."""
    kw.update(R=X.shape[0], out_rows=dout.shape[0])
    dX = torch.zeros(X.shape, dtype=torch.float64, device=X.device)
    dW = torch.zeros(W.shape, dtype=torch.float64, device=X.device)
    for e in range(W.shape[0]):
        es = [(r, o) for f, _, r, o in pairs(off, M, **kw) if f == e and o >= 0 and r >= 0]
        if es:
            r = torch.tensor([a for a, _ in es], device=X.device)
            dy = dout[torch.tensor([b for _, b in es], device=X.device)].double()
            each = dy @ W[e].double()
            dX.index_add_(0, r, each.to(dtype).double() if kw.get("rows") is not None else each)
            dW[e] = dy.t() @ X[r].double()
    return dX.to(dtype), dW


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("E,D,F,M", SHAPES)
def test_gradients_of_whole_numbers_come_out_exactly(dev, E, D, F, M, dtype):
    g = gen_of(dev, E + D + F + M)
    X, W, dout = ints(g, (M, D), 2, dtype), ints(g, (E, F, D), 2, dtype), ints(g, (M, F), 2, dtype)
    off = offsets_of(spread(M, E, g), dev)
    dX, dW = ref_grad(dout, X, W, off, M, dtype)
    for kind in (FP32, dtype):
        a, b = km.kmassign_experts_grad(dout, X, W, off, dtype=kind)
        assert torch.equal(a, dX) and b.dtype == kind and torch.equal(b, dW.to(kind))
    a, b = km.kmassign_experts_grad(dout, X, W, off, need_w=False)
    assert b is None and torch.equal(a, dX)
    a, b = km.kmassign_experts_grad(dout, X, W, off, need_x=False)
    assert a is None and torch.equal(b, dW.float())


@pytest.mark.parametrize("E,M,slots", [(4, 60, 1), (4, 700, 3), (64, 500, 2)])
def test_gradients_with_rows_and_places(dev, E, M, slots):
    """Rows named often, rows and places that are not there (beside infinities), positions of no list."""
    g = gen_of(dev, E + M + slots)
    R, D, F, out_rows = 50, 40, 72, 2 * M
    W = ints(g, (E, F, D), 2, BF16)
    rows = torch.randint(-2, (R + 3) * slots, (M,), generator=g, device=dev).int()
    places = torch.randperm(out_rows + 40, generator=g, device=dev)[:M].int() - 20
    off = offsets_of(spread(M - 9, E, g), dev, start=4)
    for kw in (dict(rows=rows, slots=slots), dict(places=places), dict(rows=rows, slots=slots, places=places), {}):
        X = ints(g, (R if "rows" in kw else M + 3, D), 2, BF16)
        dout = ints(g, (out_rows if "places" in kw else M, F), 2, BF16)
        dX, dW = ref_grad(dout, X, W, off, M, BF16, **kw)
        if kw:
            a, b = km.kmassign_experts_grad(dout, X, W, off, **kw)
        else:
            a, b = km.kmassign_experts_grad(dout, X[:M], W, off)
            dX = dX[:M]
        assert torch.equal(a, dX) and torch.equal(b, dW.float())
        # what no position of a list names is not used, whatever it holds
        named = [(r, o) for _, _, r, o in pairs(off, M, R=X.shape[0], out_rows=dout.shape[0], **kw)]
        X2, d2 = X.clone(), dout.clone()
        dead_rows = set(range(X.shape[0])) - {r for r, o in named if o >= 0}
        dead_outs = set(range(dout.shape[0])) - {o for r, o in named if r >= 0}
        X2[sorted(dead_rows)] = INF
        d2[sorted(dead_outs)] = NAN
        if kw:
            a2, b2 = km.kmassign_experts_grad(d2, X2, W, off, **kw)
            assert torch.equal(a2, dX) and torch.equal(b2, dW.float())


def test_a_list_s_end_does_not_leak_into_the_next_one(dev):
    """Contractions over positions end inside a block of 64, beside rows that are not finite."""
    for lengths in ([1, 63, 64, 65, 0, 130, 7], [200, 3], [0, 0, 5]):
        M, E, D, F = sum(lengths), len(lengths), 72, 136
        g = gen_of(dev, M)
        X, dout, W = ints(g, (M, D), 2, BF16), ints(g, (M, F), 2, BF16), ints(g, (E, F, D), 2, BF16)
        off = offsets_of(lengths, dev)
        _, dW = km.kmassign_experts_grad(dout, X, W, off, need_x=False)
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            X2, d2 = torch.full_like(X, NAN), torch.full_like(dout, INF)
            X2[lo:hi], d2[lo:hi] = X[lo:hi], dout[lo:hi]
            _, one = km.kmassign_experts_grad(d2, X2, W, off, need_x=False)
            assert torch.equal(one[e], (dout[lo:hi].double().t() @ X[lo:hi].double()).float())
            assert torch.equal(one[e], dW[e])


def test_weights_gradient_of_a_long_list(dev):
    """fp32 sums over 30,000 positions stay those of 512 at a time, added up rounded."""
    g = gen_of(dev, 1)
    M, D, F = 30000, 64, 64
    X, dout = torch.randn(M, D, generator=g, device=dev).to(BF16), torch.randn(M, F, generator=g, device=dev).to(BF16)
    _, dW = km.kmassign_experts_grad(dout, X, torch.zeros(F, D, device=dev, dtype=BF16), need_x=False)
    ref = dout.double().t() @ X.double()
    assert (dW.double() - ref).norm() <= 2 * U * 64 * ref.norm()
    _, again = km.kmassign_experts_grad(dout, X, torch.zeros(F, D, device=dev, dtype=BF16), need_x=False)
    assert torch.equal(dW, again)


def test_gradients_are_the_products_differences(dev):
    """The product is linear in each operand: with whole numbers its differences are exact."""
    g = gen_of(dev, 2)
    M, E, D, F, R, slots = 90, 5, 24, 40, 30, 3
    X, W, dout = ints(g, (R, D), 2, BF16), ints(g, (E, F, D), 2, BF16), ints(g, (M, F), 2, BF16)
    rows = torch.randperm(M, generator=g, device=dev).int()
    off = offsets_of([10, 0, 33, 40, 7], dev)
    kw = dict(rows=rows, slots=slots)
    dX, dW = km.kmassign_experts_grad(dout, X, W, off, **kw)

    def loss(x, w):
        return (km.kmassign_experts(x, w, off, dtype=FP32, **kw).double() * dout.double()).sum()
    for seed in range(4):
        stepx, stepw = ints(gen_of(dev, seed), (R, D), 1, BF16), ints(gen_of(dev, seed), (E, F, D), 1, BF16)
        assert loss(X + stepx, W) - loss(X, W) == (dX.double() * stepx.double()).sum()
        assert loss(X, W + stepw) - loss(X, W) == (dW.double() * stepw.double()).sum()


# ---- the norm ------------------------------------------------------------------------

def sums_of(D):
    """Roundings of a sum of D squares or products: at most 64 in a lane, 5 and 5 across lanes and warps."""
    return min(D, 64) + 10


def ref_norm(x, w, eps):
    rstd = 1.0 / (x.double().square().mean(-1) + eps).sqrt()
    y = x.double() * rstd[:, None]
    return rstd, y if w is None else y * w.double()


NORMS = [(1, 1), (3, 7), (5, 64), (17, 127), (4, 129), (2, 777), (700, 256), (2, 2048), (3, 2056), (2, 5001),
         (3, 8192), (1, 16384), (2, 16400), (1, 32768), (1, 32767), (2000, 40)]


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16], ids=str)
@pytest.mark.parametrize("N,D", NORMS)
def test_norm(dev, N, D, dtype):
    g = gen_of(dev, N + D)
    x = (torch.randn(N, D, generator=g, device=dev) * torch.exp(torch.randn(N, 1, generator=g, device=dev))).to(dtype)
    r = torch.randn(N, D, generator=g, device=dev).to(dtype)
    for w in (torch.randn(D, generator=g, device=dev).to(dtype), torch.randn(D, generator=g, device=dev), None):
        for res in (None, r):
            out, scales, total, rstd = km.kmassign_rmsnorm(x, w, residual=res, eps=1e-5)
            assert scales is None and out.dtype == dtype
            if res is None:
                assert total is x
            else:
                assert torch.equal(total, (x.float() + r.float()).to(dtype))
            srstd, y = ref_norm(total, w, 1e-5)
            rel = (sums_of(D) / 2 + 8) * U
            assert ((rstd.double() - srstd).abs() <= rel * srstd).all()
            tiny = 2.0 ** -25 if dtype == FP16 else 0.0
            assert ((out.double() - y).abs() <= (rel + 2 * U + OUT[dtype]) * y.abs() * 1.001 + tiny).all()


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16], ids=str)
@pytest.mark.parametrize("N,D", NORMS)
def test_norm_to_8_bits(dev, N, D, dtype):
    g = gen_of(dev, N + D)
    x = torch.randn(N, D, generator=g, device=dev).to(dtype)
    x[0] = 0
    w = torch.exp(2 * torch.randn(D, generator=g, device=dev)).to(dtype)
    out, scales, _, _ = km.kmassign_rmsnorm(x, w, dtype=E4M3)
    _, y = ref_norm(x, w, 1e-6)
    nb = -(-D // 128)
    assert out.dtype == E4M3 and scales.shape == (N, nb)
    tops = torch.nn.functional.pad(y, (0, nb * 128 - D)).view(N, nb, 128).abs().amax(-1).clamp(min=2.0 ** -100) / 448
    rel = (sums_of(D) / 2 + 12) * U
    assert ((scales.double() - tops).abs() <= rel * tops).all()
    wide = scales.double().repeat_interleave(128, 1)[:, :D]
    got = out.double() * wide
    # half a step: 2^-4 of the value, or 2^-10 of the scale where codes are subnormal
    assert ((got - y).abs() <= y.abs() * (2.0 ** -4 + 2 * rel) + wide * 2.0 ** -10 * 1.001).all()
    assert (out[0].double() == 0).all() and (scales[0] == 2.0 ** -100 / 448).all()


def test_norm_in_place_and_of_rows_that_are_not_finite(dev):
    x = torch.randn(9, 136, device=dev).to(BF16)
    r = torch.randn(9, 136, device=dev).to(BF16)
    w = torch.randn(136, device=dev).to(BF16)
    out, _, total, rstd = km.kmassign_rmsnorm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    km.kmassign_rmsnorm(a, w, residual=b, total=b, out=a)
    assert torch.equal(a, out) and torch.equal(b, total)
    a = x.clone()
    assert torch.equal(km.kmassign_rmsnorm(a, w, residual=r, total=a)[0], out) and torch.equal(a, total)
    bad = x.clone()
    bad[1, 5], bad[2, 7] = NAN, INF
    y, scales, _, s = km.kmassign_rmsnorm(bad, w, dtype=E4M3)
    same = [0] + list(range(3, 9))
    clean = km.kmassign_rmsnorm(x, w, dtype=E4M3)
    assert torch.equal(y[same].float(), clean[0][same].float()) and torch.equal(scales[same], clean[1][same])
    assert y[1].float().isnan().all() and s[1].isnan()
    assert s[2] == 0 and y[2, 7].float().isnan() and (y[2].float()[torch.arange(136, device=dev) != 7] == 0).all()


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16], ids=str)
@pytest.mark.parametrize("N,D", NORMS + [(5000, 72), (3000, 1024)])
def test_norm_gradients(dev, N, D, dtype):
    g = gen_of(dev, N + D)
    x = torch.randn(N, D, generator=g, device=dev).to(dtype)
    dout, dt = (torch.randn(N, D, generator=g, device=dev).to(dtype) for _ in range(2))
    rstd = torch.rsqrt(x.double().square().mean(-1) + 1e-6).float()
    for w in (torch.randn(D, generator=g, device=dev).to(dtype), torch.randn(D, generator=g, device=dev), None):
        gw = dout.double() * (1.0 if w is None else w.double())
        n = x.double() * rstd.double()[:, None]
        inner, size = (gw * n).mean(-1, keepdim=True), (gw * n).abs().mean(-1, keepdim=True)
        for extra in (None, dt):
            dX, dw = km.kmassign_rmsnorm_grad(dout, x, w, rstd, dtotal=extra)
            ref = rstd.double()[:, None] * (gw - n * inner)
            err = rstd.double()[:, None] * (8 * U * (gw.abs() + (n * inner).abs())
                                            + n.abs() * size * (sums_of(D) + 8) * U)
            if extra is not None:
                ref = ref + extra.double()
                err = err + U * ref.abs()
            tiny = 2.0 ** -25 if dtype == FP16 else 0.0
            assert ((dX.double() - ref).abs() <= err + OUT[dtype] * (ref.abs() + err) * 1.001 + tiny).all()
            assert (dw is None) == (w is None)
            if w is not None:
                each = dout.double() * n
                assert ((dw.double() - each.sum(0)).abs() <= (N + 3) * U * each.abs().sum(0)).all()
    again = km.kmassign_rmsnorm_grad(dout, x, None, rstd, dtotal=dt, dX=dt)[0]
    assert again is dt and torch.equal(again, dX)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16], ids=str)
@pytest.mark.parametrize("N,D", [(12000, 40), (12000, 33), (3000, 500), (4000, 129), (11000, 256)])
def test_norm_gradients_of_many_rows(dev, N, D, dtype):
    """More rows than are in flight, so that each group takes several in turn; in place as well."""
    test_norm_gradients(dev, N, D, dtype)
    g = gen_of(dev, 6)
    x, dout, w = (torch.randn(*shape, generator=g, device=dev).to(dtype) for shape in ((N, D), (N, D), (D,)))
    rstd = torch.rand(N, generator=g, device=dev)
    dX, dw = km.kmassign_rmsnorm_grad(dout, x, w, rstd)
    rows = torch.randperm(N, generator=g, device=dev)[:100]
    few, _ = km.kmassign_rmsnorm_grad(dout[rows], x[rows], w, rstd[rows])
    there, again = km.kmassign_rmsnorm_grad(dout, x, w, rstd, dX=dout)
    assert there is dout and torch.equal(there, dX) and torch.equal(again, dw)
    # Other rows beside it leave a row's sum as it was, but for the number of warps it takes: 2 (sums_of(D) + 8)
    # roundings of |n| mean |g n| < 10, and half a step of the result on both sides.
    assert torch.allclose(few.double(), dX[rows].double(), rtol=2 * OUT[dtype] + 1e-5, atol=1e-4)


def test_norm_gradients_are_differences(dev):
    g = gen_of(dev, 5)
    N, D, h = 4, 24, 1e-5
    x, w, c = (torch.randn(*s, generator=g, device=dev) for s in ((N, D), (D,), (N, D)))
    _, _, _, rstd = km.kmassign_rmsnorm(x, w)
    dX, dw = km.kmassign_rmsnorm_grad(c, x, w, rstd)

    def loss(x, w):
        return (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w * c.double()).sum()
    for i in range(D):
        step = torch.zeros(N, D, device=dev, dtype=torch.float64)
        step[i % N, i] = h
        slope = (loss(x.double() + step, w.double()) - loss(x.double() - step, w.double())) / (2 * h)
        # 64-bit rounding of the loss over 2h, h^2 of the third derivative, and the gradient's fp32
        assert (dX[i % N, i].double() - slope).abs() <= 1e-8 + 200 * U * 50
        slope = (loss(x.double(), w.double() + step[i % N]) - loss(x.double(), w.double() - step[i % N])) / (2 * h)
        assert (dw[i].double() - slope).abs() <= 1e-8 + 200 * U * 50


def test_nothing_in_nothing_out(dev):
    W = torch.ones(3, 16, 8, device=dev, dtype=BF16)
    off = torch.zeros(4, device=dev, dtype=torch.int32)
    none = torch.zeros(0, 8, device=dev, dtype=BF16)
    empty = torch.zeros(0, device=dev, dtype=torch.int32)
    assert km.kmassign_experts(none, W, off).shape == (0, 16)
    dX, dW = km.kmassign_experts_grad(torch.zeros(0, 16, device=dev, dtype=BF16), none, W, off)
    assert dX.shape == (0, 8) and (dW == 0).all()
    X = torch.ones(4, 8, device=dev, dtype=BF16)
    dX, dW = km.kmassign_experts_grad(torch.zeros(0, 16, device=dev, dtype=BF16), X, W, off, rows=empty)
    assert (dX == 0).all() and (dW == 0).all()
    # four positions that name rows of nothing: zeros
    rows = torch.arange(4, device=dev).int()
    assert (km.kmassign_experts(none, W, offsets_of([2, 1, 1], dev), rows=rows) == 0).all()
    out, scales, _, rstd = km.kmassign_rmsnorm(none, dtype=E4M3)
    assert out.shape == (0, 8) and scales.shape == (0, 1) and rstd.shape == (0,)
    dX, dw = km.kmassign_rmsnorm_grad(none, none, torch.ones(8, device=dev), rstd)
    assert dX.shape == (0, 8) and (dw == 0).all()


def test_elements_past_32_bits(dev):
    """Outputs of more than 2^31 elements, checked at both ends."""
    g = gen_of(dev, 13)
    M, D, F = 1_100_000, 16, 2048
    X, W = ints(g, (M, D), 2, BF16), ints(g, (2, F, D), 2, BF16)
    ends = torch.tensor([0, 1, M // 2, M - 2, M - 1], device=dev)
    out = km.kmassign_experts(X, W, offsets_of([5, M - 5], dev))
    ref = torch.stack([X[i].double() @ W[int(i >= 5)].double().t() for i in ends.tolist()])
    assert torch.equal(out[ends], ref.to(BF16))
    dX, _ = km.kmassign_experts_grad(out, X, W, offsets_of([5, M - 5], dev), need_w=False)
    ref = torch.stack([out[i].double() @ W[int(i >= 5)].double() for i in ends.tolist()])
    assert torch.equal(dX[ends], ref.to(BF16))
    del out, dX
    E, F, D = 1024, 2048, 1032
    X, dout = ints(g, (2 * E, D), 2, BF16), ints(g, (2 * E, F), 2, BF16)
    _, dW = km.kmassign_experts_grad(dout, X, torch.empty(E, F, D, device=dev, dtype=BF16),
                                     offsets_of([2] * E, dev), need_x=False, dtype=BF16)
    for e in (0, 511, 1023):
        ref = dout[2 * e:2 * e + 2].double().t() @ X[2 * e:2 * e + 2].double()
        assert torch.equal(dW[e], ref.to(BF16))
    del dW
    N, D = 70_000, 32768
    x = torch.empty(N, D, device=dev, dtype=BF16).normal_(generator=g)
    out, _, _, rstd = km.kmassign_rmsnorm(x)
    dX, _ = km.kmassign_rmsnorm_grad(x, x, None, rstd)
    for i in (0, N - 1):
        srstd, y = ref_norm(x[i:i + 1], None, 1e-6)
        rel = (sums_of(D) / 2 + 8) * U
        assert ((out[i].double() - y[0]).abs() <= (rel + 2 * U + OUT[BF16]) * y[0].abs() * 1.001).all()
        n = x[i].double() * rstd[i].double()
        want = rstd[i].double() * (x[i].double() - n * (x[i].double() * n).mean())
        size = x[i].double().abs() + n.abs() * (x[i].double() * n).abs().mean()
        err = rstd[i].double() * (sums_of(D) + 16) * U * size
        assert ((dX[i].double() - want).abs() <= err + OUT[BF16] * (want.abs() + err) * 1.001).all()


@pytest.mark.parametrize("M", [20_000, 70_000])
def test_the_largest_number_of_lists(dev, M):
    """1,024 of them, with narrow and wide tiles, forward and back, in 16 and 8 bits."""
    g = gen_of(dev, M)
    E, D, F = 1024, 16, 24
    lengths = spread(M, E, g)
    off = offsets_of(lengths, dev)
    expert = torch.arange(E, device=dev).repeat_interleave(torch.tensor(lengths, device=dev))
    X, W, dout = ints(g, (M, D), 3, BF16), ints(g, (E, F, D), 3, BF16), ints(g, (M, F), 2, BF16)
    w = W.double()[expert]
    ref = torch.einsum("md,mfd->mf", X.double(), w)
    assert torch.equal(km.kmassign_experts(X, W, off), ref.to(BF16))
    rows = torch.randperm(M, generator=g, device=dev).int()
    out = km.kmassign_experts(X, W, off, rows=rows, places=rows)
    want = torch.empty_like(ref)
    want[rows.long()] = torch.einsum("md,mfd->mf", X.double()[rows.long()], w)
    assert torch.equal(out, want.to(BF16))
    dX, dW = km.kmassign_experts_grad(dout, X, W, off)
    assert torch.equal(dX, torch.einsum("mf,mfd->md", dout.double(), w).to(BF16))
    each = torch.einsum("mf,md->mfd", dout.double(), X.double())
    assert torch.equal(dW, torch.zeros(E, F, D, dtype=torch.float64, device=dev).index_add_(0, expert, each).float())
    q, v, xs, ws = whole_8_bits(g, M, D, E, F)
    x, w = values(q, v, xs, ws)
    ref = torch.einsum("md,mfd->mf", x, w[expert])
    assert torch.equal(km.kmassign_experts(q, v, off, xscale=xs, wscale=ws, dtype=FP32), ref.float())


# ---- how calls are made -----------------------------------------------------------------

def test_captured_calls_replay(dev):
    """A forward and backward pass in two graphs that hold workspaces, replayed in turn with new inputs."""
    g = gen_of(dev, 7)
    N, k, E, D, F = 200, 2, 4, 64, 72
    W = ints(g, (E, F, D), 2, BF16)
    X, dout = ints(g, (N, D), 2, BF16), ints(g, (N * k, F), 2, BF16)
    idx = torch.randint(0, E, (N, k), generator=g, device=dev).int()

    def step():
        order, off = km.kmassign_lists(idx, E)
        out = km.kmassign_experts(X, W, off, rows=order, slots=k)
        dX, dW = km.kmassign_experts_grad(dout, X, W, off, rows=order, slots=k)
        y, scales, _, rstd = km.kmassign_rmsnorm(X, W[0, 0], dtype=E4M3)
        return out, dX, dW, y.float(), scales, km.kmassign_rmsnorm_grad(X, X, W[0, 0], rstd)[1]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
            graph_outs = graphs[-1][1]
        assert len(graph_outs) == 6
    for seed in range(3):
        X.copy_(ints(gen_of(dev, 100 + seed), (N, D), 2, BF16))
        idx.copy_(torch.randint(-1, E, (N, k), generator=gen_of(dev, seed), device=dev).int())
        for graph, outs in graphs:
            graph.replay()
        want = step()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_on_two_streams_at_once(dev):
    g = gen_of(dev, 8)
    E, M, D, F = 8, 3000, 512, 512
    off = offsets_of([M // E] * E, dev)
    sets = [(ints(g, (M, D), 2, BF16), ints(g, (E, F, D), 2, BF16), ints(g, (M, F), 2, BF16)) for _ in range(2)]
    rows = torch.randperm(M, generator=g, device=dev).int()

    def run(X, W, d, stream=None):
        out = km.kmassign_experts(X, W, off, rows=rows, stream=stream)
        return (out, *km.kmassign_experts_grad(d, X, W, off, rows=rows, stream=stream))
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [run(*s, stream=t) for s, t in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("E,per,D,F", [(16, 2048, 2048, 1024), (4, 10, 32768, 2048)])
def test_short_wait_bound_reports_timeout_and_context_survives(dev, E, per, D, F):
    """A wait is only held against the bound when a try of the hardware's own has come back without
    the phase, so that the products here are those with long waits (segments of 32 k-blocks)."""
    g = gen_of(dev, 6)
    M = E * per
    X, W, d = ints(g, (M, D), 1, BF16), ints(g, (E, F, D), 1, BF16), ints(g, (M, F), 1, BF16)
    off = offsets_of([per] * E, dev)
    calls = [lambda: km.kmassign_experts(X, W, off),
             lambda: km.kmassign_experts_grad(d, X, W, off, need_w=False)[0]]
    for call in calls:
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


def test_python_refusals(dev):
    X, W = torch.ones(6, 16, device=dev, dtype=BF16), torch.ones(2, 8, 16, device=dev, dtype=BF16)
    off = offsets_of([3, 3], dev)
    rows = torch.arange(6, device=dev).int()
    q, v = X.to(E4M3), W.to(E4M3)
    s, t = torch.ones(6, 1, device=dev), torch.ones(2, 1, 1, device=dev)
    d = torch.ones(6, 8, device=dev, dtype=BF16)
    for call, error, text in [
        (lambda: km.kmassign_experts(X.float(), W, off), TypeError, "bfloat16"),
        (lambda: km.kmassign_experts(X, W.half(), off), TypeError, "W must be"),
        (lambda: km.kmassign_experts(X, W), ValueError, "shape"),
        (lambda: km.kmassign_experts(X, W[0], off), ValueError, "shape"),
        (lambda: km.kmassign_experts(X, W[:, :, :8].contiguous(), off), ValueError, "disagree"),
        (lambda: km.kmassign_experts(X[:, ::2], W, off), ValueError, "contiguous"),
        (lambda: km.kmassign_experts(X, W, off.long()), TypeError, "offsets"),
        (lambda: km.kmassign_experts(X, W, off[:2]), ValueError, "offsets"),
        (lambda: km.kmassign_experts(X, W, off, rows=rows.long()), TypeError, "rows"),
        (lambda: km.kmassign_experts(X, W, off, slots=2), ValueError, "slots"),
        (lambda: km.kmassign_experts(X, W, off, rows=rows, slots=0), ValueError, "slots"),
        (lambda: km.kmassign_experts(X, W, off, rows=rows, slots=2**32 + 1), ValueError, "slots"),
        (lambda: km.kmassign_experts(q, v, off, xscale=s.clone().requires_grad_(), wscale=t), RuntimeError, "requires grad"),
        (lambda: km.kmassign_experts(X, W, off, rows=rows, places=rows[:5]), ValueError, "places"),
        (lambda: km.kmassign_experts(X, W, off, out=d[:5]), ValueError, "out"),
        (lambda: km.kmassign_experts(X, W, off, out=d.half()), TypeError, "out"),
        (lambda: km.kmassign_experts(X, W, off, dtype=FP16), TypeError, "out"),
        (lambda: km.kmassign_experts(X, W, off, xscale=s, wscale=t), ValueError, "8-bit"),
        (lambda: km.kmassign_experts(q, v, off), ValueError, "xscale"),
        (lambda: km.kmassign_experts(q, v, off, xscale=s[:5], wscale=t), ValueError, "xscale"),
        (lambda: km.kmassign_experts(q, v, off, xscale=s, wscale=t[0]), ValueError, "wscale"),
        (lambda: km.kmassign_experts(X[:, :12].contiguous(), W[:, :, :12].contiguous(), off), km.KmassignError, "UNSUPPORTED_D"),
        (lambda: km.kmassign_experts(X.requires_grad_(), W, off), RuntimeError, "requires grad"),
        (lambda: km.kmassign_experts_grad(d, X.detach(), W.clone().requires_grad_(), off), RuntimeError, "requires grad"),
        (lambda: km.kmassign_experts_grad(d[:5], X, W, off), ValueError, "dout"),
        (lambda: km.kmassign_experts_grad(d, q, v, off), TypeError, "e4m3|float8"),
        (lambda: km.kmassign_experts_grad(d, X, W, off, need_x=False, need_w=False), ValueError, "neither"),
        (lambda: km.kmassign_experts_grad(d, X, W, off, need_x=False, dX=X), ValueError, "not needed"),
        (lambda: km.kmassign_rmsnorm(X.detach(), s[:, 0]), ValueError, "weight"),
        (lambda: km.kmassign_rmsnorm(X.detach(), dtype=FP16), TypeError, "dtype"),
        (lambda: km.kmassign_rmsnorm(X.detach(), total=d), ValueError, "residual"),
        (lambda: km.kmassign_rmsnorm(X.detach(), scales=s), ValueError, "8-bit"),
        (lambda: km.kmassign_rmsnorm(X), RuntimeError, "requires grad"),
        (lambda: km.kmassign_rmsnorm_grad(d, d, None, s[:, 0].contiguous(), dweight=s), ValueError, "weight"),
    ]:
        with pytest.raises(error, match=text):
            call()


def test_writes_to_given_tensors_count_a_version(dev):
    X, W = torch.ones(6, 16, device=dev, dtype=BF16), torch.ones(2, 8, 16, device=dev, dtype=BF16)
    off, d = offsets_of([3, 3], dev), torch.ones(6, 8, device=dev, dtype=BF16)
    rstd = torch.ones(6, device=dev)
    f = torch.zeros
    cases = [
        (lambda o: km.kmassign_experts(X, W, off, out=o[0]), [f(6, 8, device=dev, dtype=BF16)]),
        (lambda o: km.kmassign_experts_grad(d, X, W, off, dX=o[0], dW=o[1]), [X.clone(), f(2, 8, 16, device=dev)]),
        (lambda o: km.kmassign_rmsnorm(X, residual=X, out=o[0], total=o[1], rstd=o[2]), [X.clone(), X.clone(), rstd.clone()]),
        (lambda o: km.kmassign_rmsnorm_grad(X, X, W[0, 0], rstd, dX=o[0], dweight=o[1]), [X.clone(), f(16, device=dev)]),
    ]
    for call, outs in cases:
        versions = [o._version for o in outs]
        call(outs)
        assert all(o._version > v for o, v in zip(outs, versions))
    assert X._version == W._version == d._version == 0


# ---- together ----------------------------------------------------------------------------

def test_a_layer_of_experts_in_8_bits(dev):
    """Norm, routing, lists, products in 8 bits, combination: against the same steps in 64 bits."""
    g = gen_of(dev, 11)
    N, k, E, D, F = 300, 2, 6, 256, 136
    x, r = (torch.randn(N, D, generator=g, device=dev).to(BF16) for _ in range(2))
    w = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(BF16)
    q, _ = ints(g, (E, F, D), 8, FP32).to(E4M3), None
    ws = torch.rand(E, -(-F // 128), 2, generator=g, device=dev) * 0.01 + 0.005
    logits = torch.randn(N, E, generator=g, device=dev)
    h, hs, total, rstd = km.kmassign_rmsnorm(x, w, residual=r, dtype=E4M3)
    idx, gate = km.kmassign_route(logits, k)
    order, off = km.kmassign_lists(idx, E)
    y = km.kmassign_experts(h, q, off, rows=order, slots=k, places=order, xscale=hs, wscale=ws)
    at = torch.arange(N * k, device=dev).view(N, k).int()
    out = km.kmassign_lookup(y, at, weights=gate)
    xv, wv = values(h, q, hs, ws)
    ref = torch.stack([torch.einsum("nd,nfd->nf", xv, wv[idx[:, j].long()]) for j in range(k)], 1)
    size = torch.stack([torch.einsum("nd,nfd->nf", xv.abs(), wv[idx[:, j].long()].abs()) for j in range(k)], 1)
    err = OUT[BF16] * ref.abs() + 8 * U * size
    want = (ref * gate.double()[..., None]).sum(1)
    bound = (err * gate.double()[..., None]).sum(1) * 1.01 + (OUT[BF16] + 8 * U) * want.abs() + 8 * U * size.sum(1)
    assert ((out.double() - want).abs() <= bound).all()


def test_training_a_layer_of_experts(dev):
    """The gradients of norm, routing weights, products and combination against autograd in 64 bits."""
    g = gen_of(dev, 12)
    N, k, E, D, F = 150, 2, 4, 64, 72
    x = torch.randn(N, D, generator=g, device=dev).to(FP16)
    w = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(FP16)
    W = (torch.randn(E, F, D, generator=g, device=dev) / 8).to(FP16)
    logits = torch.randn(N, E, generator=g, device=dev)
    dout = torch.randn(N, F, generator=g, device=dev).to(FP16)
    at = torch.arange(N * k, device=dev).view(N, k).int()

    h, _, total, rstd = km.kmassign_rmsnorm(x, w)
    idx, gate = km.kmassign_route(logits, k)
    order, off = km.kmassign_lists(idx, E)
    lists = dict(rows=order, slots=k, places=order)
    y = km.kmassign_experts(h, W, off, **lists)
    dy, dgate = km.kmassign_lookup_grad(dout, at, N * k, weights=gate, table=y, dtype=FP16)
    dh, dW = km.kmassign_experts_grad(dy, h, W, off, **lists)
    dx, dw = km.kmassign_rmsnorm_grad(dh, total, w, rstd)
    dlogits = km.kmassign_route_grad(logits, idx, dgate)

    X, V, G, L = (t.detach().double().requires_grad_() for t in (x, w, W, logits))
    hh = X / (X.square().mean(-1, keepdim=True) + 1e-6).sqrt() * V
    p = torch.softmax(L.gather(1, idx.long()), -1)
    yy = torch.stack([torch.einsum("nd,nfd->nf", hh, G[idx[:, j].long()]) for j in range(k)], 1)
    ((yy * p[..., None]).sum(1) * dout.double()).sum().backward()
    # every intermediate is rounded to fp16 once, half an ulp of 2^-11 relative each: h, y, dy, a
    # position's product, dh, and the result; a gradient's norm is off by no more than their sum
    for got, want in ((dx, X.grad), (dw, V.grad), (dW, G.grad), (dlogits, L.grad)):
        assert (got.double() - want).norm() <= 6 * 2.0 ** -11 * want.norm()


def test_the_measured_cases_agree_with_their_plain_forms(dev):
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    for case in cases.listed():
        small = dict(case, N=min(case["N"], 257))
        state = cases.prepare(small, 1)
        cases.own = False
        want = cases.run(state)
        cases.own = True
        got = cases.run(state)
        for a, b in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, want))):
            if b is None:
                assert a is None
                continue
            assert a.dtype == b.dtype and a.shape == b.shape
            # roundings to 8 bits may fall the other way beside a border, by a step
            share = {E4M3: 2.0 ** -6, BF16: 2.0 ** -7, FP16: 2.0 ** -10, FP32: 2.0 ** -16}[a.dtype]
            assert (a.double() - b.double()).norm() <= share * b.double().norm(), case["name"]
