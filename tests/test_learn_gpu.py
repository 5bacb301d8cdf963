"""Routing, lookup, their gradients, inverted lists and clipping on the GPU,
against plain 64-bit implementations (numpy).

Tolerances.  U = 2^-24 is half an fp32 ulp; OUT[type] half an ulp of an output
type, relative.  Sums of n fp32 terms are allowed n roundings of the sum of
magnitudes.  expf is allowed 2 ulp, and exp(x - m) the rounding of x - m, which
is relative |x - m| U.  Choices without a bias, lists and integer-valued sums
are exact."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import means_nearest_centroid_gb300 as km

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-44, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from means_nearest_centroid_gb300 import _build
    _build.build()
    km.library()
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- routing ----------------------------------------------------------------

def ref_scores(x, score):
    off = ~(x > -INF)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return off, np.where(off, 0.0, 1.0 / (1.0 + np.exp(-x)))
        m = np.max(np.where(off, -INF, x), 1, keepdims=True)
        p = np.where(off, 0.0, np.exp(x - m))
        return off, np.where(p > 0, p / p.sum(1, keepdims=True), 0.0)


def ref_keys(x, score, bias, groups, topk_groups, top):
    """Keys of the experts still in the choice (-inf: not selectable), in 64 bits."""
    off, s = ref_scores(x, score)
    key = np.where(off, -INF, x if bias is None else s + bias)
    key = np.where(np.isnan(key), -INF, key)
    if topk_groups < groups:
        N, E = x.shape
        m = key if bias is not None or top == 1 else np.where(off, -INF, s)
        m = -np.sort(-m.reshape(N, groups, -1), 2)[:, :, :top]
        g = np.where(m[:, :, 0] == -INF, -INF, np.where(m == -INF, 0.0, m).sum(2))
        out = np.argsort(-g, 1, kind="stable")[:, topk_groups:]
        gone = np.zeros((N, groups), bool)
        np.put_along_axis(gone, out, True, 1)
        key = np.where(np.repeat(gone, E // groups, 1), -INF, key)
    return key, s


def ref_choice(key, k):
    idx = np.argsort(-key, 1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(key, idx, 1) == -INF, -1, idx)


def ref_weights(x, s, idx, score, renorm, scale):
    at = np.maximum(idx, 0)
    live = idx >= 0
    w = np.where(live, np.take_along_axis(s, at, 1), 0.0)
    if renorm and score == "softmax":
        c = np.where(live, np.take_along_axis(x, at, 1), -INF)
        with np.errstate(all="ignore"):
            w = np.where(live, np.exp(c - c.max(1, keepdims=True)), 0.0)
    if renorm:
        t = w.sum(1, keepdims=True)
        w = np.where(t > 0, w / np.where(t > 0, t, 1.0), 0.0)
    return w * scale


def weight_bound(x, k):
    E = x.shape[1]
    spread = np.where(np.isfinite(x), np.abs(x), 0.0).max()
    return (2 * min(spread, 104.0) + E / 8 + k + 12) * 2 * U


def make_logits(N, E, dtype, seed, mask=0.05):
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(N, E, generator=g)
    x[torch.rand(N, E, generator=g) < mask] = -INF
    x[torch.rand(N, E, generator=g) < mask / 4] = NAN
    x[torch.rand(N, E, generator=g) < mask / 4] = torch.finfo(dtype).min
    if N > 4:
        x[1] = -INF                      # nothing to select
        x[2] = 0.5                       # all equal
        x[3] = -INF
        x[3, E // 2] = 1.0               # one expert only
        x[4] = torch.finfo(dtype).min    # lowest value everywhere: ordinary numbers
    return x.to(dtype)


SHAPES = [(1, 1, 1), (5, 2, 2), (37, 7, 3), (64, 8, 8), (33, 16, 5), (19, 31, 31), (50, 32, 32),
          (21, 33, 4), (40, 64, 6), (17, 72, 6), (9, 128, 1), (30, 200, 16), (65, 256, 8),
          (7, 384, 32), (6, 512, 10), (5, 777, 7), (8, 1024, 32)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k", SHAPES)
def test_route_without_bias(dev, N, E, k, score, dtype):
    X = make_logits(N, E, dtype, seed=N * 1000 + E)
    x = f64(X)
    key, s = ref_keys(x, score, None, 1, 1, 2)
    want = ref_choice(key, k)
    for renorm in (False, True):
        idx, w = km.kmassign_route(X.to(dev), k, score=score, renorm=renorm, scale=2.5)
        assert np.array_equal(idx.cpu().numpy(), want)
        ref = ref_weights(x, s, want, score, renorm, 2.5)
        assert np.all(np.abs(f64(w) - ref) <= weight_bound(x, k) * ref + 2 ** -125)


GROUPS = [(33, 16, 3, 4, 2), (20, 32, 4, 8, 3), (65, 256, 8, 8, 4), (11, 96, 6, 3, 2), (9, 160, 5, 32, 7),
          (12, 24, 2, 12, 5), (8, 128, 16, 16, 2), (10, 30, 10, 2, 1), (13, 62, 3, 31, 30), (7, 6, 1, 6, 2),
          (6, 32, 2, 32, 5)]


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k,groups,topk", GROUPS)
def test_route_groups(dev, N, E, k, groups, topk, score, top):
    """Groups by keys of at most 8 significant bits, so that their sums and the order of the
    sigmoid's and softmax's sums are decided far above rounding; ties go to the lower group."""
    g = torch.Generator().manual_seed(E + groups)
    X = torch.randint(-6, 7, (N, E), generator=g).float() / 2
    X[torch.rand(N, E, generator=g) < 0.1] = -INF
    X[0, : E // groups] = -INF            # a group with nothing in it
    x = f64(X)
    key, s = ref_keys(x, score, None, groups, topk, top)
    if top == 2 and topk < groups:
        # rows whose group sums are closer than rounding (but not equal) prove nothing
        off, sc = ref_scores(x, score)
        m = -np.sort(-np.where(off, -INF, sc).reshape(N, groups, -1), 2)[:, :, :2]
        gk = -np.sort(-np.where(m == -INF, 0.0, m).sum(2), 1)
        gap = gk[:, topk - 1] - gk[:, topk]
        sound = (gap > 1e-5 * gk[:, topk - 1]) | (topk == groups)
    else:
        sound = np.ones(N, bool)
    assert sound.sum() > 0
    idx, w = km.kmassign_route(X.to(dev), k, score=score, groups=groups, topk_groups=topk,
                               group_top=top)
    want = ref_choice(key, k)
    assert np.array_equal(idx.cpu().numpy()[sound], want[sound])
    ref = ref_weights(x, s, want, score, True, 1.0)
    assert np.all((np.abs(f64(w) - ref) <= weight_bound(x, k) * ref + 2 ** -125)[sound])


@pytest.mark.parametrize("groups,topk", [(1, 1), (8, 3)])
def test_route_equal_scores_follow_the_bias_exactly(dev, groups, topk):
    """All logits 0: a sigmoid's score is 0.5 exactly and the keys are the bias, ties included."""
    E, k = 64, 8
    X = torch.zeros(6, E)
    X[3, 5] = -INF
    bias = torch.randint(-4, 5, (E,), generator=torch.Generator().manual_seed(1)).float() / 8
    bias[7] = -INF
    bias[9] = NAN
    key, s = ref_keys(f64(X), "sigmoid", f64(bias), groups, topk, 2)
    idx, w = km.kmassign_route(X.to(dev), k, score="sigmoid", bias=bias.to(dev), groups=groups,
                               topk_groups=topk)
    assert np.array_equal(idx.cpu().numpy(), ref_choice(key, k))
    assert torch.equal(w.cpu(), torch.full((6, k), 0.125))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k,groups,topk", [(200, 256, 8, 8, 4), (100, 72, 6, 1, 1), (300, 16, 2, 4, 2),
                                               (64, 512, 16, 16, 16), (40, 1024, 8, 16, 5)])
def test_route_with_bias(dev, N, E, k, groups, topk, score):
    """Keys are fp32 sums of a score (a few ulp of at most 1) and a bias: a choice may differ from
    the 64-bit one only among keys within 16 U (1 + |bias|) of each other."""
    g = torch.Generator().manual_seed(N)
    X = make_logits(N, E, torch.float32, N)
    bias = 0.2 * torch.randn(E, generator=g)
    x, b = f64(X), f64(bias)
    key, s = ref_keys(x, score, b, groups, topk, 2)
    idx, w = km.kmassign_route(X.to(dev), k, score=score, bias=bias.to(dev), groups=groups,
                               topk_groups=topk, renorm=False)
    got = idx.cpu().numpy()
    want = ref_choice(key, k)
    tol = (16 + (E / 32 + 104 if score == "softmax" else 0)) * 2 * U * 2
    wrong = 0
    for i in range(N):
        if np.array_equal(got[i], want[i]):
            continue
        a, c = key[i, got[i]], key[i, want[i]]
        ok = np.array_equal(got[i] < 0, want[i] < 0) and np.all(np.abs(a - c)[want[i] >= 0] <= tol)
        wrong += 1
        assert ok or groups > topk, i
    assert wrong <= max(1, N // 50)      # near-ties are rare; a group's near-tie moves a row
    ref = ref_weights(x, s, got, score, False, 1.0)
    assert np.all(np.abs(f64(w) - ref) <= weight_bound(x, k) * ref + 2 ** -125)


def test_route_infinite_logit(dev):
    X = torch.tensor([[0.0, INF, 1.0, -INF]], device=dev)
    idx, w = km.kmassign_route(X, 2, score="sigmoid")
    assert idx.tolist() == [[1, 2]] and abs(w.sum().item() - 1.0) < 4 * U
    idx, w = km.kmassign_route(X, 2, score="softmax")
    assert idx.tolist() == [[1, 2]] and torch.isnan(w).all()


def test_route_underflowing_selection(dev):
    """Sigmoids that are all 0 in fp32 give weights 0; a renormalised softmax far below the row's
    best expert (which a bias keeps out) does not underflow."""
    X = torch.full((1, 8), -200.0, device=dev)
    idx, w = km.kmassign_route(X, 3, score="sigmoid")
    assert idx.tolist() == [[0, 1, 2]] and w.tolist() == [[0.0, 0.0, 0.0]]
    X[0, 4] = 100.0
    bias = torch.zeros(8, device=dev)
    bias[4] = -INF
    idx, w = km.kmassign_route(X, 2, score="softmax", bias=bias)
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


def test_route_offsets_past_32_bits(dev):
    N, E = 4_400_000, 1000               # 4.4e9 elements
    X = torch.zeros(N, E, dtype=torch.bfloat16, device=dev)
    X[N - 1, 777] = 3.0
    X[N - 1, 11] = 2.0
    idx, w = km.kmassign_route(X, 2)
    assert idx[N - 1].tolist() == [777, 11] and idx[N - 2].tolist() == [0, 1]
    dw = torch.ones(N, 2, device=dev)
    dw[:, 1] = -1.0
    d = km.kmassign_route_grad(X, idx, dw)
    p = 1 / (1 + np.exp(-1.0))
    assert abs(d[N - 1, 777].item() - 2 * p * (1 - p)) < 2 ** -8
    assert d[N - 2, 0].item() == 0.5 and d[N - 2, 1].item() == -0.5 and d[N - 2, 2:].abs().max().item() == 0


def ref_route_grad(x, idx, dw, score, renorm, scale):
    N, E = x.shape
    ok = (idx >= 0) & (idx < E)
    off, s = ref_scores(x, score)
    G = np.zeros((N, E))
    sel = np.zeros((N, E), bool)
    for i in range(N):
        G[i, idx[i][ok[i]]] = dw[i][ok[i]]
        sel[i, idx[i][ok[i]]] = True
    sel &= ~off
    G = np.where(sel, G, 0.0)
    if score == "sigmoid":
        slope = np.where(off, 0.0, s * (1 - s))
        if not renorm:
            return scale * slope * G, scale * slope * np.abs(G)
        t = np.where(sel, s, 0.0).sum(1, keepdims=True)
        t1 = np.where(t > 0, t, 1.0)
        mean, amean = (s * G).sum(1, keepdims=True) / t1, (s * np.abs(G)).sum(1, keepdims=True) / t1
        f = np.where(sel & (t > 0), scale * slope / t1, 0.0)
        return f * (G - mean), f * (np.abs(G) + amean)
    if renorm:
        c = np.where(sel, x, -INF)
        with np.errstate(all="ignore"):
            p = np.where(sel, np.exp(c - c.max(1, keepdims=True)), 0.0)
        t = p.sum(1, keepdims=True)
        p = p / np.where(t > 0, t, 1.0)
    else:
        p = s
    return (scale * p * (G - (p * G).sum(1, keepdims=True)),
            scale * p * (np.abs(G) + (p * np.abs(G)).sum(1, keepdims=True)))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k", SHAPES)
def test_route_grad(dev, N, E, k, score, renorm, dtype):
    X = make_logits(N, E, dtype, seed=N + E)
    Xd = X.to(dev)
    idx, _ = km.kmassign_route(Xd, k, score=score)
    g = torch.Generator().manual_seed(3)
    dw = torch.randn(N, k, generator=g)
    idx[-1, 0] = E + 3                        # an id of no expert
    dw[idx.cpu() < 0] = NAN                   # what stands at free slots is ignored
    d = km.kmassign_route_grad(Xd, idx, dw.to(dev), score=score, renorm=renorm, scale=2.5)
    ref, size = ref_route_grad(f64(X), idx.cpu().numpy(), f64(dw), score, renorm, 2.5)
    bound = 2 * weight_bound(f64(X), k) * size + OUT[dtype] * np.abs(ref) + TINY[dtype] + 2 ** -120
    assert d.dtype == dtype
    assert np.all(np.abs(f64(d) - ref) <= bound)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_grad_against_differences(dev, score, renorm):
    """Central differences (step 1e-5, in 64 bits) of sum dw * w with the choice held: their error
    is below 1e-8 here, fp32's is that of test_route_grad."""
    N, E, k = 4, 12, 3
    X = torch.randn(N, E, generator=torch.Generator().manual_seed(5))
    idx, _ = km.kmassign_route(X.to(dev), k, score=score)
    dw = torch.randn(N, k, generator=torch.Generator().manual_seed(6))
    d = f64(km.kmassign_route_grad(X.to(dev), idx, dw.to(dev), score=score, renorm=renorm, scale=1.5))
    x, i, h = f64(X), idx.cpu().numpy(), 1e-5

    def loss(z):
        return (f64(dw) * ref_weights(z, ref_scores(z, score)[1], i, score, renorm, 1.5)).sum()
    for a in range(N):
        for e in range(E):
            up, down = x.copy(), x.copy()
            up[a, e] += h
            down[a, e] -= h
            assert abs(d[a, e] - (loss(up) - loss(down)) / (2 * h)) <= 1e-8 + 64 * U


# ---- lists --------------------------------------------------------------------

def check_lists(dev, ids, K):
    order, offsets = km.kmassign_lists(torch.from_numpy(ids).to(dev), K)
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < K)
    at = np.nonzero(ok)[0]
    want = at[np.argsort(flat[at], kind="stable")]
    o = order.cpu().numpy()
    assert np.array_equal(o[: len(want)], want) and np.all(o[len(want):] == -1)
    counts = np.bincount(flat[at], minlength=K)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))


@pytest.mark.parametrize("M", [1, 2, 31, 33, 1000, 1024, 1025, 4095, 4096, 4097, 10000, 155648, 155649,
                               700_001])
@pytest.mark.parametrize("K", [1, 2, 3, 255, 256, 257, 1024, 1025, 5000, 8192, 8193, 100_000, 1_500_000])
def test_lists(dev, M, K):
    g = np.random.default_rng(M + K)
    check_lists(dev, g.integers(-2, K + 2, M).astype(np.int32), K)


@pytest.mark.parametrize("M", [300, 50_000])
@pytest.mark.parametrize("K", [40, 70_000])
def test_lists_extremes(dev, M, K):
    g = np.random.default_rng(0)
    for ids in (np.full(M, K - 1), np.zeros(M), np.full(M, -1), np.full(M, K), np.arange(M)[::-1] % K,
                np.where(g.random(M) < 0.9, 7, g.integers(0, K, M)), np.full(M, 2**31 - 1),
                np.full(M, -2**31)):
        check_lists(dev, ids.astype(np.int32), K)


def test_lists_shape_and_empty(dev):
    check_lists(dev, np.arange(24, dtype=np.int32).reshape(6, 4) % 5, 5)
    order, offsets = km.kmassign_lists(torch.empty(0, dtype=torch.int32, device=dev), 7)
    assert order.numel() == 0 and offsets.tolist() == [0] * 8


def test_lists_many_ids(dev):
    g = np.random.default_rng(4)
    check_lists(dev, (g.random(5_000_000) ** 3 * 30_000).astype(np.int32), 30_000)


def test_lists_of_an_assignment(dev):
    """The inverted file of a k-means assignment: each list holds its centroid's points."""
    import workloads
    X, C = workloads.blobs(5000, 300, 64, seed=3)
    idx = km.kmassign(X.to(dev), C.to(dev))
    check_lists(dev, idx.cpu().numpy(), 300)


# ---- lookup -------------------------------------------------------------------

def make_ids(N, k, K, seed):
    g = np.random.default_rng(seed)
    ids = (g.random((N, k)) ** 2 * K).astype(np.int32)
    ids[g.random((N, k)) < 0.1] = -1
    ids[g.random((N, k)) < 0.05] = K
    if N > 2:
        ids[1] = -7                          # a point of no row
    return torch.from_numpy(ids)


def ref_lookup(t, ids, w, scale):
    ok = (ids >= 0) & (ids < t.shape[0])
    c = np.where(ok, w, 0.0) * scale
    rows = t[np.where(ok, ids, 0)]
    return (rows * c[..., None]).sum(1), (np.abs(rows) * np.abs(c)[..., None]).sum(1)


LOOKUPS = [(1, 1, 1, 1), (7, 1, 5, 3), (50, 1, 1000, 64), (33, 2, 40, 100), (65, 8, 300, 256), (20, 9, 64, 250),
           (5, 33, 50, 17), (300, 1, 50, 1025), (3, 4, 9, 4096), (129, 3, 77, 8)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,k,K,D", LOOKUPS)
def test_lookup(dev, N, k, K, D, dtype):
    g = torch.Generator().manual_seed(D)
    T = torch.randn(K, D, generator=g).to(dtype)
    ids = make_ids(N, k, K, D)
    w = torch.randn(N, k, generator=g)
    w[(ids < 0) | (ids >= K)] = NAN          # weights of skipped ids are not read into the sum
    Td = T.to(dev)
    for weights in (None, w):
        shaped = ids if k > 1 else ids.reshape(N)
        wd = None if weights is None else weights.reshape(shaped.shape).to(dev)
        out = km.kmassign_lookup(Td, shaped.to(dev), weights=wd, scale=0.75)
        ref, size = ref_lookup(f64(T), ids.numpy(), np.ones((N, k)) if weights is None else np.nan_to_num(f64(w)),
                               0.75)
        bound = (k + 2) * U * size + OUT[dtype] * np.abs(ref) + TINY[dtype]
        assert np.all(np.abs(f64(out) - ref) <= bound)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("D,shift", [(64, 0), (64, 1), (64, 2), (64, 4), (63, 0), (62, 1), (60, 0), (1, 0)])
def test_lookup_copies_bits_at_any_alignment(dev, D, shift, dtype):
    buf = torch.randn(100 * D + 8, generator=torch.Generator().manual_seed(1)).to(dtype).to(dev)
    T = buf[shift: shift + 100 * D].view(100, D)
    ids = torch.randint(0, 100, (41,), generator=torch.Generator().manual_seed(2)).int().to(dev)
    outs = torch.full((41 * D + 8,), 7.0, dtype=dtype, device=dev)
    out = outs[shift: shift + 41 * D].view(41, D)
    km.kmassign_lookup(T, ids, out=out)
    assert torch.equal(out, T[ids.long()])
    assert (outs[:shift] == 7).all() and (outs[shift + 41 * D:] == 7).all()


# ---- gradient of the lookup -----------------------------------------------------

def ref_lookup_grad(d, ids, w, K, scale, padding=-1):
    ok = (ids >= 0) & (ids < K) & (ids != padding)
    c = np.where(ok, w, 0.0) * scale
    out, size, n = np.zeros((K, d.shape[1])), np.zeros((K, d.shape[1])), np.zeros(K)
    i, j = np.nonzero(ok)
    np.add.at(out, ids[i, j], d[i] * c[i, j][:, None])
    np.add.at(size, ids[i, j], np.abs(d[i] * c[i, j][:, None]))
    np.add.at(n, ids[i, j], 1)
    return out, size, n


def check_grad(got, ref, size, n, dtype, extra=0.0):
    bound = (n + 3)[:, None] * U * size + OUT[dtype] * (np.abs(ref) + extra) + TINY[dtype]
    assert np.all(np.abs(f64(got) - ref) <= bound)


GRADS = LOOKUPS + [(3000, 1, 10, 65), (2000, 4, 3000, 72), (1500, 3, 2, 264), (6000, 1, 20000, 16)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,k,K,D", GRADS)
def test_lookup_grad(dev, N, k, K, D, dtype):
    g = torch.Generator().manual_seed(N)
    T = torch.randn(K, D, generator=g).to(dtype)
    dout = torch.randn(N, D, generator=g).to(dtype)
    ids = make_ids(N, k, K, N)
    w = torch.randn(N, k, generator=g)
    w[(ids < 0) | (ids >= K)] = NAN
    shaped = ids if k > 1 else ids.reshape(N)
    i = ids.numpy()
    for weights in (None, w):
        wd = None if weights is None else weights.reshape(shaped.shape).to(dev)
        w64 = np.ones((N, k)) if weights is None else np.nan_to_num(f64(w))
        ref, size, n = ref_lookup_grad(f64(dout), i, w64, K, 0.75)
        for kind in {torch.float32, dtype}:
            dt, dwt = km.kmassign_lookup_grad(dout.to(dev), shaped.to(dev), K, weights=wd,
                                              table=T.to(dev) if weights is not None else None,
                                              scale=0.75, dtype=kind)
            assert dt.dtype == kind
            check_grad(dt, ref, size, n, kind)
            again, _ = km.kmassign_lookup_grad(dout.to(dev), shaped.to(dev), K, weights=wd,
                                               table=T.to(dev) if weights is not None else None,
                                               scale=0.75, dtype=kind)
            assert torch.equal(dt, again)     # the order of every sum is fixed
        if weights is None:
            assert dwt is None
        else:
            ok = (i >= 0) & (i < K)
            rows = f64(T)[np.where(ok, i, 0)] * f64(dout)[:, None]
            want = np.where(ok, rows.sum(2) * 0.75, 0.0)
            bound = (D + 3) * U * np.where(ok, np.abs(rows).sum(2) * 0.75, 0.0)
            assert np.all(np.abs(f64(dwt).reshape(N, k) - want) <= bound)


@pytest.mark.parametrize("N,K,D", [(70_000, 3, 40), (40_000, 900, 128), (20_000, 50_000, 24), (9000, 1, 2050),
                                   (300_000, 70, 8)])
def test_lookup_grad_integers_exact(dev, N, K, D):
    """Integer data whose sums stay below 2^24: every fp32 step is exact, rows that span many
    chunks of the sorted ids included."""
    g = torch.Generator().manual_seed(K)
    dout = torch.randint(-4, 5, (N, D), generator=g).to(torch.bfloat16)
    r = np.random.default_rng(K)
    ids = np.where(r.random(N) < 0.5, 0, r.integers(0, K, N)).astype(np.int32)
    dt, _ = km.kmassign_lookup_grad(dout.to(dev), torch.from_numpy(ids).to(dev), K)
    ref, _, _ = ref_lookup_grad(f64(dout), ids[:, None], np.ones((N, 1)), K, 1.0)
    assert np.array_equal(f64(dt), ref)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_lookup_grad_accumulates_and_pads(dev, kind):
    N, K, D = 500, 60, 48
    g = torch.Generator().manual_seed(9)
    dout = torch.randn(N, D, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, 30, (N,), generator=g).int()
    old = torch.randn(K, D, generator=g).to(kind)
    got = old.clone().to(dev)
    km.kmassign_lookup_grad(dout.to(dev), ids.to(dev), K, dtable=got, accumulate=True, padding=4)
    ref, size, n = ref_lookup_grad(f64(dout), ids.numpy()[:, None], np.ones((N, 1)), K, 1.0, padding=4)
    check_grad(got, f64(old) + ref, size + np.abs(f64(old)), n + 1, kind)
    assert torch.equal(got[30:].cpu(), old[30:]) and torch.equal(got[4].cpu(), old[4])
    got.fill_(NAN)                            # written whole without accumulate
    km.kmassign_lookup_grad(dout.to(dev), ids.to(dev), K, dtable=got, padding=4)
    check_grad(got, ref, size, n, kind)
    assert (got[30:] == 0).all() and (got[4] == 0).all()


def test_lookup_grad_no_points(dev):
    d = torch.empty(0, 16, device=dev)
    i = torch.empty(0, dtype=torch.int32, device=dev)
    out = torch.full((9, 16), NAN, device=dev)
    km.kmassign_lookup_grad(d, i, 9, dtable=out)
    assert (out == 0).all()
    out.fill_(3.0)
    km.kmassign_lookup_grad(d, i, 9, dtable=out, accumulate=True)
    assert (out == 3).all()


def test_lookup_grad_at_odd_alignment(dev):
    N, K, D = 77, 20, 62
    g = torch.Generator().manual_seed(2)
    buf = torch.randn(N * D + 8, generator=g).to(torch.bfloat16).to(dev)
    ids = torch.randint(0, K, (N,), generator=g).int().to(dev)
    outs = torch.full((K * D + 8,), 7.0, dtype=torch.bfloat16, device=dev)
    dout, out = buf[1: 1 + N * D].view(N, D), outs[3: 3 + K * D].view(K, D)
    km.kmassign_lookup_grad(dout, ids, K, dtable=out)
    ref, size, n = ref_lookup_grad(f64(dout), ids.cpu().numpy()[:, None], np.ones((N, 1)), K, 1.0)
    check_grad(out, ref, size, n, torch.bfloat16)
    assert (outs[:3] == 7).all() and (outs[3 + K * D:] == 7).all()


def test_lookup_against_differences(dev):
    """Both gradients against central differences of sum dout * lookup in 64 bits (linear in the
    table and in the weights, so the differences are exact up to 1e-9)."""
    N, k, K, D = 3, 2, 4, 5
    g = torch.Generator().manual_seed(1)
    T, w, d = torch.randn(K, D, generator=g), torch.randn(N, k, generator=g), torch.randn(N, D, generator=g)
    ids = torch.tensor([[0, 2], [2, 2], [-1, 3]], dtype=torch.int32)
    dt, dw = km.kmassign_lookup_grad(d.to(dev), ids.to(dev), K, weights=w.to(dev), table=T.to(dev), scale=2.0)

    def loss(t, v):
        return (ref_lookup(t, ids.numpy(), v, 2.0)[0] * f64(d)).sum()
    h = 1e-3
    for arr, got in ((f64(T), f64(dt)), (f64(w), f64(dw))):
        for at in np.ndindex(arr.shape):
            up, down = arr.copy(), arr.copy()
            up[at] += h
            down[at] -= h
            diff = (loss(up, f64(w)) - loss(down, f64(w)) if arr.shape == (K, D)
                    else loss(f64(T), up) - loss(f64(T), down)) / (2 * h)
            assert abs(got[at] - diff) <= 1e-9 + 64 * U


def test_lookup_offsets_past_32_bits(dev):
    K, D = 70_000, 65_536                     # 4.6e9 elements
    T = torch.zeros(K, D, dtype=torch.bfloat16, device=dev)
    T[K - 1] = torch.arange(D, device=dev).remainder(200).to(torch.bfloat16)
    ids = torch.tensor([K - 1, 0, K - 1], dtype=torch.int32, device=dev)
    out = km.kmassign_lookup(T, ids, scale=2.0)
    assert torch.equal(out[0], T[K - 1] * 2) and torch.equal(out[2], out[0]) and (out[1] == 0).all()
    T.fill_(1.0)
    km.kmassign_lookup_grad(out, ids, K, dtable=T)
    assert torch.equal(T[K - 1], (out[0].float() * 2).to(torch.bfloat16))
    assert (T[K - 2] == 0).all() and (T[0] == 0).all() and (T[K // 2] == 0).all()


# ---- clipping -------------------------------------------------------------------

def make_grads(shapes, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(size * torch.randn(*s, generator=g)).to(TYPES[i % 3]) for i, s in enumerate(shapes)]


def check_clip(grads, outs, norm, max_norm):
    total = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    assert abs(norm.item() - total) <= 40 * U * total
    c = min(1.0, max_norm / (total + 1e-6))
    for g, o in zip(grads, outs):
        ref = f64(g) * c
        assert o.dtype == g.dtype
        assert np.all(np.abs(f64(o) - ref) <= (48 * U + OUT[g.dtype]) * np.abs(ref) + TINY[g.dtype])


CLIPS = [[(1,)], [(3, 5)], [(1000,), (64, 64), (7,), (0,), (129, 33)], [(70_000,), (16_385,), (32_768,)],
         [(5,)] * 300, [(17, 3)] * 257 + [(40_000,)], [(600_000,), (1_100_001,)]]


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("shapes", CLIPS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_clip(dev, shapes, max_norm):
    grads = make_grads(shapes, len(shapes))
    gd = [g.to(dev) for g in grads]
    outs = [torch.full_like(g, NAN) for g in gd]
    norm = km.kmassign_clip(gd, max_norm, out=outs)
    assert norm.shape == () and all(torch.equal(a.cpu(), b) for a, b in zip(gd, grads))
    check_clip(grads, outs, norm, max_norm)
    assert torch.equal(km.kmassign_grad_norm(gd), norm)
    again = km.kmassign_clip(gd, max_norm)     # in place
    assert torch.equal(again, norm)
    assert all(torch.equal(a, b) for a, b in zip(gd, outs))


def test_clip_misaligned_views(dev):
    buf = torch.randn(200_000, generator=torch.Generator().manual_seed(0))
    for dtype in TYPES:
        b = buf.to(dtype).to(dev)
        views = [b[1:50_000], b[50_003:50_004], b[60_001:200_000]]
        keep = b.clone()
        grads = [v.cpu().clone() for v in views]
        norm = km.kmassign_clip(views, 2.0)
        check_clip(grads, views, norm, 2.0)
        for lo, hi in ((0, 1), (50_000, 50_003), (50_004, 60_001)):
            assert torch.equal(b[lo:hi], keep[lo:hi])


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-15, 1e15, 1e22, 1e30])
@pytest.mark.parametrize("n", [10, 100_003])
def test_clip_norm_over_the_whole_range(dev, n, size):
    for dtype in (torch.float32, torch.bfloat16):
        g = (size * torch.randn(n, generator=torch.Generator().manual_seed(n))).to(dtype)
        want = np.sqrt((f64(g) ** 2).sum())
        assert abs(km.kmassign_grad_norm([g.to(dev)]).item() - want) <= 40 * U * want


def test_clip_special_values(dev):
    zero = torch.zeros(100_000, device=dev)
    assert km.kmassign_clip([zero], 1.0).item() == 0 and (zero == 0).all()
    g = torch.ones(70_000, device=dev)
    g[69_999] = INF
    assert km.kmassign_clip([g], 1.0).item() == INF
    assert torch.isnan(g[69_999]) and (g[:69_999] == 0).all()       # c = 0, by the formula
    h = torch.ones(70_000, device=dev)
    h[3] = NAN
    assert np.isnan(km.kmassign_clip([h], 1.0).item()) and torch.isnan(h).all()
    assert km.kmassign_clip([], 1.0).item() == 0
    assert km.kmassign_grad_norm([torch.empty(0, device=dev)]).item() == 0
    k = torch.full((9,), 2.0, device=dev)
    assert km.kmassign_clip([k], INF).item() == 6.0 and (k == 2).all()


# ---- streams, refusals, the whole path --------------------------------------------

def test_on_another_stream(dev):
    """Inputs made late on a side stream are seen by calls given that stream."""
    s = torch.cuda.Stream(dev)
    T = torch.zeros(4096, 256, device=dev)
    ids = torch.zeros(30_000, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        T.fill_(2.0)
        ids.fill_(5)
        out = torch.empty(30_000, 256, device=dev)
    km.kmassign_lookup(T, ids, out=out, stream=s)
    with torch.cuda.stream(s):
        dt, _ = km.kmassign_lookup_grad(out, ids, 4096)
        order, offsets = km.kmassign_lists(ids, 4096)
        norm = km.kmassign_clip([dt], 1.0)
        idx, w = km.kmassign_route(out, 3)
    s.synchronize()
    assert (out == 2).all() and offsets[5].item() == 0 and offsets[6].item() == 30_000
    assert torch.equal(order, torch.arange(30_000, dtype=torch.int32, device=dev))
    assert abs(norm.item() - 60_000 * 16) <= 40 * U * 960_000
    assert (idx == torch.arange(3, device=dev)).all() and abs(w.sum().item() - 30_000) < 1


def test_refuses_on_gpu(dev):
    x = torch.zeros(8, 16, device=dev)
    i = torch.zeros(8, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="contiguous"):
        km.kmassign_route(x.T, 2)
    with pytest.raises(TypeError):
        km.kmassign_route(x.double(), 2)
    with pytest.raises(ValueError, match="shape"):
        km.kmassign_route(x, 2, bias=torch.zeros(5, device=dev))
    with pytest.raises(km.KmassignError):
        km.kmassign_route(x, 17)
    with pytest.raises(ValueError, match="shape"):
        km.kmassign_route_grad(x, torch.zeros(7, 2, dtype=torch.int32, device=dev), x)
    with pytest.raises(TypeError):
        km.kmassign_lookup(x, i.long())
    with pytest.raises(ValueError, match="shape"):
        km.kmassign_lookup(x, i, weights=torch.zeros(3, device=dev))
    with pytest.raises(ValueError, match="shape"):
        km.kmassign_lookup(x, i, out=torch.zeros(8, 15, device=dev))
    with pytest.raises(ValueError, match="needs the table"):
        km.kmassign_lookup_grad(x, i, 4, weights=torch.zeros(8, device=dev))
    with pytest.raises(ValueError, match="accumulate"):
        km.kmassign_lookup_grad(x, i, 4, accumulate=True)
    with pytest.raises(km.KmassignError):
        km.kmassign_lookup_grad(x, i, 4, dtype=torch.float16)
    with pytest.raises(ValueError, match="one tensor per gradient"):
        km.kmassign_clip([x], 1.0, out=[])
    with pytest.raises(km.KmassignError):
        km.kmassign_clip([x], -1.0)
    host = torch.zeros(8, 16)
    rc = km.library().kmassign_lookup(host.data_ptr(), 0, 8, 16, i.data_ptr(), None, 8, 1, 1.0,
                                      x.data_ptr(), None)
    assert rc == km.STATUS["KMASSIGN_ERR_NOT_DEVICE"]


def test_soft_codes_example_learns(dev):
    spec = importlib.util.spec_from_file_location("soft_codes", os.path.join(ROOT, "examples", "soft_codes.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, used = m.train(steps=40)
    assert losses[-1] < 0.5 * losses[0]
    assert m.train(steps=3)[0] == losses[:3]   # the same bits again


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [31, 33, 47, 129, 2047])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_lookup_odd_rows_at_the_table_s_ends(dev, D, shift, dtype):
    """Odd rows are gathered word by word; the first and the last row's words end with the table,
    whose neighbours in memory hold NaN."""
    K = 5
    buf = torch.full((K * D + 16,), NAN, dtype=dtype)
    buf[shift: shift + K * D] = torch.randn(K * D, generator=torch.Generator().manual_seed(D)).to(dtype)
    bd = buf.to(dev)
    T = bd[shift: shift + K * D].view(K, D)
    ids = torch.tensor([0, K - 1, 2, 0, K - 1, -1, K], dtype=torch.int32, device=dev)
    w = torch.tensor([1.0, 2.0, 0.5, -1.0, 1.0, NAN, NAN], device=dev)
    out = km.kmassign_lookup(T, ids, weights=w)
    want = T[ids[:5].long()].float() * w[:5, None]
    assert torch.equal(out[:5], want.to(dtype)) and (out[5:] == 0).all()


def test_in_a_captured_graph(dev):
    """The calls, their temporaries included, run from a captured graph with new inputs."""
    N, E, k, D = 600, 64, 4, 48
    g = torch.Generator().manual_seed(0)
    X = torch.randn(N, E, generator=g).to(dev)
    T = torch.randn(E, D, generator=g).to(torch.bfloat16).to(dev)
    dY = torch.randn(N, D, generator=g).to(torch.bfloat16).to(dev)

    def step():
        idx, w = km.kmassign_route(X, k, score="sigmoid", groups=8, topk_groups=3)
        Y = km.kmassign_lookup(T, idx, weights=w)
        dT, dw = km.kmassign_lookup_grad(dY, idx, E, weights=w, table=T)
        dX = km.kmassign_route_grad(X, idx, dw, score="sigmoid")
        order, offsets = km.kmassign_lists(idx, E)
        norm = km.kmassign_clip([dT, dX], 1.0)
        return [idx, w, Y, dT, dw, dX, order, offsets, norm]
    side = torch.cuda.Stream(dev)
    with torch.cuda.stream(side):
        step()                               # first calls set the device up
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    for seed in (1, 2):
        X.copy_(torch.randn(N, E, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [3000, 100_000])
def test_lists_and_gradient_with_very_many_rows(dev, M):
    """30 million rows: three digits of a sort, most rows empty."""
    K = 30_000_000
    ids = np.random.default_rng(M).integers(0, K, M).astype(np.int32)
    check_lists(dev, ids, K)
    dout = torch.randint(-4, 5, (M, 1), generator=torch.Generator().manual_seed(1)).float()
    dt, _ = km.kmassign_lookup_grad(dout.to(dev), torch.from_numpy(ids).to(dev), K)
    want = np.zeros(K)
    np.add.at(want, ids, f64(dout)[:, 0])
    assert np.array_equal(f64(dt)[:, 0], want)


def test_clip_more_than_2_31_elements(dev):
    n = 2 ** 31 + 100_003
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=dev)
    g[-1] = 3.0
    norm = km.kmassign_clip([g], 100.0)
    want = np.sqrt(0.25 * (n - 1) + 9.0)
    assert abs(norm.item() - want) <= 40 * U * want
    c = 100.0 / want
    for i in (0, 2 ** 31 - 1, 2 ** 31, n - 2, n - 1):
        ref = (3.0 if i == n - 1 else 0.5) * c
        assert abs(g[i].item() - ref) <= (48 * U + 2.0 ** -8) * ref


def test_sigmoid_weights_are_the_quotient_s_bits(dev):
    """Weights of single experts over all magnitudes: 1 / (1 + exp(-x)), each step rounded once;
    and the same bits where the selection forms its keys (a zero bias orders by the scores)."""
    x = torch.cat([torch.linspace(-110, 110, 400_001), torch.randn(100_000) * 3]).to(dev)
    idx, w = km.kmassign_route(x[:, None].contiguous(), 1, score="sigmoid", renorm=False)
    t = torch.exp(-x)                      # CUDA's expf
    want = (1.0 / (1.0 + t).double()).float()
    assert torch.equal(w[:, 0], want)
    # rows of 8 neighbours: descending scores, ties to the lower index
    rows = x[: 400_000].view(-1, 8).contiguous()
    idx, w = km.kmassign_route(rows, 8, score="sigmoid", bias=torch.zeros(8, device=dev), renorm=False)
    s = want[: 400_000].view(-1, 8)
    value, order = s.sort(dim=1, descending=True, stable=True)
    assert torch.equal(idx.long(), order) and torch.equal(w, value)


@pytest.mark.parametrize("M", [2047, 2048, 2049, 4097, 5000, 8191, 12_288, 16_383, 16_384, 16_385])
@pytest.mark.parametrize("K", [1, 2, 700, 1024, 1025, 200_000, 3_000_000])
def test_lists_around_the_cluster_s_sizes(dev, M, K):
    """Up to 16,384 ids one cluster sorts; shares of its blocks that end early, ids left out."""
    g = np.random.default_rng(M * 7 + K)
    check_lists(dev, np.where(g.random(M) < 0.3, K // 2, g.integers(-1, K + 1, M)).astype(np.int32), K)
    check_lists(dev, np.where(g.random(M) < 0.999, -1, g.integers(0, K, M)).astype(np.int32), K)


@pytest.mark.parametrize("N,K,D", [(5000, 20_000, 33), (16_384, 9000, 130), (16_385, 9000, 130), (4097, 60_001, 7)])
def test_lookup_grad_zeroes_the_whole_table(dev, N, K, D):
    """The zeros that the sort writes besides reach every element, whatever the table's ends."""
    for kind in (torch.float32, torch.bfloat16):
        for shift in (0, 1, 3):
            buf = torch.full((K * D + 8,), 7.0, dtype=kind, device=dev)
            out = buf[shift: shift + K * D].view(K, D)
            ids = torch.full((N,), K // 3, dtype=torch.int32, device=dev)
            dout = torch.ones(N, D, dtype=torch.bfloat16, device=dev)
            km.kmassign_lookup_grad(dout, ids, K, dtable=out)
            want = float(torch.tensor(float(N)).to(kind))
            assert (out[K // 3] == want).all()
            assert (out[: K // 3] == 0).all() and (out[K // 3 + 1:] == 0).all()
            assert (buf[:shift] == 7).all() and (buf[shift + K * D:] == 7).all()
