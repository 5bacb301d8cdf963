"""Learned assignments on the GPU at the edges of what the entry points accept.

Tolerances and helpers are those of test_learn_gpu."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import means_nearest_centroid_gb300 as km
from means_nearest_centroid_gb300 import _build
from test_learn_gpu import (  # noqa: F401
    INF, NAN, TYPES, U, check_clip, dev, f64, make_grads, make_logits, ref_choice, ref_keys, ref_weights, weight_bound)

pytestmark = pytest.mark.gpu


# ---- routing --------------------------------------------------------------------

@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (96, 6), (30, 10), (8, 4)])
def test_route_groups_with_an_infinite_logit(dev, E, groups, top, renorm):  # noqa: F811
    """The group of a +inf logit comes first, wherever it lies, and the softmax weights of the row
    are NaN; a sigmoid's score there is 1, which two experts of another group can beat."""
    per = E // groups
    X = torch.randn(5, E, generator=torch.Generator().manual_seed(E)).to(dev)
    X[1, E - 1] = INF                       # the last group
    X[2, per], X[2, E - 2] = INF, INF       # two groups
    X[3] = -INF
    X[3, E - per] = INF                     # nothing but it
    idx, w = km.kmassign_route(X, 2, groups=groups, topk_groups=2, group_top=top, renorm=renorm)
    assert idx[1, 0].item() == E - 1 and idx[2].tolist() == [per, E - 2]
    assert idx[3].tolist() == [E - per, -1] and w[3, 1].item() == 0
    assert torch.isnan(w[1:3]).all() and torch.isnan(w[3, 0])
    rest = X[1].clone()                     # second: the best of the second group and the last one's others
    rest[E - 1] = -INF
    if top == 2:                            # all other groups' sums are 0: the lowest is the second
        rest[per: E - per] = -INF
    assert idx[1, 1].item() == rest.argmax().item()
    for i in (0, 4):
        one, _ = km.kmassign_route(X[i: i + 1], 2, groups=groups, topk_groups=2, group_top=top)
        assert torch.equal(one[0], idx[i]) and torch.isfinite(w[i]).all()
    Y = torch.full((1, E), -9.0, device=dev)
    Y[0, E - 1] = INF
    Y[0, :2] = 0.5
    idx, w = km.kmassign_route(Y, 1, score="sigmoid", groups=groups, topk_groups=1, group_top=top)
    assert idx.item() == (0 if top == 2 else E - 1) and w.item() == 1.0


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("k", [3, 12, 20])
def test_sigmoid_gradient_where_scores_underflow(dev, k, renorm):  # noqa: F811
    """A sigmoid below x = -88.7 is 0 in the weights (1 / (1 + inf)), and a row of such scores has
    weights 0: no gradient there, while the others' is what it is without that expert."""
    N, E = 6, 32
    gen = torch.Generator().manual_seed(k)
    X = torch.full((N, E), -200.0)
    X[:, :k] = torch.tensor([-90.0, -95.0, -100.0, -103.0, -120.0]).repeat(8)[torch.randperm(40, generator=gen)[:k]]
    X[1:, 1] = torch.randn(N - 1, generator=gen)
    X[2:, 2] = torch.randn(N - 2, generator=gen)
    dw = torch.randn(N, k, generator=gen)
    idx = torch.arange(k, dtype=torch.int32).repeat(N, 1)
    d = km.kmassign_route_grad(X.to(dev), idx.to(dev), dw.to(dev), score="sigmoid", renorm=renorm).cpu()
    s = 1 / (1 + torch.exp(-X.double()))
    assert (d[0] == 0).all() and (d[X < -89] == 0).all()
    if renorm:
        assert (d[1].abs() <= 64 * U).all()     # the only score: its weight is 1
        t = s[2:, 1] + s[2:, 2]
        want = s[2:, 1] * s[2:, 2] * (1 - s[2:, 1]) / t ** 2 * (dw[2:, 1] - dw[2:, 2])
        assert ((d[2:, 1] - want).abs() <= 64 * U * (want.abs() + 1)).all()
    else:
        want = (s * (1 - s))[2:, 1:3] * dw[2:, 1:3]
        assert ((d[2:, 1:3] - want).abs() <= 64 * U).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k", [(9, 2, 2), (33, 5, 4), (40, 30, 12), (21, 64, 32), (18, 100, 8), (17, 128, 20),
                                   (12, 200, 32), (7, 700, 9)])
def test_route_grad_of_repeated_experts(dev, N, E, k, score, renorm):  # noqa: F811
    """A row may name an expert twice: weights w_j = s_e(j) (/ sum_l s_e(l)) of each place, whose
    gradients add up; bounds as in test_route_grad, and k more roundings of the sum."""
    gen = torch.Generator().manual_seed(N)
    X = torch.randn(N, E, generator=gen)
    idx = torch.randint(-1, max(2, E // 3), (N, k), generator=gen).int()
    idx[0] = E - 1                                     # one expert everywhere
    dw = torch.randn(N, k, generator=gen)
    d = km.kmassign_route_grad(X.to(dev), idx.to(dev), dw.to(dev), score=score, renorm=renorm, scale=1.5)
    again = km.kmassign_route_grad(X.to(dev), idx.to(dev), dw.to(dev), score=score, renorm=renorm, scale=1.5)
    assert torch.equal(d, again)
    x = X.double().requires_grad_()
    live = (idx >= 0).double()
    # a renormalised softmax: the denominator over all experts cancels
    s = torch.sigmoid(x) if score == "sigmoid" else torch.exp(x) if renorm else torch.softmax(x, 1)
    w = s.gather(1, idx.clamp(min=0).long()) * live
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    (1.5 * w * dw.double()).sum().backward()
    # magnitudes: of each place's own term and of what the others' share takes from it
    amean = (w.detach() * dw.double().abs()).sum(1, keepdim=True)
    size = torch.zeros(N, E, dtype=torch.float64).scatter_add_(
        1, idx.clamp(min=0).long(), 1.5 * w.detach() * (dw.double().abs() + amean))
    if score == "softmax" and not renorm:
        size += 1.5 * s.detach() * amean
    bound = (2 * weight_bound(x.detach().numpy(), k) + (k + 1) * U) * size.numpy() + 2 ** -120
    assert ((d.cpu().double() - x.grad).abs().numpy() <= bound).all()


def selected_weight_bound(x, idx, scored):
    """Relative bound of a row's weights, from its own selected logits: expf (2 ulp), the rounding
    of x - max (relative |x - max| U), sums of E and of k terms, a division and two products."""
    E, k = x.shape[1], idx.shape[1]
    at = np.take_along_axis(x, np.maximum(idx, 0), 1)
    top = np.max(np.where(np.isnan(x), -INF, x), 1, keepdims=True)
    with np.errstate(invalid="ignore"):
        away = np.where(idx >= 0, np.minimum(np.abs(at - top), 104.0), 0.0)
    if scored == "sigmoid":
        away = np.zeros_like(away)            # exp(-x) takes x as it is
    return (2 * away + E / 8 + k + 12) * 2 * U


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k,groups,topk", [(400, 256, 8, 8, 4), (300, 72, 6, 6, 3), (300, 16, 2, 4, 2),
                                               (128, 512, 16, 16, 7), (40, 1024, 8, 16, 5), (200, 256, 8, 1, 1)])
def test_route_with_bias_row_by_row(dev, N, E, k, groups, topk, score, top):  # noqa: F811
    """The whole choice with a bias and groups: a row may differ from the 64-bit one only where its
    own deciding group sums, or its own deciding keys, are closer than their fp32 error; in no row
    is an expert named twice, out of range, masked or outside topk groups.  Keys: a score of at
    most 1 and a bias below 1.1, each rounding at most 2 U of 2; a softmax's scores relatively
    (2 |x - max| + E / 8 + 12) U of at most exp(x - max), so at most (2 / e + E / 8 + 12) U."""
    gen = torch.Generator().manual_seed(E + k)
    X = make_logits(N, E, torch.float32, N + 1)
    bias = 0.2 * torch.randn(E, generator=gen)
    bias.clamp_(-1.0, 1.0)
    x, b = f64(X), f64(bias)
    key, s = ref_keys(x, score, b, 1, 1, top)             # all groups' keys
    per = E // groups
    m = -np.sort(-key.reshape(N, groups, per), 2)[:, :, :top]
    of_group = np.where(m[:, :, 0] == -INF, -INF, np.where(m == -INF, 0.0, m).sum(2))
    tol = 2 * (2 / np.e + E / 8 + 12 + 4) * U             # of two keys' difference
    idx, w = km.kmassign_route(X.to(dev), k, score=score, bias=bias.to(dev), groups=groups,
                               topk_groups=topk, group_top=top, renorm=False)
    got = idx.cpu().numpy()
    differ = 0
    for i in range(N):
        mine = got[i][got[i] >= 0]
        assert len(set(mine.tolist())) == len(mine) and (mine < E).all() and (key[i, mine] > -INF).all()
        assert (got[i][len(mine):] == -1).all()           # free slots come last
        chosen = set((mine // per).tolist())
        assert len(chosen) <= topk
        order = np.argsort(-of_group[i], kind="stable")
        kept = set(order[:topk].tolist())
        if groups > topk:
            last, next_ = of_group[i, order[topk - 1]], of_group[i, order[topk]]
            if next_ > -INF and last - next_ <= 2 * tol:  # a near-tie of groups: either side is right
                edge = {g for g in range(groups) if abs(of_group[i, g] - last) <= 4 * tol}
                assert chosen <= kept | edge
                differ += 1
                continue
        allowed = np.where(np.isin(np.arange(E) // per, list(kept)), key[i], -INF)
        want = ref_choice(allowed[None], k)[0]
        assert np.array_equal(got[i] < 0, want < 0)
        on = want >= 0
        assert (np.abs(key[i, got[i][on]] - key[i, want[on]]) <= tol).all() and (allowed[mine] > -INF).all()
    assert differ <= N // 20
    ref = ref_weights(x, s, got, score, False, 1.0)
    assert (np.abs(f64(w) - ref) <= selected_weight_bound(x, got, score) * ref + 2 ** -125).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k", [(64, 8, 8), (40, 64, 6), (30, 200, 16), (65, 256, 8), (8, 1024, 32)])
def test_route_weights_by_their_own_logits(dev, N, E, k, score, renorm, dtype):  # noqa: F811
    """Weights to the bound of the logits that were selected, not of the lowest in the matrix."""
    X = make_logits(N, E, dtype, seed=E)
    x = f64(X)
    idx, w = km.kmassign_route(X.to(dev), k, score=score, renorm=renorm, scale=2.5)
    got = idx.cpu().numpy()
    key, s = ref_keys(x, score, None, 1, 1, 2)
    assert np.array_equal(got, ref_choice(key, k))
    ref = ref_weights(x, s, got, score, renorm, 2.5)
    assert (np.abs(f64(w) - ref) <= selected_weight_bound(x, got, score) * ref + 2 ** -125).all()


def test_route_softmax_with_bias_and_an_infinite_logit(dev):  # noqa: F811
    """Every score of the row is NaN, so every key is, and none is selected."""
    X = torch.zeros(3, 12, device=dev)
    X[1, 4] = INF
    idx, w = km.kmassign_route(X, 2, bias=torch.zeros(12, device=dev))
    assert idx.tolist() == [[0, 1], [-1, -1], [0, 1]] and w[1].tolist() == [0.0, 0.0]


def test_reciprocal_has_the_quotient_s_bits(dev, tmp_path):  # noqa: F811
    """Routing's reciprocal against the division, for every significand and exponents of its range."""
    lib = str(tmp_path / "libreciprocal_check.so")
    source = os.path.join(os.path.dirname(os.path.abspath(__file__)), "reciprocal_check.cu")
    subprocess.run([_build.nvcc(), *_build.NVCC_FLAGS, "-shared", "-I", _build.CSRC, source, "-o", lib], check=True)
    check = ctypes.CDLL(lib).reciprocal_check
    check.argtypes, check.restype = [ctypes.c_int, ctypes.c_void_p], ctypes.c_int
    count = torch.zeros(1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    for e in [*range(0, 125, 31), 1, 2, 123]:
        assert check(e, count.data_ptr()) == 0
        torch.cuda.synchronize()
        assert count.item() == 0, e


@pytest.mark.parametrize("E", [8, 16, 64, 100])
def test_choice_does_not_depend_on_the_batch(dev, E):  # noqa: F811
    """Sigmoids near 1 take few values, so a last bit decides an order; a logit below -87 in a
    warp has all its scores formed by divisions.  The same choice with and without it."""
    N, k = 64, min(E, 32)
    gen = torch.Generator().manual_seed(E)
    X = 8 + 9 * torch.rand(N, E, generator=gen)
    X[::3] = 4 * torch.randn(X[::3].shape, generator=gen)
    bias = torch.zeros(E, device=dev)

    def choice(x):
        return km.kmassign_route(x.to(dev), k, score="sigmoid", bias=bias)
    idx, w = choice(X)
    low = X.clone()
    low[1::2, 0] = -100.0                     # every second row: one at least in each warp
    got, v = choice(low)
    assert torch.equal(got[::2], idx[::2]) and torch.equal(v[::2], w[::2])
    for i in (0, 2, 6, N - 2):
        one, u = choice(X[i: i + 1])
        assert torch.equal(one[0], idx[i]) and torch.equal(u[0], w[i])
    # by the fp32 quotients themselves, with and without such a logit in the row
    for x, chosen in ((X, idx), (low, got)):
        s = (1.0 / (1.0 + torch.exp(-x.to(dev))).double()).float()
        assert torch.equal(chosen.long(), s.sort(dim=1, descending=True, stable=True).indices[:, :k])


# ---- clipping -------------------------------------------------------------------

@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("full,empty", [(256, 1), (256, 300), (512, 3), (24, 1), (25, 400), (257, 255)])
def test_clip_with_empty_tensors_at_the_end(dev, full, empty, max_norm):  # noqa: F811
    """A launch takes up to 256 tensors; what follows the last one that has elements takes none."""
    for shapes in ([(5,)] * full + [(0,)] * empty, [(0,)] * empty + [(5,)] * full,
                   [(5,)] * (full // 2) + [(0,)] * empty + [(5,)] * (full - full // 2) + [(0,)]):
        grads = make_grads(shapes, full)
        gd = [g.to(dev) for g in grads]
        outs = [torch.full_like(g, NAN) for g in gd]
        norm = km.kmassign_clip(gd, max_norm, out=outs)
        check_clip(grads, outs, norm, max_norm)
        assert torch.equal(km.kmassign_grad_norm(gd), norm)
        assert torch.equal(km.kmassign_clip(gd, max_norm), norm)     # in place
        assert all(torch.equal(a, b) for a, b in zip(gd, outs))


def clip_time(grads):
    """GPU time of one clipping in place, in ms: the launches wait in the stream until the host
    has made them all."""
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    torch.cuda._sleep(600_000_000)
    start.record()
    km.kmassign_clip(grads, 1.0)
    end.record()
    assert not start.query()              # the GPU has not begun: the span holds no host time
    torch.cuda.synchronize()
    return start.elapsed_time(end)


def test_clip_of_many_tensors_takes_time_in_proportion(dev):  # noqa: F811
    """8 times the tensors take 8 times as long (twice that is allowed), not 64 times: the norm's
    partial sums are added once, not by every block of every launch."""
    flat = torch.randn(32_768 * 5, generator=torch.Generator().manual_seed(0)).to(dev)
    grads = list(flat.split(5))
    keep = flat.clone()
    assert abs(km.kmassign_grad_norm(grads).item() - km.kmassign_grad_norm([flat]).item()) < 1e-3
    few, many = (min(clip_time(g) for _ in range(3)) for g in (grads[:4096], grads))
    assert many < 16 * few, (few, many)
    flat.copy_(keep)
    norm = km.kmassign_clip(grads, 1.0)
    check_clip([keep.cpu()], [flat.cpu()], norm, 1.0)


# ---- streams ----------------------------------------------------------------------

def calls_with_large_outputs(dev):  # noqa: F811
    """Calls whose outputs have 32 MiB each, by name."""
    N, D, k = 1 << 14, 512, 8
    rows = torch.zeros(N, D, device=dev)
    ids = torch.zeros(N, dtype=torch.int32, device=dev)
    logits = torch.zeros(1 << 20, k, device=dev)
    many = torch.zeros(1 << 20, k, dtype=torch.int32, device=dev)
    dw = torch.zeros(1 << 20, k, device=dev)
    X = torch.zeros(1 << 20, 16, dtype=torch.bfloat16, device=dev)
    return {
        "route": lambda s: km.kmassign_route(logits, k, stream=s),
        "route_grad": lambda s: [km.kmassign_route_grad(logits, many, dw, stream=s)],
        "lists": lambda s: [km.kmassign_lists(many, 4, stream=s)[0]],
        "lookup": lambda s: [km.kmassign_lookup(rows, ids, stream=s)],
        "lookup_grad": lambda s: [km.kmassign_lookup_grad(rows, ids, N, stream=s)[0]],
        "topk": lambda s: km.kmassign_topk(X, X[:64], k, stream=s),
        "update": lambda s: [km.kmassign_update(X, ids.new_zeros(1 << 20), 1 << 19, stream=s)[0]],
    }


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["route", "route_grad", "lists", "lookup", "lookup_grad", "topk", "update"])
def test_outputs_of_a_call_on_another_stream_are_its_own(dev, name, handle):  # noqa: F811
    """Memory freed on the current stream, behind work that still reads it, is not what a call on
    another stream writes its outputs to."""
    call = calls_with_large_outputs(dev)[name]
    s = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    call(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full((1 << 23,), 7.0, device=dev) for _ in range(4)]
    places = {t.data_ptr() for t in old}
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    kept = [t.clone() for t in old]           # still to come when the call below is made
    del old
    outs = call(s.cuda_stream if handle else s)
    s.synchronize()
    assert all(t.numel() * t.element_size() == 1 << 25 for t in outs)
    assert not places & {t.data_ptr() for t in outs}
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in kept)


def test_update_on_another_stream_starts_from_its_zeros(dev):  # noqa: F811
    """The sums' zeros belong to the call's stream, not to the current one's queue."""
    s = torch.cuda.Stream(dev)
    X = torch.ones(3000, 64, dtype=torch.bfloat16, device=dev)
    idx = torch.zeros(3000, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    sums, counts = km.kmassign_update(X, idx, 5, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        got, n = sums.cpu(), counts.cpu()
    torch.cuda.synchronize()
    for t in (got, sums.cpu()):
        assert (t[0] == 3000).all() and (t[1:] == 0).all()
    assert n.tolist() == counts.tolist() == [3000, 0, 0, 0, 0]


def test_default_stream_by_handle(dev):  # noqa: F811
    X = torch.randn(100, 16, generator=torch.Generator().manual_seed(0)).to(dev)
    idx, w = km.kmassign_route(X, 3, stream=0)
    other, v = km.kmassign_route(X, 3)
    assert torch.equal(idx, other) and torch.equal(w, v)


# ---- autograd -----------------------------------------------------------------------

def test_inputs_that_require_grad_are_refused_in_grad_mode(dev):  # noqa: F811
    """No result is silently cut off from the graph: such inputs raise, but under no_grad and in
    the forward and backward of an autograd function."""
    x = torch.randn(8, 16, device=dev)
    p = x.clone().requires_grad_()
    i = torch.zeros(8, 2, dtype=torch.int32, device=dev)
    w = torch.ones(8, 2, device=dev)
    wp = w.clone().requires_grad_()
    calls = [lambda: km.kmassign_route(p, 2), lambda: km.kmassign_route(p * 2, 2),
             lambda: km.kmassign_route_grad(p, i, w), lambda: km.kmassign_route_grad(x, i, wp),
             lambda: km.kmassign_lookup(p, i), lambda: km.kmassign_lookup(x, i, weights=wp),
             lambda: km.kmassign_lookup_grad(p, i, 8),
             lambda: km.kmassign_lookup_grad(x, i, 8, weights=wp, table=x),
             lambda: km.kmassign_lookup_grad(x, i, 8, weights=w, table=p),
             lambda: km.kmassign_grad_norm([x, p]), lambda: km.kmassign_clip([x, p], 1.0),
             lambda: km.kmassign_clip([x], 1.0, out=[p])]
    before = p.detach().clone()
    with pytest.raises(TypeError):           # what is no tensor is told as before
        km.kmassign_lookup_grad(x, i, 8, weights=[1.0], table=x)
    with pytest.raises(TypeError):
        km.kmassign_lookup_grad(x, i, 8, weights=w, table=[1.0])
    for call in calls:
        with pytest.raises(RuntimeError, match="requires grad"):
            call()
    assert torch.equal(p, before)
    with torch.no_grad():
        for call in calls:
            call()
    km.kmassign_route(x, 2, score="sigmoid", bias=torch.zeros(16, device=dev, requires_grad=True))


def test_as_an_autograd_function(dev):  # noqa: F811
    """The lookup and its gradient inside a torch.autograd.Function, against torch's own."""
    class Lookup(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, idx, weights):
            ctx.save_for_backward(table, idx, weights)
            return km.kmassign_lookup(table, idx, weights=weights)

        @staticmethod
        def backward(ctx, dout):
            table, idx, weights = ctx.saved_tensors
            dtable, dw = km.kmassign_lookup_grad(dout, idx, table.shape[0], weights=weights, table=table)
            return dtable, None, dw

    gen = torch.Generator().manual_seed(0)
    table = torch.randn(10, 6, generator=gen).to(dev).requires_grad_()
    weights = torch.randn(30, 3, generator=gen).to(dev).requires_grad_()
    idx = torch.randint(0, 10, (30, 3), generator=gen).int().to(dev)
    c = torch.randn(30, 6, generator=gen).to(dev)
    (Lookup.apply(table, idx, weights) * c).sum().backward()
    t, v = table.detach().double().requires_grad_(), weights.detach().double().requires_grad_()
    ((t[idx.long()] * v[..., None]).sum(1) * c.double()).sum().backward()
    # at most 90 terms an element of magnitude below 20
    assert (table.grad - t.grad).abs().max() <= 100 * U * 90 * 20
    assert (weights.grad - v.grad).abs().max() <= 10 * U * 6 * 20


def test_writes_to_given_tensors_are_seen_by_autograd(dev):  # noqa: F811
    """Every tensor of the caller that a call writes to counts a version, so that a backward pass
    that has saved it raises; the inputs' versions stay."""
    x, big = torch.randn(8, 16, device=dev), torch.randn(8, 16, device=dev)
    i = torch.zeros(8, 2, dtype=torch.int32, device=dev)
    w = torch.ones(8, 2, device=dev)

    def f(*shape):
        return torch.zeros(shape, device=dev)

    def z(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=dev)
    cases = [
        (lambda o: km.kmassign_route(x, 2, idx=o[0], weights=o[1]), [z(8, 2), f(8, 2)]),
        (lambda o: km.kmassign_route(x, 2, weights=o[0]), [f(8, 2)]),
        (lambda o: km.kmassign_route_grad(x, i, w, dlogits=o[0]), [f(8, 16)]),
        (lambda o: km.kmassign_lists(i, 4, order=o[0], offsets=o[1]), [z(16), z(5)]),
        (lambda o: km.kmassign_lookup(x, i, out=o[0]), [f(8, 16)]),
        (lambda o: km.kmassign_lookup_grad(x, i, 8, weights=w, table=big, dtable=o[0], dweights=o[1]),
         [f(8, 16), f(8, 2)]),
        (lambda o: km.kmassign_lookup_grad(x, i, 8, dtable=o[0], accumulate=True), [f(8, 16)]),
        (lambda o: km.kmassign_grad_norm([x], norm=o[0]), [f()]),
        (lambda o: km.kmassign_clip([o[0], o[1]], 1.0, norm=o[2]), [big.clone(), f(3), f()]),
        (lambda o: km.kmassign_clip([x], 1.0, out=[o[0]]), [f(8, 16)]),
    ]
    for call, outs in cases:
        versions = [o._version for o in outs]
        call(outs)
        assert all(o._version > v for o, v in zip(outs, versions))
    assert x._version == i._version == w._version == 0
    p = torch.randn(8, 16, device=dev, requires_grad=True)
    y = (p * big).sum()
    km.kmassign_clip([big], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        inner = torch.ones(8, 16, device=dev)
        km.kmassign_clip([inner], 1.0)
    km.kmassign_clip([inner], 1.0)


def test_clip_tells_which_tensor_it_cannot_take(dev):  # noqa: F811
    x = torch.randn(8, 16, device=dev)
    for bad, error, text in ((torch.zeros(3), ValueError, "CUDA"), (x.T, ValueError, "contiguous"),
                             (x.double(), TypeError, "float32"), ([1.0], TypeError, "Tensor")):
        keep = x.clone()
        for grads in ([x, bad], [bad, x], [x, x[:2], bad]):
            with pytest.raises(error, match=text):
                km.kmassign_clip(grads, 1e-3)
            with pytest.raises(error, match=text):
                km.kmassign_grad_norm(grads)
            with pytest.raises((error, ValueError), match=f"{text}|sizes|one tensor"):
                km.kmassign_clip([x] * len(grads), 1e-3, out=grads)
        assert torch.equal(x, keep)
