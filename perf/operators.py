"""The operators around a learned assignment, as they are measured: routing points to table rows, looking
the rows up, the gradients of both, the inverted lists of an assignment and the clipping of gradients.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true, with the
library's entry points.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # A decoding step's routing: sixteen points, sigmoid scores with a balance bias, 4 of 8 groups.
        {"name": "route_decode", "op": "route", "N": 16, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # The same router over a long batch.
        {"name": "route_batch", "op": "route", "N": 65536, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # Training that router: the weights' gradient back to the logits of the selected rows.
        {"name": "route_grad_batch", "op": "route_grad", "N": 65536, "E": 256, "k": 8, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # A softmax over all experts without renormalisation, half-precision logits, ragged sizes.
        {"name": "route_grad_softmax", "op": "route_grad", "N": 30011, "E": 72, "k": 6, "score": "softmax",
         "renorm": False, "scale": 1.0, "dtype": "bf16"},
        # A generation step's embedding lookup.
        {"name": "lookup_decode", "op": "lookup", "N": 8, "k": 1, "K": 131072, "D": 2048, "weighted": False,
         "scale": 45.25, "dtype": "bf16", "skew": 4.0},
        # Soft codes: each point is the weighted sum of its 8 nearest of 16,384 codes.
        {"name": "lookup_mixture", "op": "lookup", "N": 65536, "k": 8, "K": 16384, "D": 256, "weighted": True,
         "scale": 1.0, "dtype": "bf16", "skew": 1.0},
        # The gradient of an embedding table over a training batch of tokens with a few frequent ones.
        {"name": "lookup_grad_tokens", "op": "lookup_grad", "N": 16384, "k": 1, "K": 131072, "D": 2048,
         "weighted": False, "scale": 45.25, "dtype": "bf16", "grad": "fp32", "skew": 4.0},
        # The gradients of the soft codes: of the table and of the weights; odd sizes.
        {"name": "lookup_grad_mixture", "op": "lookup_grad", "N": 30011, "k": 8, "K": 16384, "D": 250,
         "weighted": True, "scale": 1.0, "dtype": "bf16", "grad": "bf16", "skew": 1.5},
        # The token lists of the experts in a decoding step.
        {"name": "lists_decode", "op": "lists", "M": 512, "K": 256, "skew": 1.0},
        # The inverted lists of a million points over 4,096 centroids, with some ids to leave out.
        {"name": "lists_points", "op": "lists", "M": 1048576, "K": 4096, "skew": 1.5},
        # A small model's half-precision gradients, inside the bound about as often as not.
        {"name": "clip_small", "op": "clip", "layers": 2, "width": 250, "dtype": "bf16", "max_norm": 1.0},
        # The fp32 gradients of a quarter of a billion parameters.
        {"name": "clip_large", "op": "clip", "layers": 10, "width": 2048, "dtype": "fp32", "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "lookup", "lookup_grad", "lists", "clip"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    if op in ("route", "route_grad"):
        E = _log(rng, 8, 512)
        k = rng.randint(1, min(E, 16))
        case = {"op": op, "N": _log(rng, 1, 65536 if E <= 256 else 32768), "E": E, "k": k, "score": rng.choice(["sigmoid", "softmax"]),
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "dtype": dtype}
        if op == "route":
            groups = rng.choice([g for g in range(1, 17) if E % g == 0 and E // g >= 2])
            need = -(-k // (E // groups))
            case.update(bias=case["score"] == "sigmoid" and rng.random() < 0.6, groups=groups,
                        topk_groups=rng.randint(need, groups), group_top=rng.choice([1, 2]))
        return case
    if op in ("lookup", "lookup_grad"):
        k = rng.choice([1, 1, 1, 2, 4, 7, 8])
        D = _log(rng, 16, 4096)
        K = _log(rng, 16, min(131072, (1 << 28) // D))
        N = _log(rng, 1, min(65536, (1 << 27) // (D * k)))
        case = {"op": op, "N": N, "k": k, "K": K, "D": D, "weighted": k > 1 or rng.random() < 0.2,
                "scale": rng.choice([1.0, 0.5, round(math.sqrt(D), 2)]), "dtype": dtype, "skew": rng.choice([1.0, 1.5, 4.0])}
        if op == "lookup_grad":
            case["grad"] = rng.choice(["fp32", dtype])
        return case
    if op == "lists":
        return {"op": op, "M": _log(rng, 1, 1 << 21), "K": _log(rng, 2, 1 << 20), "skew": rng.choice([1.0, 1.5, 4.0])}
    return {"op": op, "layers": rng.randint(1, 10), "width": _log(rng, 32, 2048), "dtype": dtype,
            "max_norm": rng.choice([0.1, 1.0, 1e4])}


def _shapes(case):
    """A model's parameters: for each layer two square matrices, a wide one and two vectors."""
    W = case["width"]
    return [(W, W), (W, W), (W, 5 * W), (W,), (5 * W,)] * case["layers"]


def _distinct(K, skew, M):
    """How many of K rows M draws of floor(K u^skew) are expected to name."""
    edge = (np.arange(K + 1, dtype=np.float64) / K) ** (1.0 / skew)
    return float(np.sum(-np.expm1(M * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12)))))


def work(case):
    op = case["op"]
    if op == "route":
        N, E, k = case["N"], case["E"], case["k"]
        return {"bytes": N * E * BYTES[case["dtype"]] + 4 * E * case["bias"] + 8 * N * k, "flops": 10 * N * E}
    if op == "route_grad":
        N, E, k, b = case["N"], case["E"], case["k"], BYTES[case["dtype"]]
        logits = N * k if case["score"] == "sigmoid" or case["renorm"] else N * E
        return {"bytes": logits * b + 8 * N * k + N * E * b, "flops": 4 * N * E}
    if op == "lists":
        return {"bytes": 8 * case["M"] + 4 * (case["K"] + 1), "flops": 0}
    if op == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        return {"bytes": 2 * n * BYTES[case["dtype"]], "flops": 3 * n}
    N, k, K, D, b = case["N"], case["k"], case["K"], case["D"], BYTES[case["dtype"]]
    rows = _distinct(K, case["skew"], N * k)
    ids = N * k * (8 if case["weighted"] else 4)
    if op == "lookup":
        return {"bytes": int(rows * D * b) + N * D * b + ids, "flops": 2 * N * k * D}
    more = (int(rows * D * b) + 4 * N * k) if case["weighted"] else 0
    return {"bytes": N * D * b + K * D * BYTES[case["grad"]] + ids + more, "flops": (4 if case["weighted"] else 2) * N * k * D}


# --------------------------------------------------------------------------------------------- inputs

def _ids(K, skew, shape, gen, left_out):
    """Row ids, low ones more frequent where skew > 1; a share `left_out` of them is -1 or K (no row)."""
    u = torch.rand(shape, generator=gen, device=DEVICE, dtype=torch.float64)
    ids = (u.pow_(skew) * K).to(torch.int64).clamp_(0, K - 1)
    if left_out:
        v = torch.rand(shape, generator=gen, device=DEVICE)
        ids = torch.where(v < left_out, torch.where(v < left_out / 2, -1, K), ids)
    return ids.to(torch.int32)


def _distinct_ids(N, E, k, gen):
    """k different experts a row, as a router gives them; one row in fifty has a free slot."""
    idx = torch.rand(N, E, generator=gen, device=DEVICE).argsort(-1)[:, :k].to(torch.int32)
    if k > 1:
        free = torch.rand(N, generator=gen, device=DEVICE) < 0.02
        idx[:, -1] = torch.where(free, -1, idx[:, -1])
    return idx.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    state = {"case": dict(case)}
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEVICE)  # noqa: E731
    op = case["op"]
    if op in ("route", "route_grad"):
        N, E = case["N"], case["E"]
        # Logits of a few units, one expert in two hundred masked away.
        x = 1.5 * normal(N, E)
        x.masked_fill_(torch.rand(N, E, generator=gen, device=DEVICE) < 0.005, -math.inf)
        state["logits"] = x.to(TYPES[case["dtype"]])
        if op == "route":
            # A balance bias is the sum of many small equal steps.
            step = torch.randint(-100, 101, (E,), generator=gen, device=DEVICE)
            state["bias"] = step.float() / 1024 if case["bias"] else None
        else:
            state["idx"] = _distinct_ids(N, E, case["k"], gen)
            state["dweights"] = normal(N, case["k"])
        return state
    if op == "lists":
        state["idx"] = _ids(case["K"], case["skew"], (case["M"],), gen, 0.02)
        return state
    if op == "clip":
        kind = TYPES[case["dtype"]]
        size = 10.0 ** float(torch.empty(1, device="cpu").uniform_(-4.5, -1.5, generator=torch.Generator().manual_seed(int(seed))))
        state["grads"] = [(size * normal(*s)).to(kind) for s in _shapes(case)]
        state["out"] = [torch.empty_like(g) for g in state["grads"]]
        return state
    N, k, K, D = case["N"], case["k"], case["K"], case["D"]
    kind = TYPES[case["dtype"]]
    shape = (N, k) if k > 1 else (N,)
    state["idx"] = _ids(K, case["skew"], shape, gen, 0.01)
    state["weights"] = torch.rand(shape, generator=gen, device=DEVICE) if case["weighted"] else None
    if op == "lookup" or case["weighted"]:
        state["table"] = (0.02 * normal(K, D)).to(kind)
    if op == "lookup_grad":
        state["dout"] = normal(N, D).to(kind)
    return state


# ---------------------------------------------------------------------------------------- plain forms

def _plain_route(case, logits, bias):
    k, groups = case["k"], case["groups"]
    x = logits.float()
    masked = torch.isnan(x) | (x == -math.inf)
    low = torch.full_like(x, -math.inf)
    if case["score"] == "softmax":
        part = torch.where(masked, 0.0, torch.exp(x - torch.where(masked, low, x).amax(-1, keepdim=True)))
        score = part / part.sum(-1, keepdim=True)
    else:
        part = score = torch.where(masked, 0.0, 1.0 / (1.0 + torch.exp(-x)))
    key = x if bias is None else score + bias
    key = torch.where(masked | torch.isnan(key), low, key)
    if groups > 1:
        N, E = x.shape
        top = case["group_top"]
        member = key if bias is not None or top == 1 else torch.where(masked, low, part)
        best = member.view(N, groups, E // groups).sort(dim=-1, descending=True).values[..., :top]
        of_group = torch.where(best == -math.inf, 0.0, best).sum(-1)
        of_group = torch.where(best[..., 0] == -math.inf, -math.inf, of_group)
        stay = of_group.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        kept = torch.zeros(N, groups, dtype=torch.bool, device=x.device).scatter_(1, stay, True)
        key = torch.where(kept.repeat_interleave(E // groups, 1), key, low)
    value, idx = key.sort(dim=-1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    free = value == -math.inf
    if not case["renorm"]:
        w = score.gather(1, idx)
    elif case["score"] == "softmax":
        chosen = torch.where(free, -math.inf, x.gather(1, idx))
        w = torch.where(free, 0.0, torch.exp(chosen - chosen.amax(-1, keepdim=True)))
        w = w / w.sum(-1, keepdim=True)
    else:
        w = torch.where(free, 0.0, score.gather(1, idx))
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(free, -1, idx).to(torch.int32), torch.where(free, 0.0, w * case["scale"])


def _plain_route_grad(case, logits, idx, dweights):
    x = logits.float()
    masked = torch.isnan(x) | (x == -math.inf)
    free = (idx < 0) | (idx >= x.shape[1])
    at = torch.where(free, 0, idx).long()
    g = torch.where(free, 0.0, dweights) * case["scale"]
    chosen = x.gather(1, at)
    out = torch.zeros_like(x)
    if case["score"] == "sigmoid":
        s = torch.where(free | masked.gather(1, at), 0.0, 1.0 / (1.0 + torch.exp(-chosen)))
        if case["renorm"]:
            total = s.sum(-1, keepdim=True)
            d = torch.where(total > 0, s * (1.0 - s) / total * (g - (s * g).sum(-1, keepdim=True) / total), 0.0)
        else:
            d = s * (1.0 - s) * g
    elif case["renorm"]:
        gone = free | masked.gather(1, at)
        chosen = torch.where(gone, -math.inf, chosen)
        p = torch.where(gone, 0.0, torch.exp(chosen - chosen.amax(-1, keepdim=True)))
        p = p / p.sum(-1, keepdim=True)
        d = torch.where(gone, 0.0, p * (g - (p * g).sum(-1, keepdim=True)))
    else:
        p = torch.where(masked, 0.0, torch.exp(x - torch.where(masked, -math.inf, x).amax(-1, keepdim=True)))
        p = torch.where(masked, 0.0, p / p.sum(-1, keepdim=True))
        full = out.scatter_add(1, at, g)
        return (p * (full - (p * full).sum(-1, keepdim=True))).to(logits.dtype)
    return out.scatter_add_(1, at, torch.where(free, 0.0, d)).to(logits.dtype)


def _plain_rows(table, idx, weights):
    """fp32 rows [N, k, D] that the ids name (zero where none), and the weights [N, k] in their places."""
    idx = idx.view(idx.shape[0], -1)
    there = (idx >= 0) & (idx < table.shape[0])
    w = there.float() if weights is None else torch.where(there, weights.view(idx.shape), 0.0)
    return table[torch.where(there, idx, 0).long()].float(), w, there


def _plain_lookup(case, table, idx, weights):
    rows, w, _ = _plain_rows(table, idx, weights)
    return ((rows * w.unsqueeze(-1)).sum(1) * case["scale"]).to(table.dtype)


def _plain_lookup_grad(case, dout, idx, weights, table):
    K = case["K"]
    two = idx.view(idx.shape[0], -1)
    there = (two >= 0) & (two < K)
    d = dout.float().unsqueeze(1)
    w = there.float() if weights is None else torch.where(there, weights.view(two.shape), 0.0)
    each = (d * w.unsqueeze(-1) * case["scale"]).view(-1, d.shape[-1])
    dtable = torch.zeros(K + 1, d.shape[-1], device=d.device).index_add_(0, torch.where(there, two, K).long().view(-1), each)
    dtable = dtable[:K].to(TYPES[case["grad"]])
    if weights is None:
        return dtable, None
    rows, _, _ = _plain_rows(table, idx, weights)
    return dtable, torch.where(there, (rows * d).sum(-1) * case["scale"], 0.0).view(idx.shape)


def _plain_lists(idx, K):
    there = (idx >= 0) & (idx < K)
    row, order = torch.where(there, idx, K).sort(stable=True)
    offsets = torch.zeros(K + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.bincount(row, minlength=K + 1)[:K].cumsum(0)
    return torch.where(row < K, order, -1).to(torch.int32), offsets.to(torch.int32)


def _plain_clip(grads, max_norm):
    norm = torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()
    c = (max_norm / (norm + 1e-6)).clamp(max=1.0)
    return norm, [(g.float() * c).to(g.dtype) for g in grads]


# ------------------------------------------------------------------------------------------ the calls

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import means_nearest_centroid_gb300 as km

        if op == "route":
            return km.kmassign_route(state["logits"], case["k"], score=case["score"], bias=state["bias"],
                                     groups=case["groups"], topk_groups=case["topk_groups"],
                                     group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
        if op == "route_grad":
            return km.kmassign_route_grad(state["logits"], state["idx"], state["dweights"], score=case["score"],
                                          renorm=case["renorm"], scale=case["scale"])
        if op == "lookup":
            return km.kmassign_lookup(state["table"], state["idx"], weights=state["weights"], scale=case["scale"])
        if op == "lookup_grad":
            return km.kmassign_lookup_grad(state["dout"], state["idx"], case["K"], weights=state["weights"],
                                           table=state.get("table"), scale=case["scale"], dtype=TYPES[case["grad"]])
        if op == "lists":
            return km.kmassign_lists(state["idx"], case["K"])
        norm = km.kmassign_clip(state["grads"], case["max_norm"], out=state["out"])
        return norm, state["out"]
    if op == "route":
        return _plain_route(case, state["logits"], state["bias"])
    if op == "route_grad":
        return _plain_route_grad(case, state["logits"], state["idx"], state["dweights"])
    if op == "lookup":
        return _plain_lookup(case, state["table"], state["idx"], state["weights"])
    if op == "lookup_grad":
        return _plain_lookup_grad(case, state["dout"], state["idx"], state["weights"], state.get("table"))
    if op == "lists":
        return _plain_lists(state["idx"], case["K"])
    return _plain_clip(state["grads"], case["max_norm"])


# ------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits; None for whole numbers."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "lists":
        return None
    if op == "clip":
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        return torch.tensor(norm, dtype=torch.float64), [g.double() * c for g in s["grads"]]
    if op == "route":
        x = s["logits"].double().cpu().numpy()
        N, E = x.shape
        off = np.isnan(x) | np.isneginf(x)
        with np.errstate(all="ignore"):
            if case["score"] == "softmax":
                p = np.where(off, 0.0, np.exp(x - np.max(np.where(off, -np.inf, x), 1, keepdims=True)))
                p = np.nan_to_num(p / p.sum(1, keepdims=True))
            else:
                p = np.where(off, 0.0, 1.0 / (1.0 + np.exp(-x)))
            # keys are held in 32 bits where a bias is added
            key = x.copy() if s["bias"] is None else p.astype(np.float32) + s["bias"].cpu().numpy()
            key[off] = -np.inf
            G = case["groups"]
            if G > 1:
                m = key if s["bias"] is not None or case["group_top"] == 1 else np.where(off, -np.inf, p)
                m = -np.sort(-m.reshape(N, G, E // G), axis=2)[:, :, :case["group_top"]]
                gk = np.where(np.isneginf(m[:, :, 0]), -np.inf, np.where(np.isneginf(m), 0, m).sum(2))
                out_of = np.argsort(-gk, axis=1, kind="stable")[:, case["topk_groups"]:]
                gone = np.zeros((N, G), dtype=bool)
                np.put_along_axis(gone, out_of, True, 1)
                key[np.repeat(gone, E // G, axis=1)] = -np.inf
            sel = np.argsort(-key, axis=1, kind="stable")[:, :case["k"]]
            empty = np.isneginf(np.take_along_axis(key, sel, 1))
            w = np.where(empty, 0.0, np.take_along_axis(p, sel, 1))
            if case["renorm"]:
                w = np.nan_to_num(w / w.sum(1, keepdims=True))
        return None, w * case["scale"]
    if op == "route_grad":
        x = s["logits"].double()
        idx = s["idx"].long()
        ok = (idx >= 0) & (idx < x.shape[1])
        # dense gradient of the weights, dense selection
        g = torch.zeros_like(x).scatter_add_(1, idx.clamp(0, x.shape[1] - 1), s["dweights"].double() * ok)
        sel = torch.zeros_like(x).scatter_add_(1, idx.clamp(0, x.shape[1] - 1), ok.double()) > 0
        live = ~(torch.isnan(x) | torch.isinf(x))
        z = torch.where(live, x, 0.0)
        if case["score"] == "sigmoid":
            p = torch.sigmoid(z) * live
            if case["renorm"]:
                p = p * sel
                total = p.sum(1, keepdim=True)
                d = p * (1 - p) * (g * total - (p * g).sum(1, keepdim=True)) / total ** 2
                d = torch.nan_to_num(d)
            else:
                d = p * (1 - p) * g
        else:
            over = live & sel if case["renorm"] else live
            p = torch.softmax(torch.where(over, z, -1e300), 1) * over
            d = p * (g - (p * g).sum(1, keepdim=True))
        return d * case["scale"]
    idx = s["idx"].long().view(case["N"], -1)
    ok = (idx >= 0) & (idx < case["K"])
    at = idx.clamp(0, case["K"] - 1)
    w = torch.ones(idx.shape, dtype=torch.float64, device=idx.device) if s["weights"] is None else s["weights"].double().view(idx.shape)
    w = w * ok * case["scale"]
    steps = range(idx.shape[1])
    if op == "lookup":
        return sum(s["table"][at[:, j]].double() * w[:, j:j + 1] for j in steps)
    d = s["dout"].double()
    dtable = torch.zeros(case["K"], case["D"], dtype=torch.float64, device=d.device)
    for j in steps:
        dtable.index_add_(0, at[:, j], d * w[:, j:j + 1])
    if s["weights"] is None:
        return dtable, None
    dw = torch.stack([(s["table"][at[:, j]].double() * d).sum(1) for j in steps], 1) * ok * case["scale"]
    return dtable, dw.view(s["idx"].shape)
