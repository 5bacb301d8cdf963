"""Experts behind a router, as they are measured: the root-mean-square norm in front of them (with the
residual's addition and an output in 8 bits), the products grouped by expert, the same in 8 bits with a scale
for each block of 128, and the gradients.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true, with the
library's entry points.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2, "e4m3": 1}
BLOCK = 128          # columns that share a scale; of weights, BLOCK rows too
TOP = 448.0          # e4m3's largest number
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # A decoding step's norm in front of 8-bit experts: sixteen rows, the residual added on the way.
        {"name": "norm_decode", "op": "norm", "N": 16, "D": 2048, "dtype": "bf16", "out": "e4m3", "residual": True},
        # The same over a long batch.
        {"name": "norm_batch", "op": "norm", "N": 65536, "D": 2048, "dtype": "bf16", "out": "e4m3", "residual": True},
        # Training: the norm's gradients, the residual stream's own gradient added.
        {"name": "norm_grad_batch", "op": "norm_grad", "N": 65536, "D": 2048, "dtype": "bf16", "residual": True},
        # Rows of an odd length in 32 bits.
        {"name": "norm_grad_ragged", "op": "norm_grad", "N": 30011, "D": 777, "dtype": "fp32", "residual": False},
        # A decoding step's experts: sixteen points, 8 of 256 experts each; the weights are what counts.
        {"name": "experts_decode", "op": "experts", "N": 16, "k": 8, "E": 256, "D": 2048, "F": 1024, "dtype": "bf16",
         "form": "in", "skew": 1.0},
        # A training batch's first product: points gathered by expert.
        {"name": "experts_batch", "op": "experts", "N": 16384, "k": 8, "E": 64, "D": 2048, "F": 1024, "dtype": "bf16",
         "form": "in", "skew": 1.0},
        # A second product, its rows put back to their points' places; odd sizes, uneven experts.
        {"name": "experts_back", "op": "experts", "N": 5003, "k": 3, "E": 40, "D": 1000, "F": 712, "dtype": "fp16",
         "form": "out", "skew": 1.5},
        # The gradients of the first product: of the points and of all experts' weights.
        {"name": "experts_grad_batch", "op": "experts_grad", "N": 16384, "k": 8, "E": 64, "D": 2048, "F": 1024,
         "dtype": "bf16", "grad": "bf16", "form": "in", "skew": 1.0},
        # The gradients of the second one.
        {"name": "experts_grad_back", "op": "experts_grad", "N": 5003, "k": 3, "E": 40, "D": 1000, "F": 712,
         "dtype": "fp16", "grad": "fp32", "form": "out", "skew": 1.5},
        # A decoding step's experts in 8 bits.
        {"name": "experts8_decode", "op": "experts8", "N": 16, "k": 8, "E": 256, "D": 2048, "F": 1024, "dtype": "bf16",
         "form": "in", "skew": 1.0},
        # A long batch of prompts through 8-bit experts.
        {"name": "experts8_batch", "op": "experts8", "N": 16384, "k": 8, "E": 64, "D": 2048, "F": 1024, "dtype": "bf16",
         "form": "in", "skew": 1.0},
        # One layer of 8-bit weights for all points (an expert that all share).
        {"name": "product8", "op": "experts8", "N": 8003, "k": 1, "E": 1, "D": 4096, "F": 4096, "dtype": "bf16",
         "form": "all", "skew": 1.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "experts", "experts", "experts_grad", "experts_grad", "experts8", "experts8"])
    if op in ("norm", "norm_grad"):
        D = _log(rng, 16, 16384)
        case = {"op": op, "N": _log(rng, 1, min(65536, (1 << 27) // D)), "D": D,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "residual": rng.random() < 0.6}
        if op == "norm":
            case["out"] = rng.choice(["e4m3", case["dtype"]])
        return case
    step = 16 if op == "experts8" else 8
    form = rng.choice(["in", "in", "out"] + (["all"] if op != "experts_grad" else []))
    E = 1 if form == "all" else _log(rng, 1, 256)
    k = 1 if form == "all" else rng.randint(1, min(E, 8))
    D = step * _log(rng, 2, 4096 // step)
    F = 8 * _log(rng, 2, min(4096 // 8, (1 << 26) // (D * E)))
    # no more products than the largest listed case, no more gathered rows, and weights of 1 GB at most
    N = _log(rng, 1, max(2, min(16384, (1 << 38) // (k * D * F), (1 << 28) // (k * max(D, F)))))
    case = {"op": op, "N": N, "k": k, "E": E, "D": D, "F": F, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
            "form": form, "skew": rng.choice([1.0, 1.0, 1.5])}
    if op == "experts_grad":
        case["grad"] = rng.choice(["fp32", case["dtype"]])
    return case


def _blocks(n):
    return -(-n // BLOCK)


def _named(case):
    """How many experts at least one point is expected to go to."""
    E, p = case["E"], case["k"] / case["E"]
    return E * (1.0 - (1.0 - min(p, 1.0)) ** case["N"])


def work(case):
    N, D, b = case["N"], case["D"], BYTES[case["dtype"]]
    if case["op"] == "norm":
        out = D * BYTES[case["out"]] + (4 * _blocks(D) if case["out"] == "e4m3" else 0)
        return {"bytes": N * ((3 if case["residual"] else 1) * D * b + out + 4) + D * b, "flops": 6 * N * D}
    if case["op"] == "norm_grad":
        return {"bytes": N * ((4 if case["residual"] else 3) * D * b + 4) + D * (b + 4), "flops": 10 * N * D}
    k, E, F = case["k"], case["E"], case["F"]
    M, named = N * k, _named(case)
    rows = N if case["form"] == "in" else M
    ids = 0 if case["form"] == "all" else 4 * M + 4 * (E + 1)
    if case["op"] == "experts8":
        x = rows * (D + 4 * _blocks(D))
        w = named * (F * D + 4 * _blocks(F) * _blocks(D))
        return {"bytes": int(x + w + ids + M * F * b), "flops": 2 * M * F * D}
    if case["op"] == "experts":
        return {"bytes": int(rows * D * b + named * F * D * b + ids + M * F * b), "flops": 2 * M * F * D}
    return {"bytes": int(2 * rows * D * b + named * F * D * b + M * F * b + E * F * D * BYTES[case["grad"]] + ids),
            "flops": 4 * M * F * D}


# --------------------------------------------------------------------------------------------- inputs

def _in_8_bits(x, rows):
    """Codes and scales of x [..., R, D], a scale for each block of BLOCK columns and `rows` rows."""
    R, D = x.shape[-2:]
    up = torch.nn.functional.pad(x, (0, _blocks(D) * BLOCK - D, 0, -(-R // rows) * rows - R))
    tiles = up.view(*x.shape[:-2], up.shape[-2] // rows, rows, _blocks(D), BLOCK)
    scale = tiles.abs().amax(dim=(-3, -1)).clamp_(min=1e-30) / TOP
    codes = (tiles / scale[..., :, None, :, None]).to(torch.float8_e4m3fn).view(up.shape)
    return codes[..., :R, :D].contiguous(), scale.contiguous()


def _choice(case, gen):
    """k different experts a point, low ones more often where skew > 1; one point in fifty has a free slot."""
    N, k, E = case["N"], case["k"], case["E"]
    often = (torch.arange(E, device=DEVICE) + 1.0) ** (1.0 / case["skew"] - 1.0)
    key = torch.rand(N, E, generator=gen, device=DEVICE).clamp_(min=1e-9).log_().div_(often)
    idx = key.argsort(-1, descending=True)[:, :k].to(torch.int32)
    if k > 1:
        free = torch.rand(N, generator=gen, device=DEVICE) < 0.02
        idx[:, -1] = torch.where(free, -1, idx[:, -1])
    return idx.contiguous()


def _lists(idx, E):
    """The slots of each expert in turn, and where each one's begin; -1 behind the last."""
    flat = idx.view(-1)
    expert, order = torch.where(flat < 0, E, flat).sort(stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.bincount(expert, minlength=E + 1)[:E].cumsum(0)
    return torch.where(expert < E, order, -1).to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEVICE)  # noqa: E731
    N, D, kind = case["N"], case["D"], TYPES[case["dtype"]]
    state = {"case": dict(case)}
    if case["op"] in ("norm", "norm_grad"):
        # Rows of different sizes with a few large columns, as hidden states have them.
        wide = torch.exp(0.5 * normal(D))
        x = (normal(N, D) * wide * torch.exp(normal(N, 1))).to(kind)
        state["weight"] = (1.0 + 0.1 * normal(D)).to(kind)
        if case["op"] == "norm":
            state["x"] = x
            state["residual"] = (normal(N, D) * wide).to(kind) if case["residual"] else None
            return state
        state["total"] = x
        state["rstd"] = torch.rsqrt(x.double().square().mean(-1) + EPS).float()
        state["dout"] = (0.1 * normal(N, D)).to(kind)
        state["dtotal"] = (0.1 * normal(N, D)).to(kind) if case["residual"] else None
        return state
    k, E, F = case["k"], case["E"], case["F"]
    M = N * k
    if case["form"] == "all":
        state["order"] = state["offsets"] = None
        state["most"] = N
    else:
        state["order"], state["offsets"] = _lists(_choice(case, gen), E)
        # the capacity that a padded batch of products needs
        state["most"] = max(1, int(state["offsets"].diff().max()))
    x = normal(N if case["form"] != "out" else M, D)
    w = normal(E, F, D).mul_(D ** -0.5)
    if case["op"] == "experts8":
        # Columns and blocks of weights of different sizes: the scales differ.
        x.mul_(torch.exp(0.5 * normal(D)))
        w.mul_(torch.exp(0.5 * normal(E, F, 1)))
        state["x"], state["xscale"] = _in_8_bits(x, 1)
        state["w"], state["wscale"] = _in_8_bits(w, BLOCK)
    else:
        state["x"], state["w"] = x.to(kind), w.to(kind)
    if case["form"] == "all":
        state["w"] = state["w"][0]
        state["wscale"] = state["wscale"][0] if "wscale" in state else None
    if case["op"] == "experts_grad":
        state["dout"] = (0.1 * normal(M, F)).to(kind)
    return state


# ---------------------------------------------------------------------------------------- plain forms

def _plain_norm(case, x, weight, residual):
    total = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    t = total.float()
    rstd = torch.rsqrt(t.square().mean(-1) + EPS)
    y = t * rstd[:, None] * weight.float()
    if case["out"] != "e4m3":
        return y.to(x.dtype), None, total, rstd
    N, D = y.shape
    tiles = torch.nn.functional.pad(y, (0, _blocks(D) * BLOCK - D)).view(N, -1, BLOCK)
    scales = tiles.abs().amax(-1).clamp(min=2.0 ** -100) / TOP
    codes = (tiles / scales[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(N, -1)
    return codes[:, :D].contiguous(), scales, total, rstd


def _plain_norm_grad(dout, total, weight, rstd, dtotal):
    t = total.float() * rstd[:, None]
    d = dout.float()
    g = d * weight.float()
    dx = (g - t * (g * t).mean(-1, keepdim=True)) * rstd[:, None]
    if dtotal is not None:
        dx = dx + dtotal.float()
    return dx.to(total.dtype), (d * t).sum(0)


def _values(state, name):
    """fp32 values of the points or the weights, scales applied."""
    x = state[name].float()
    scale = state.get(name + "scale")
    if scale is None:
        return x
    wide = scale.repeat_interleave(BLOCK, -1)[..., :x.shape[-1]]
    if name == "w":
        wide = wide.repeat_interleave(BLOCK, -2)[..., :x.shape[-2], :]
    return x * wide


def _padded(state):
    """Every expert's list positions [E, most], which of them are there, and the slots [E, most] they stand for."""
    offsets, order = state["offsets"].long(), state["order"].long()
    at = offsets[:-1, None] + torch.arange(state["most"], device=offsets.device)
    there = at < offsets[1:, None]
    at = torch.where(there, at, 0)
    return at, there, torch.where(there, order[at], 0)


def _plain_experts(state):
    case = state["case"]
    x, w = _values(state, "x"), _values(state, "w")
    kind = TYPES[case["dtype"]]
    if case["form"] == "all":
        return (x @ w.transpose(-1, -2)).to(kind)
    at, there, slot = _padded(state)
    take, put = (slot // case["k"], at) if case["form"] == "in" else (at, slot)
    M = case["N"] * case["k"]
    y = torch.bmm(x[take], w.transpose(-1, -2)).to(kind)
    out = torch.zeros(M + 1, case["F"], dtype=kind, device=x.device)
    out[torch.where(there, put, M)] = y
    return out[:M]


def _plain_experts_grad(state):
    case = state["case"]
    x, w, dout = state["x"].float(), state["w"].float(), state["dout"].float()
    at, there, slot = _padded(state)
    take, put = (slot // case["k"], at) if case["form"] == "in" else (at, slot)
    dy = dout[put] * there[..., None]
    rows = x.shape[0]
    dx = torch.zeros(rows + 1, case["D"], device=x.device)
    dx.index_add_(0, torch.where(there, take, rows).view(-1), torch.bmm(dy, w).view(-1, case["D"]))
    dw = torch.bmm(dy.transpose(-1, -2), x[take])
    return dx[:rows].to(state["x"].dtype), dw.to(TYPES[case["grad"]])


# ------------------------------------------------------------------------------------------ the calls

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import means_nearest_centroid_gb300 as km

        if op == "norm":
            return km.kmassign_rmsnorm(state["x"], state["weight"], residual=state["residual"], eps=EPS,
                                       dtype=TYPES[case["out"]])
        if op == "norm_grad":
            return km.kmassign_rmsnorm_grad(state["dout"], state["total"], state["weight"], state["rstd"],
                                            dtotal=state["dtotal"])
        lists = {"offsets": state["offsets"]}
        if case["form"] == "in":
            lists.update(rows=state["order"], slots=case["k"])
        elif case["form"] == "out":
            lists.update(places=state["order"])
        if op == "experts":
            return km.kmassign_experts(state["x"], state["w"], **lists)
        if op == "experts8":
            return km.kmassign_experts(state["x"], state["w"], xscale=state["xscale"], wscale=state["wscale"],
                                       dtype=TYPES[case["dtype"]], **lists)
        return km.kmassign_experts_grad(state["dout"], state["x"], state["w"], dtype=TYPES[case["grad"]], **lists)
    if op == "norm":
        return _plain_norm(case, state["x"], state["weight"], state["residual"])
    if op == "norm_grad":
        return _plain_norm_grad(state["dout"], state["total"], state["weight"], state["rstd"], state["dtotal"])
    if op == "experts_grad":
        return _plain_experts_grad(state)
    return _plain_experts(state)


# ------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    N, D = case["N"], case["D"]
    if case["op"] == "norm":
        total = s["x"].double()
        if case["residual"]:
            # the sum is kept in the rows' type, and the norm is taken of what is kept
            total = (total + s["residual"].double()).to(s["x"].dtype).double()
        ms = (total * total).sum(1) / D
        y = total / (ms + EPS).sqrt().unsqueeze(1) * s["weight"].double()
        rstd = 1.0 / (ms + EPS).sqrt()
        if case["out"] != "e4m3":
            return y, None, total, rstd
        scales = torch.stack([b.abs().max(1).values for b in y.split(BLOCK, 1)], 1).clamp(min=2.0 ** -100) / TOP
        codes = torch.cat([(b / scales[:, i:i + 1]).float().to(torch.float8_e4m3fn).double()
                           for i, b in enumerate(y.split(BLOCK, 1))], 1)
        return codes, scales, total, rstd
    if case["op"] == "norm_grad":
        d, t, w, r = s["dout"].double(), s["total"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
        inner = (d * w * t).sum(1, keepdim=True) / D
        dx = r * d * w - r ** 3 * inner * t
        return dx + (s["dtotal"].double() if case["residual"] else 0.0), (d * t * r).sum(0)
    k, E, F = case["k"], case["E"], case["F"]
    M = N * k
    if s["offsets"] is None:
        edges, order = [0, N], torch.arange(N, device=DEVICE)
    else:
        edges, order = s["offsets"].tolist(), s["order"].long()
    w_of = s["w"].view(E, F, D)

    def weights(e):
        w = w_of[e].double()
        if case["op"] == "experts8":
            t = s["wscale"].view(E, _blocks(F), _blocks(D))[e].double()
            w = w * t[torch.arange(F, device=DEVICE) // BLOCK][:, torch.arange(D, device=DEVICE) // BLOCK]
        return w

    def points(rows):
        x = s["x"][rows].double()
        if case["op"] == "experts8":
            x = x * s["xscale"][rows].double()[:, torch.arange(D, device=DEVICE) // BLOCK]
        return x

    if case["op"] == "experts_grad":
        dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEVICE)
        dw = torch.zeros(E, F, D, dtype=torch.float64, device=DEVICE)
    else:
        out = torch.zeros(M, F, dtype=torch.float64, device=DEVICE)
    for e in range(E):
        place = torch.arange(edges[e], edges[e + 1], device=DEVICE)
        if not len(place):
            continue
        slot = order[place]
        rows, put = {"in": (slot // k, place), "out": (place, slot), "all": (place, place)}[case["form"]]
        if case["op"] == "experts_grad":
            dy = s["dout"][put].double()
            dx.index_add_(0, rows, dy @ weights(e))
            dw[e] = dy.t() @ points(rows)
        else:
            out[put] = points(rows) @ weights(e).t()
    return (dx, dw) if case["op"] == "experts_grad" else out
