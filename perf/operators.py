"""The operators for training and serving low-rank adapters beside a compressed
weight, as cases that can be timed: the global gradient norm and clipping over
many tensors, the grouping of a batch's tokens by adapter, and the adapters'
product and its gradients.

``run`` computes a case either with elementary torch operations in 32 bits
(``own`` false) or through the package's entry points (``own`` true);
``exact`` computes it in 64 bits from the definitions:

    norm      |G| = sqrt(sum over all tensors of g^2)
    clip      c = min(1, max_norm / (|G| + 1e-6)),  g' = c*g
    plan      the tokens in stable order of their adapter, each adapter's first
              place in that order, and its tiles of at most 128 tokens
    forward   out = y + s_a (x A_a^T) B_a^T        for a token of adapter a
    backward  d = s_a dy B_a,  dx' = dx + d A_a,
              dA_a = sum d^T x,  dB_a = sum s_a dy^T (x A_a^T)

A token whose adapter is -1 has none: its out is y and its dx' is dx.  Adapter
a uses the first ranks[a] of the R rows of A_a (columns of B_a).
"""
import math
import random

import torch

own = False

TILE = 128       # tokens in a tile of the plan
MAX_NORM = 1.0
EPS = 1e-6

# The most that a drawn case may ask for, set by the largest listed ones.
MOST_VALUES = 162_000_000
MOST_MOVED = 8192 * (4096 + 2 * 8192)
MOST_PRODUCT = 16 * 64 * 8192 * (4096 + 8192)


def _grads(name, kind, tensors, values, dtype, flat, scale):
    return {"name": name, "kind": kind, "tensors": tensors, "values": values, "dtype": dtype, "flat": flat,
            "scale": scale}


def _plan(name, tokens, adapters, runs, none):
    return {"name": name, "kind": "plan", "tokens": tokens, "adapters": adapters, "runs": runs, "none": none}


def _apply(name, kind, tokens, adapters, rank, ins, outs, runs, none, mixed):
    return {"name": name, "kind": kind, "tokens": tokens, "adapters": adapters, "rank": rank, "ins": ins,
            "outs": outs, "runs": runs, "none": none, "mixed": mixed}


def listed():
    return [
        # the gradients of a few adapters of one projection: latency is what counts
        _grads("norm_adapters", "norm", 14, 65_536, "bf16", False, 1e-2),
        # every gradient of a 162-million-value model (the fused steps' workload), logged without clipping
        _grads("norm_162m", "norm", 290, 162_000_000, "bf16", False, 1e-3),
        # gradients accumulated in 32 bits beside 16-bit ones, as views of packed buckets at odd offsets
        _grads("clip_buckets", "clip", 75, 20_000_003, "mixed", True, 1e-2),
        # the clipping before a fused step over 162 million values
        _grads("clip_162m", "clip", 290, 162_000_000, "bf16", False, 1e-3),
        # one decode step of a server: every request brings one token, any adapter
        _plan("plan_decode", 256, 64, False, True),
        # a batch of prompts, each a run of tokens with one adapter
        _plan("plan_prompts", 16_384, 32, True, True),
        # one request being decoded
        _apply("token", "forward", 1, 16, 16, 4096, 4096, False, False, False),
        # a decode batch of many requests, adapters in any order
        _apply("decode", "forward", 64, 64, 16, 4096, 4096, False, True, False),
        # a ragged batch: odd sizes, ranks of their own, requests without an adapter
        _apply("ragged", "forward", 777, 5, 24, 1001, 2047, True, True, True),
        # prompts of many requests
        _apply("prompts", "forward", 8192, 16, 64, 4096, 8192, True, True, False),
        # training several adapters at once on a shared projection of 1024 to 4096
        _apply("train_several", "backward", 2048, 4, 32, 1024, 4096, True, True, True),
        # training one adapter on long sequences
        _apply("train_one", "backward", 16_384, 1, 64, 4096, 4096, True, False, False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm; 3072 is left out."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v == 3072 else v


def draw(rng):
    kind = rng.choice(["norm", "clip", "plan", "forward", "forward", "backward"])
    if kind in ("norm", "clip"):
        tensors = _spread(rng, 1, 400)
        values = max(tensors, _spread(rng, 4096, MOST_VALUES))
        case = _grads("", kind, tensors, values, rng.choice(["bf16", "f32", "mixed"]), rng.random() < 0.5,
                      rng.choice([1e-7, 1e-3, 1e-2, 1.0]))
    elif kind == "plan":
        case = _plan("", _spread(rng, 1, 16_384), _spread(rng, 1, 256), rng.random() < 0.5, rng.random() < 0.5)
    else:
        while True:
            tokens = _spread(rng, 1, 16_384)
            size = (tokens, _spread(rng, 1, 128), rng.choice([4, 8, 16, 32, 64, 128, _spread(rng, 1, 128)]),
                    rng.choice([256, 512, 1024, 4096, 8192, _spread(rng, 64, 8192)]),
                    rng.choice([256, 512, 1024, 4096, 8192, _spread(rng, 64, 8192)]))
            t, n, r, k, m = size
            if t * (k + 2 * m) <= MOST_MOVED and t * n * r * (k + m) <= MOST_PRODUCT:
                break
        case = _apply("", kind, *size, rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.4)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _sizes(case):
    """The tensors' sizes: a few large ones and many small ones, odd as they come, `values` in all."""
    tensors, values = case["tensors"], case["values"]
    rng = random.Random(tensors * 1_000_003 + values)
    weight = [2.0 ** rng.uniform(0, 12) for _ in range(tensors)]
    total = sum(weight)
    sizes = [max(1, int(values * w / total)) for w in weight]
    big = sizes.index(max(sizes))
    sizes[big] = max(1, sizes[big] + values - sum(sizes))
    return sizes


def _kinds(case):
    return {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}[case["dtype"]]


def _buckets(case, kinds):
    """One zeroed buffer for each type, and a view of its type's for each tensor: packed (odd offsets) in a flat
    case, else every view begins a 256-byte line."""
    sizes = _sizes(case)
    line = 1 if case["flat"] else 128
    buffers, views = [], [None] * len(sizes)
    for k, dtype in enumerate(kinds):
        mine = list(range(k, len(sizes), len(kinds)))
        room = [(sizes[i] + line - 1) // line * line for i in mine]
        buffers.append(torch.zeros(sum(room), dtype=dtype, device="cuda"))
        for i, part in zip(mine, buffers[-1].split(room) if mine else []):
            views[i] = part[:sizes[i]]
    return buffers, views


def _gradients(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    views = _buckets(case, _kinds(case))[1]
    for g in views:
        g.copy_(torch.randn(g.numel(), generator=gen, device="cuda").mul_(case["scale"]))
    return views


def _index(case, seed):
    """Each token's adapter: runs of tokens (requests one after another) or any order; -1 for none."""
    rng = random.Random(seed * 7919 + case["tokens"])
    t, n = case["tokens"], case["adapters"]
    low = -1 if case["none"] else 0
    if not case["runs"]:
        index = [rng.randint(low, n - 1) for _ in range(t)]
    else:
        index = []
        while len(index) < t:
            index += [rng.randint(low, n - 1)] * rng.randint(1, max(1, 2 * t // (n + 1)))
    return torch.tensor(index[:t], dtype=torch.int32, device="cuda")


def _order(index, adapters):
    """The stable grouping of the tokens by adapter (those without one last), from comparisons and running sums."""
    tokens = index.numel()
    group = torch.where(index < 0, adapters, index).long()
    one = (group[:, None] == torch.arange(adapters + 1, device=index.device)).int()
    count = one.sum(0)
    starts = torch.zeros(adapters + 2, dtype=torch.int32, device=index.device)
    starts[1:] = count.cumsum(0)
    place = starts[group] + one.cumsum(0).gather(1, group[:, None])[:, 0] - 1
    order = torch.empty(tokens, dtype=torch.int32, device=index.device)
    order[place.long()] = torch.arange(tokens, dtype=torch.int32, device=index.device)
    # tiles: group by group, rows of (adapter, first place, tokens, 0); the rest of the table is zero
    rows = (tokens + TILE - 1) // TILE + min(adapters + 1, tokens)
    per = (count + TILE - 1) // TILE
    end = per.cumsum(0)
    row = torch.arange(rows, device=index.device)
    g = (row[:, None] >= end).sum(1).clamp(max=adapters)
    nth = row - (end - per)[g]
    used = row < end[-1]
    first = starts[g] + TILE * nth
    tiles = torch.stack([torch.where(g == adapters, -1, g), first, (starts[g + 1] - first).clamp(max=TILE),
                         torch.zeros_like(row)], 1)
    return order, starts, torch.where(used[:, None], tiles, 0).int()


def _tensors(case, seed):
    """x, y (or dy and dx), A, B, scales, ranks and each token's adapter."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    t, n, r, k, m = case["tokens"], case["adapters"], case["rank"], case["ins"], case["outs"]
    channel = torch.exp(0.5 * normal(k))       # some channels of activations are far larger than others
    state = {"index": _index(case, seed), "x": (normal(t, k) * channel).bfloat16(),
             "a": (normal(n, r, k) / math.sqrt(k)).bfloat16(), "b": (normal(n, m, r) * 0.05).bfloat16(),
             "scale": torch.rand(n, generator=gen, device="cuda") + 0.5, "ranks": None}
    if case["mixed"]:
        state["ranks"] = torch.randint(1, r + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    if case["kind"] == "forward":
        state["y"] = normal(t, m).bfloat16()
    else:
        state["dy"] = (normal(t, m) * 1e-2).bfloat16()
        state["dx"] = (normal(t, k) * 1e-2).bfloat16()
    return state


def prepare(case, seed):
    kind = case["kind"]
    if kind in ("norm", "clip"):
        state = {"grads": _gradients(case, seed)}
        if kind == "clip":
            state["buffers"], state["out"] = _buckets(case, _kinds(case))
    elif kind == "plan":
        state = {"index": _index(case, seed)}
    else:
        state = _tensors(case, seed)
        state["plan"] = _order(state["index"], case["adapters"])      # made once for a batch
        if kind == "backward":
            state["xa"] = _inner(state, state["x"], state["a"])       # the forward pass keeps it
    return {"case": case, **state}


# -------------------------------------------------------------- plain form

def _mask(state):
    """[tokens, adapters, R]: whether a token's adapter uses that rank."""
    n, r = state["a"].shape[:2]
    mine = state["index"][:, None] == torch.arange(n, device="cuda")
    if state["ranks"] is None:
        return mine[:, :, None].expand(-1, -1, r)
    return mine[:, :, None] & (torch.arange(r, device="cuda") < state["ranks"][:, None])


def _inner(state, x, a):
    """[tokens, R]: x A_a^T of each token's own adapter."""
    n, r, k = a.shape
    all_of = (x.float() @ a.float().reshape(n * r, k).t()).view(-1, n, r)
    return torch.where(_mask(state), all_of, 0.0).sum(1)


def _norm(grads):
    return torch.cat([g.reshape(-1).float() for g in grads]).square().sum().sqrt()


def _plain(state):
    kind = state["case"]["kind"]
    if kind == "norm":
        return _norm(state["grads"])
    if kind == "clip":
        norm = _norm(state["grads"])
        c = (MAX_NORM / (norm + EPS)).clamp(max=1.0)
        [out.copy_(g.float() * c) for out, g in zip(state["out"], state["grads"])]
        return norm, state["buffers"]
    if kind == "plan":
        return _order(state["index"], state["case"]["adapters"])
    n, r, k = state["a"].shape
    m = state["b"].shape[1]
    a = state["a"].float().reshape(n * r, k)
    b = state["b"].float().transpose(1, 2).reshape(n * r, m)
    x = state["x"].float()
    mask = _mask(state)
    s = state["scale"][None, :, None]
    if kind == "forward":
        v = torch.where(mask, (x @ a.t()).view(-1, n, r) * s, 0.0)
        return (state["y"].float() + v.view(-1, n * r) @ b).bfloat16()
    dy = state["dy"].float()
    d = torch.where(mask, (dy @ b.t()).view(-1, n, r) * s, 0.0).view(-1, n * r)
    v = torch.where(mask, state["xa"][:, None, :] * s, 0.0).view(-1, n * r)
    dx = (state["dx"].float() + d @ a).bfloat16()
    da = (d.t() @ x).bfloat16().view(n, r, k)
    db = (v.t() @ dy).view(n, r, m).transpose(1, 2).bfloat16().contiguous()
    return dx, da, db


def run(state):
    if not own:
        return _plain(state)
    from lossless_bf16_tensor_gb300 import adapters, grads
    kind = state["case"]["kind"]
    if kind == "norm":
        return grads.grad_norm(state["grads"])
    if kind == "clip":
        norm = grads.clip_grads(state["grads"], MAX_NORM, out=state["out"])
        return norm, state["buffers"]
    if kind == "plan":
        plan = adapters.adapter_plan(state["index"], state["case"]["adapters"])
        return plan.order, plan.starts, plan.tiles
    bank = adapters.AdapterBank(state["a"], state["b"], state["scale"], state["ranks"])
    plan = adapters.AdapterPlan(*state["plan"])
    if kind == "forward":
        return adapters.adapter_apply(state["x"], bank, plan, state["y"])
    return adapters.adapter_grads(state["dy"], state["x"], state["xa"], bank, plan, state["dx"])


# ------------------------------------------------------------ work and exact

def work(case):
    kind = case["kind"]
    if kind in ("norm", "clip"):
        v = case["values"]
        wide = sum(_sizes(case)[1::2]) if case["dtype"] == "mixed" else (v if case["dtype"] == "f32" else 0)
        size = 2 * v + 2 * wide
        return {"bytes": size + 4, "flops": 2 * v} if kind == "norm" else {"bytes": 2 * size + 4, "flops": 3 * v}
    t, n = case["tokens"], case["adapters"]
    if kind == "plan":
        rows = (t + TILE - 1) // TILE + min(n + 1, t)
        return {"bytes": 4 * (2 * t + n + 2 + 4 * rows), "flops": 0}
    r, k, m = case["rank"], case["ins"], case["outs"]
    weights = 2 * min(n, t) * r * (k + m)
    if kind == "forward":
        return {"bytes": 2 * t * (k + 2 * m) + weights + 4 * t, "flops": 2 * t * r * (k + m)}
    # dy, x, dx in and dx' out, the kept x A^T, the weights that are used and all their gradients
    return {"bytes": 2 * t * (3 * k + m) + 4 * t * r + weights + 2 * n * r * (k + m) + 4 * t,
            "flops": 4 * t * r * (k + m)}


def exact(case, seed):
    kind = case["kind"]
    if kind == "plan":
        return None
    if kind in ("norm", "clip"):
        made = _gradients(case, seed)
        total = 0.0
        for g in made:
            total += float((g.double() ** 2).sum())
        norm = torch.tensor(math.sqrt(total), dtype=torch.float64)
        if kind == "norm":
            return norm
        c = min(1.0, MAX_NORM / (math.sqrt(total) + EPS))
        buffers, views = _buckets(case, [torch.float64] * len(_kinds(case)))
        for out, g in zip(views, made):
            out.copy_(g.double() * c)
        return norm, buffers
    s = _tensors(case, seed)
    n, r = s["a"].shape[:2]
    out = (s["y"] if kind == "forward" else s["dx"]).double()
    da, db = torch.zeros_like(s["a"], dtype=torch.float64), torch.zeros_like(s["b"], dtype=torch.float64)
    for i in range(n):
        rows = (s["index"] == i).nonzero()[:, 0]
        if not rows.numel():
            continue
        used = r if s["ranks"] is None else int(s["ranks"][i])
        a, b = s["a"][i, :used].double(), s["b"][i, :, :used].double()
        x, f = s["x"][rows].double(), float(s["scale"][i])
        v = x @ a.t() * f
        if kind == "forward":
            out[rows] += v @ b.t()
            continue
        dy = s["dy"][rows].double()
        d = dy @ b * f
        out[rows] += d @ a
        da[i, :used] = d.t() @ x
        db[i, :, :used] = dy.t() @ v
    return out if kind == "forward" else (out, da, db)
