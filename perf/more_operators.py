"""The operators at the two ends of a language model, around the matrix of its
vocabulary, as cases that can be timed: the lookup of tokens' rows with its
gradient, and the cross entropy of a projection onto the vocabulary with its
gradients, which keeps no logits.

``run`` computes a case either with elementary torch operations in 32 bits
(``own`` false) or through the package's entry points (``own`` true);
``exact`` computes it in 64 bits from the definitions:

    lookup       out_i = f E_{t_i}                       (0 for t_i < 0)
    lookup_grad  dE_v = dE0_v + f sum over t_i = v of dy_i
    loss         z_iv = x_i W_v,  l_i = log sum_v exp z_iv,  loss_i = l_i - z_{i,t_i}
    grads        g_iv = c_i (exp(z_iv - l_i) - [v = t_i]),  dx = g W,  dW = g^T x
    step         the mean of the losses, and its gradients

A token with t_i < 0 has no row, no loss (0; its l_i is returned as it is) and
no gradients, and does not count in the mean.
"""
import math

import torch

own = False

# The most that a drawn case may ask for, set by the largest listed ones.
MOST_TABLE = 131_072 * 4096
MOST_ROWS = 16_384 * 4096
MOST_PRODUCT = 8192 * 32_768 * 4096
MOST_LOGITS = 8192 * 32_768


def _rows(name, kind, tokens, vocab, cols, dtype, factor, none, wide, base=False):
    """A case of the lookup: `wide` ids are int64, `base` is a gradient that the sums are added to."""
    return {"name": name, "kind": kind, "tokens": tokens, "vocab": vocab, "cols": cols, "dtype": dtype, "factor": factor,
            "none": none, "wide": wide, "base": base}


def _loss(name, kind, tokens, vocab, cols, none, wide, frozen=False):
    """A case of the loss: `none` is the share of tokens without a target, `frozen` leaves dW out."""
    return {"name": name, "kind": kind, "tokens": tokens, "vocab": vocab, "cols": cols, "none": none, "wide": wide,
            "frozen": frozen}


def listed():
    return [
        # one request being decoded: its last token's row
        _rows("token", "lookup", 1, 32_768, 4096, "bf16", 1.0, 0.0, True),
        # a padded batch of odd sizes on a 32-bit table, rows scaled as some models do
        _rows("lookup_ragged", "lookup", 777, 10_007, 1001, "f32", 31.6, 0.3, False),
        # prompts of many requests
        _rows("lookup_prompts", "lookup", 16_384, 131_072, 4096, "bf16", 1.0, 0.0, True),
        # a training batch of a small model
        _rows("table_small", "lookup_grad", 2048, 32_768, 1024, "bf16", 1.0, 0.1, True),
        # a padded batch whose table is also the projection: added to that one's gradient, in 32 bits, odd sizes
        _rows("table_tied", "lookup_grad", 5000, 10_007, 1001, "f32", 31.6, 0.3, False, True),
        # a training batch of long sequences over a large vocabulary
        _rows("table_prompts", "lookup_grad", 16_384, 131_072, 4096, "bf16", 1.0, 0.0, True),
        # one token scored
        _loss("score_token", "loss", 1, 32_768, 4096, 0.0, True),
        # a padded batch of odd sizes being evaluated
        _loss("score_ragged", "loss", 777, 5003, 1001, 0.3, False),
        # sequences being evaluated
        _loss("evaluate", "loss", 8192, 32_768, 4096, 0.0, True),
        # fine-tuning below a frozen projection, the prompts' tokens without a target
        _loss("frozen", "grads", 2048, 65_536, 1024, 0.5, True, True),
        # a training step of a small model, loss and gradients
        _loss("step", "step", 1000, 10_007, 1024, 0.1, True),
        # a training batch's gradients at a larger model's projection
        _loss("train", "grads", 8192, 32_768, 4096, 0.05, True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lookup", "lookup_grad", "loss", "grads", "grads", "step"])
    wide = rng.random() < 0.5
    none = rng.choice([0.0, 0.0, 0.1, 0.5, 0.9])
    while True:
        t = _spread(rng, 1, 16_384)
        v = rng.choice([1024, 32_768, 65_536, 131_072, _spread(rng, 2, 131_072), _spread(rng, 2, 131_072)])
        k = rng.choice([64, 512, 1024, 2048, 4096, _spread(rng, 8, 8192), _spread(rng, 8, 8192)])
        if kind in ("lookup", "lookup_grad"):
            if v * k <= MOST_TABLE and t * k <= MOST_ROWS:
                break
        elif t * v * k <= MOST_PRODUCT and t * v <= MOST_LOGITS and v * k <= MOST_TABLE // 2:
            break
    if kind in ("lookup", "lookup_grad"):
        case = _rows("", kind, t, v, k, rng.choice(["bf16", "bf16", "f32"]) if v * k <= MOST_TABLE // 2 else "bf16",
                     rng.choice([1.0, round(math.sqrt(k), 3)]), none, wide, kind == "lookup_grad" and rng.random() < 0.5)
    else:
        case = _loss("", kind, t, v, k, none, wide, kind == "grads" and rng.random() < 0.4)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(case, gen):
    """Each token's id: small ids are frequent (even over the logarithm, as words come), and a share has none: -1
    where a batch is padded, -100 where a target is left out."""
    t, v = case["tokens"], case["vocab"]
    u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(v + 1)) - 1).long().clamp(0, v - 1)
    if case["none"]:
        # runs of 16 tokens, as padding and prompts come
        runs = torch.rand((t + 15) // 16, generator=gen, device="cuda") < case["none"]
        ids[runs.repeat_interleave(16)[:t]] = -1 if "factor" in case else -100
    return ids if case["wide"] else ids.int()


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _row_tensors(case, seed):
    gen = _generator(seed)
    t, v, k = case["tokens"], case["vocab"], case["cols"]
    state = {"ids": _ids(case, gen)}
    if case["kind"] == "lookup":
        state["table"] = (torch.randn(v, k, generator=gen, device="cuda") * 0.02).to(_type(case))
    else:
        state["dy"] = (torch.randn(t, k, generator=gen, device="cuda") * 1e-3).to(_type(case))
        if case["base"]:
            state["base"] = (torch.randn(v, k, generator=gen, device="cuda") * 1e-3).to(_type(case))
    return state


def _loss_tensors(case, seed):
    """x, W, targets and each token's share c of the loss.  Logits spread over a few units, and x leans towards its
    target's row by a different amount for each token: some are sure, some are wrong."""
    gen = _generator(seed)
    t, v, k = case["tokens"], case["vocab"], case["cols"]
    state = {"ids": _ids(case, gen)}
    w = (torch.randn(v, k, generator=gen, device="cuda") * (2.0 / math.sqrt(k))).bfloat16()
    x = torch.randn(t, k, generator=gen, device="cuda")
    lean = torch.rand(t, 1, generator=gen, device="cuda") * 4.0
    x += lean * w[state["ids"].long().clamp(min=0)].float()
    state["x"], state["w"] = x.bfloat16(), w
    if case["kind"] == "grads":
        state["c"] = torch.rand(t, generator=gen, device="cuda") * (2.0 / t)
    return state


def prepare(case, seed):
    if "factor" in case:
        state = _row_tensors(case, seed)
    else:
        state = _loss_tensors(case, seed)
        if case["kind"] == "grads":      # the forward pass keeps these
            state["loss"], state["lse"] = _losses(state["x"], state["w"], state["ids"])[:2]
        if case["kind"] == "step":       # the leaves of a training program
            state["x"].requires_grad_(True)
            state["w"].requires_grad_(True)
    return {"case": case, **state}


# -------------------------------------------------------------- plain form

def _losses(x, w, ids):
    """loss, l and z in 32 bits."""
    z = x.float() @ w.float().t()
    top = z.amax(1, keepdim=True)
    lse = (z - top).exp().sum(1).log() + top[:, 0]
    mine = z.gather(1, ids.long().clamp(min=0)[:, None])[:, 0]
    return torch.where(ids < 0, 0.0, lse - mine), lse, z


def _gradients(x, w, ids, lse, z, c, frozen):
    g = (z - lse[:, None]).exp_()
    here = torch.arange(x.shape[0], device=x.device)
    g[here, ids.long().clamp(min=0)] -= 1.0
    g *= torch.where(ids < 0, 0.0, c)[:, None]
    dx = (g @ w.float()).to(x.dtype)
    return (dx,) if frozen else (dx, (g.t() @ x.float()).to(w.dtype))


def _plain(state):
    case = state["case"]
    kind, ids = case["kind"], state["ids"]
    if kind == "lookup":
        rows = state["table"][ids.long().clamp(min=0)].float() * case["factor"]
        return torch.where(ids[:, None] < 0, 0.0, rows).to(state["table"].dtype)
    if kind == "lookup_grad":
        dy, v = state["dy"], case["vocab"]
        sums = torch.zeros(v + 1, dy.shape[1], device="cuda")
        sums.index_add_(0, torch.where(ids < 0, v, ids).long(), dy.float())
        sums = sums[:v] * case["factor"]
        if case["base"]:
            sums += state["base"].float()
        return sums.to(dy.dtype)
    x, w = state["x"].detach(), state["w"].detach()
    loss, lse, z = _losses(x, w, ids)
    if kind == "loss":
        return loss, lse
    if kind == "grads":
        return _gradients(x, w, ids, state["lse"], z, state["c"], case["frozen"])
    count = (ids >= 0).sum().clamp(min=1).float()
    c = (1.0 / count).expand(x.shape[0])
    return (loss.sum() / count, *_gradients(x, w, ids, lse, z, c, False))


def run(state):
    if not own:
        return _plain(state)
    from lossless_bf16_tensor_gb300 import vocab
    case = state["case"]
    kind, ids = case["kind"], state["ids"]
    if kind == "lookup":
        return vocab.embedding(ids, state["table"], case["factor"])
    if kind == "lookup_grad":
        return vocab.embedding_grad(state["dy"], ids, case["vocab"], case["factor"], base=state.get("base"))
    x, w = state["x"], state["w"]
    if kind == "loss":
        return vocab.cross_entropy(x, w, ids)
    if kind == "grads":
        dx, dw = vocab.cross_entropy_grads(x, w, ids, state["loss"], state["lse"], state["c"],
                                           weight_grad=not case["frozen"])
        return (dx,) if case["frozen"] else (dx, dw)
    loss = vocab.linear_cross_entropy(x, w, ids)
    return (loss.detach(), *torch.autograd.grad(loss, (x, w)))


# ------------------------------------------------------------ work and exact

def work(case):
    t, v, k = case["tokens"], case["vocab"], case["cols"]
    ids = t * (8 if case["wide"] else 4)
    kind = case["kind"]
    if "factor" in case:
        size = 4 if case["dtype"] == "f32" else 2
        some = t * (1.0 - case["none"])
        if kind == "lookup":     # frequent rows are read again from the cache at best: each row that is there, once
            return {"bytes": size * k * (min(some, v) + t) + ids, "flops": t * k}
        return {"bytes": size * k * (some + v * (2 if case["base"] else 1)) + ids, "flops": 2 * some * k}
    one = 2 * t * v * k
    if kind == "loss":           # the logits
        return {"bytes": 2 * k * (t + v) + ids + 8 * t, "flops": one}
    some = 1.0 - case["none"]    # what has no target has no gradient
    outs = 2 * k * (t + (0 if case["frozen"] else v))
    if kind == "grads":          # the logits again, dx and dW
        return {"bytes": 2 * k * (t + v) + outs + ids + 12 * t, "flops": one * some * (2 if case["frozen"] else 3)}
    return {"bytes": 2 * k * (t + v) + outs + ids, "flops": one * some * 3}


def exact(case, seed):
    kind, v, k = case["kind"], case["vocab"], case["cols"]
    s = _row_tensors(case, seed) if "factor" in case else _loss_tensors(case, seed)
    ids = s["ids"].long()
    some = (ids >= 0).nonzero()[:, 0]
    if kind == "lookup":
        out = torch.zeros(case["tokens"], k, dtype=torch.float64, device="cuda")
        out[some] = s["table"].double()[ids[some]] * case["factor"]
        return out
    if kind == "lookup_grad":
        out = s["base"].double() if case["base"] else torch.zeros(v, k, dtype=torch.float64, device="cuda")
        return out.index_put_((ids[some],), s["dy"][some].double() * case["factor"], accumulate=True)
    x, w = s["x"].double(), s["w"].double()
    t = x.shape[0]
    loss, lse = torch.zeros(t, dtype=torch.float64, device="cuda"), torch.zeros(t, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    share = s["c"].double() if kind == "grads" else torch.full((t,), 1.0 / max(1, some.numel()), dtype=torch.float64,
                                                               device="cuda")
    rows = list(range(0, t, 1024)) if kind == "loss" else list(range(0, some.numel(), 1024))
    every = torch.arange(t, device="cuda") if kind == "loss" else some
    for first in rows:
        r = every[first:first + 1024]
        z = torch.mm(x[r], w.t())
        lse[r] = torch.logsumexp(z, 1)
        mine = torch.nn.functional.one_hot(ids[r].clamp(min=0), v).bool()
        loss[r] = torch.where(ids[r] < 0, 0.0, lse[r] - z[mine])
        if kind == "loss":
            continue
        p = torch.softmax(z, 1)
        g = torch.where(mine, torch.expm1(z - lse[r][:, None]), p) * share[r][:, None]
        dx[r] = torch.mm(g, w)
        if not case.get("frozen"):
            dw.addmm_(g.t(), x[r])
    if kind == "loss":
        return loss, lse
    if kind == "grads":
        return (dx,) if case["frozen"] else (dx, dw)
    return loss.sum() / max(1, some.numel()), dx, dw
