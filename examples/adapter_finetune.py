"""Train two adapters at once on a frozen, losslessly compressed projection, then
serve them token by token.

    python examples/adapter_finetune.py [--steps 30]

One step: the projection and the adapters' part in one call (each token with its
own adapter), what autograd saves kept compressed, the adapters' gradients
clipped by their global norm, and the fused AdamW step on the adapters'
compressed weights and moments.  The data is synthetic: each task's target is
the projection with a low-rank change of its own.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_bf16_tensor_gb300 import binding as B  # noqa: E402
from lossless_bf16_tensor_gb300.activations import compressed_activations  # noqa: E402
from lossless_bf16_tensor_gb300.adapters import AdapterBank, adapter_linear, adapter_plan  # noqa: E402
from lossless_bf16_tensor_gb300.grads import clip_grads  # noqa: E402

BF16 = torch.bfloat16


def compress(x: torch.Tensor, cb, level="CLEAN") -> B.CompressedTensor:
    t = B.CompressedTensor(x.numel(), level)
    B.lct_encode(x.contiguous().view(torch.int16).view(-1), cb, t)
    return t


class CompressedAdamW:
    """AdamW on one parameter whose weights and moments stay compressed; the
    parameter itself holds the decoded weights for the next forward pass."""

    def __init__(self, p: torch.Tensor, scale: float):
        self.p = p
        # moments start at zero and have no scale yet: their codebooks put zeros first
        self.books = [B.lct_codebook_build("gaussian", scale)] + \
                     [B.lct_codebook_build_zero_atom("laplace", s, 0.0, 0.1) for s in (1e-4, 1e-8)]
        start = (p.data, torch.zeros_like(p), torch.zeros_like(p))
        self.state = [compress(v, cb, "HIGH") for v, cb in zip(start, self.books)]

    def step(self, lr: float, t: int) -> None:
        new = [B.CompressedTensor(s.n, "HIGH") for s in self.state]
        (w, m, v), (cw, cm, cv) = self.state, self.books
        B.lct_adamw_step_fused(w, cw, m, cm, v, cv, self.p.grad.view(torch.int16).view(-1), lr, 0.9, 0.99, 1e-8, 0.0, t,
                               *new)
        self.state = new
        B.lct_decode(new[0], cw, self.p.data.view(torch.int16).view(-1))


def main(steps: int = 30, k: int = 512, n: int = 1024, rank: int = 16, tokens: int = 1024) -> list[float]:
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    # the frozen projection, compressed; nothing keeps it dense
    dense = normal(n, k, scale=0.02).to(BF16)
    cb = B.lct_codebook_build("gaussian", 0.02)
    w = compress(dense, cb)
    print("projection: %d values, %.3fx compressed" % (w.n, w.compression_ratio()))

    tasks = 2
    targets = [dense.float() + normal(n, 4, scale=0.05) @ normal(4, k, scale=0.05) for _ in range(tasks)]
    a = torch.nn.Parameter(normal(tasks, rank, k, scale=1 / math.sqrt(k)).to(BF16))
    b = torch.nn.Parameter(torch.zeros(tasks, n, rank, device="cuda", dtype=BF16))
    bank = AdapterBank(a, b, torch.full((tasks,), 2.0, device="cuda"))
    optimizers = [CompressedAdamW(a, 1 / math.sqrt(k)), CompressedAdamW(b, 0.02)]
    saved = compressed_activations(B.lct_codebook_build("gaussian", 1.0))

    losses = []
    for step in range(1, steps + 1):
        # a batch of both tasks' sequences, and a few tokens that no adapter changes
        index = torch.arange(tokens, device="cuda", dtype=torch.int32) * (tasks + 1) // tokens
        index = torch.where(index == tasks, -1, index)
        x = normal(tokens, k).to(BF16)
        want = torch.stack([x.float() @ t.t() for t in targets] + [x.float() @ dense.float().t()])
        want = want[index.long(), torch.arange(tokens, device="cuda")]
        plan = adapter_plan(index, bank.adapters)
        with saved:
            y = adapter_linear(x, w, cb, bank, plan)
            loss = (y.float() - want).square().mean()
        a.grad = b.grad = None
        loss.backward()
        norm = clip_grads([a.grad, b.grad], max_norm=0.003)
        for o in optimizers:
            o.step(3e-3, step)
        losses.append(loss.item())
        if step % 5 == 0 or step == 1:
            print("step %2d  loss %.5f  gradient norm %.4f" % (step, losses[-1], norm.item()))
    saved.flush()
    print("saved tensors: %(compressed)d compressed, %(fallback)d not" % saved.stats)

    # serving: single tokens of three requests, each with its own adapter or none
    index = torch.tensor([1, -1, 0], device="cuda", dtype=torch.int32)
    x = normal(3, k).to(BF16)
    with torch.no_grad():
        y = adapter_linear(x, w, cb, bank, adapter_plan(index, tasks)).float()
    for i, (got, task) in enumerate(zip(y, index.tolist())):
        ref = x[i].float() @ (targets[task] if task >= 0 else dense.float()).t()
        print("request %d (adapter %2d): off the target by %.4f, of %.4f" % (i, task, (got - ref).std(), ref.std()))
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=30)
    main(parser.parse_args().steps)
