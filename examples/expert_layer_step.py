#!/usr/bin/env python3
"""A data-parallel training step of a small model with an expert layer on P
virtual ranks: libhc's operators make every rank's gradients, its collectives
make them one, and the clipping scales their mean.

Model (per rank, its own batch of tokens): embedding, norm, router, an expert
layer of two products an expert, the block boundary and an output product,
distilled from a teacher's top logits.

  x = embedding(ids)                              hc.embedding
  n = norm of x                                   hc.block_norm (residual 0)
  p = softmax of the router's top logits          torch
  rows of n by expert                             hc.expert_plan, hc.embedding
  h = max(rows W_up, 0); y = h W_down             hc.expert_matmul
  c = sum of p y over a token's experts           hc.expert_combine
  r, z = block boundary of (c, x)                 hc.block_norm
  logits = z W_out; loss, dlogits                 torch.matmul, hc.distill
  the same backwards                              hc.*_grad, torch.matmul
  sum of all gradients over the ranks             hc.allreduce (Ring, fused)
  their mean, clipped                             hc.clip_grads

  python examples/expert_layer_step.py [--ranks 4] [--steps 10]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import collective_communication_algorithms_gb300 as hc  # noqa: E402

VOCAB, DIM, HIDDEN, EXPERTS, CHOICES, TOP, PADDING = 500, 64, 96, 6, 2, 8, 0
SCALE = DIM ** 0.5


class Rank:
    """One rank's batch, parameters and gradient buffers (views of one flat
    vector, what the AllReduce works on)."""

    def __init__(self, rank, tokens):
        g = torch.Generator("cuda").manual_seed(100 + rank)
        p = torch.Generator("cuda").manual_seed(1)  # the same parameters on every rank
        shapes = {"table": (VOCAB, DIM), "router": (DIM, EXPERTS), "up": (EXPERTS, HIDDEN, DIM),
                  "down": (EXPERTS, DIM, HIDDEN), "out": (DIM, VOCAB), "norm": (DIM,), "post": (DIM,), "pre": (DIM,)}
        sizes = {k: (torch.Size(s).numel() + 3) // 4 * 4 for k, s in shapes.items()}
        self.grads_flat = torch.zeros(sum(sizes.values()), device="cuda")
        self.params, self.grads, at = {}, {}, 0
        for k, s in shapes.items():
            one = len(s) == 1
            self.params[k] = torch.ones(s, device="cuda") if one else torch.randn(s, generator=p, device="cuda") * s[-1] ** -0.5
            self.grads[k] = self.grads_flat[at:at + torch.Size(s).numel()].view(s)
            at += sizes[k]
        self.ids = torch.randint(0, VOCAB, (tokens,), generator=g, device="cuda")
        teach = torch.randn(VOCAB, VOCAB, generator=p, device="cuda") * 3
        top = teach[self.ids].topk(TOP, dim=1)
        self.teacher_logits, self.teacher_ids = top.values.contiguous(), top.indices.contiguous()
        self.row_weight = (self.ids != PADDING).float()

    def gradients(self, tokens_of_all_ranks):
        """Forward and backward; returns the rank's summed loss (a device scalar)."""
        q, gr = self.params, self.grads
        x = hc.embedding(q["table"], self.ids, scale=SCALE)["out"]
        first = hc.block_norm(x, x, post_weight=q["norm"], residual_scale=0.0, next_norm=False)
        n = first["r"]
        scores = n @ q["router"]
        chosen = scores.topk(CHOICES, dim=1)
        self.experts = chosen.indices
        p = torch.softmax(chosen.values, dim=1).contiguous()
        plan = hc.expert_plan(self.experts, EXPERTS)
        rows = hc.embedding(n, plan["tokens"])["out"]
        up = hc.expert_matmul(rows, q["up"], plan["offsets"])["out"]
        h = up.clamp(min=0)
        y = hc.expert_matmul(h, q["down"], plan["offsets"])["out"]
        c = hc.expert_combine(y, plan["slots"], weights=p)["out"]
        b = hc.block_norm(c, x, post_weight=q["post"], pre_weight=q["pre"])
        logits = b["z"] @ q["out"]
        d = hc.distill(logits, self.teacher_logits, self.teacher_ids, row_weight=self.row_weight, grad=logits,
                       temperature=2.0, scale=1.0 / tokens_of_all_ranks)  # in place
        # backwards
        torch.matmul(b["z"].t(), logits, out=gr["out"])
        dz = logits @ q["out"].t()
        bg = hc.block_norm_grad(None, dz, c, x, b["post_rstd"], b["pre_rstd"], post_weight=q["post"],
                                pre_weight=q["pre"], grad_post_weight=gr["post"], grad_pre_weight=gr["pre"])
        cg = hc.expert_combine_grad(bg["grad_y"], plan["slots"], y=y, weights=p)
        dh = hc.expert_matmul_grad(cg["grad_y"], plan["offsets"], x=h, weight=q["down"], grad_weight=gr["down"])["grad_x"]
        drows = hc.expert_matmul_grad(torch.where(up > 0, dh, 0.0), plan["offsets"], x=rows, weight=q["up"],
                                      grad_weight=gr["up"])["grad_x"]
        dn = hc.expert_combine(drows, plan["slots"])["out"]  # the gradient of the gather
        gp = cg["grad_weights"]
        dscores = torch.zeros_like(scores).scatter_(1, self.experts, p * (gp - (p * gp).sum(dim=1, keepdim=True)))
        torch.matmul(n.t(), dscores, out=gr["router"])
        dn.addmm_(dscores, q["router"].t())
        fg = hc.block_norm_grad(dn, None, x, x, first["post_rstd"], None, post_weight=q["norm"],
                                grad_post_weight=gr["norm"], residual_scale=0.0)
        dx = bg["grad_x"] + fg["grad_y"]
        hc.embedding_grad(dx, self.ids, gr["table"], scale=SCALE, padding_id=PADDING)
        return d["loss"].sum()

    def update(self, rate):
        for k, v in self.params.items():
            v.sub_(self.grads[k], alpha=rate)


def step(ranks, tokens_of_all_ranks, max_norm, rate):
    """One step of all ranks; returns (loss, the gradients' norm before clipping)."""
    loss = sum(r.gradients(tokens_of_all_ranks) for r in ranks)
    hc.allreduce([r.grads_flat for r in ranks])  # in place
    norms = [hc.clip_grads(list(r.grads.values()), max_norm)["norm"] for r in ranks]
    for r in ranks:
        r.update(rate)
    return loss, norms[0]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    tokens = 256
    ranks = [Rank(r, tokens) for r in range(a.ranks)]
    for i in range(a.steps):
        loss, norm = step(ranks, a.ranks * tokens, max_norm=1.0, rate=0.5)
        print("step %2d  loss %.5f  gradient norm %.4f" % (i, float(loss), float(norm)))


if __name__ == "__main__":
    main()
