#!/usr/bin/env python3
"""A data-parallel training step of a small student model on P virtual ranks:
the training operators of libhc make every rank's gradients, its collectives
make them one.

Model (per rank, its own batch of tokens): embedding, one block (a product, its
norm, gate and scaled residual, the next norm) and an output product, distilled
from a teacher's top logits.

  x = embedding(ids)                        hc.embedding
  y = x W1                                  torch.matmul
  r, z = block boundary of (y, x)           hc.block_norm
  logits = z W2                             torch.matmul
  loss, dlogits                             hc.distill
  dz, dW2; then dy, dx and the weights'     torch.matmul, hc.block_norm_grad
  dW1, dx; then the table's                 torch.matmul, hc.embedding_grad
  sum of all gradients over the ranks       hc.allreduce (Ring, fused)

The vocabulary-parallel form of the lookup is there too: every rank holds a
part of the table's rows, and a sum AllReduce of the ranks' lookups is the
whole one.

  python examples/data_parallel_step.py [--ranks 4] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import collective_communication_algorithms_gb300 as hc  # noqa: E402

VOCAB, DIM, TOP, PADDING = 1000, 256, 8, 0


class Rank:
    """One rank's batch, parameters, gradient buffers (views of one flat
    vector, what the AllReduce works on) and bound calls."""

    def __init__(self, rank, tokens, dtype=torch.float32):
        g = torch.Generator("cuda").manual_seed(100 + rank)
        p = torch.Generator("cuda").manual_seed(1)  # the same parameters on every rank
        shapes = {"table": (VOCAB, DIM), "w1": (DIM, DIM), "w2": (DIM, VOCAB), "post_weight": (DIM,),
                  "gate": (1, DIM), "pre_weight": (DIM,)}
        sizes = {k: (int(torch.Size(s).numel()) + 3) // 4 * 4 for k, s in shapes.items()}
        self.grads_flat = torch.zeros(sum(sizes.values()), device="cuda")
        self.params, self.grads, at = {}, {}, 0
        for k, s in shapes.items():
            one = k in ("post_weight", "pre_weight", "gate")
            self.params[k] = torch.ones(s, device="cuda") if one else torch.randn(s, generator=p, device="cuda") * DIM ** -0.5
            self.grads[k] = self.grads_flat[at:at + torch.Size(s).numel()].view(s)
            at += sizes[k]
        self.ids = torch.randint(0, VOCAB, (tokens,), generator=g, device="cuda")
        # a teacher that only looks at the token: the same for all ranks
        teach = torch.randn(VOCAB, VOCAB, generator=p, device="cuda") * 3
        top = teach[self.ids].topk(TOP, dim=1)
        self.teacher_logits, self.teacher_ids = top.values.contiguous(), top.indices.contiguous()
        self.row_weight = (self.ids != PADDING).float()

    def bind(self, tokens_of_all_ranks):
        q, gr = self.params, self.grads
        self.embed = hc.bind_embedding(q["table"], self.ids, scale=DIM ** 0.5)
        self.x = self.embed.outputs["out"]
        self.y = torch.empty_like(self.x)
        self.norm = hc.bind_block_norm(self.y, self.x, q["post_weight"], q["gate"], q["pre_weight"])
        f = self.norm.outputs
        self.logits = torch.empty(self.ids.numel(), VOCAB, device="cuda")
        self.loss = hc.bind_distill(self.logits, self.teacher_logits, self.teacher_ids, self.row_weight,
                                    grad=self.logits, temperature=2.0, scale=1.0 / tokens_of_all_ranks)  # in place
        self.dz = torch.empty_like(self.x)
        self.norm_grad = hc.bind_block_norm_grad(None, self.dz, self.y, self.x, f["post_rstd"], f["pre_rstd"],
                                                 q["post_weight"], q["gate"], q["pre_weight"],
                                                 grad_post_weight=gr["post_weight"], grad_gate=gr["gate"],
                                                 grad_pre_weight=gr["pre_weight"])
        self.dx = self.norm_grad.outputs["grad_x"]
        self.embed_grad = hc.bind_embedding_grad(self.dx, self.ids, gr["table"], scale=DIM ** 0.5, padding_id=PADDING)

    def gradients(self):
        """Forward and backward; returns the rank's summed loss (a device scalar)."""
        q, gr, f = self.params, self.grads, self.norm.outputs
        self.embed()
        torch.matmul(self.x, q["w1"], out=self.y)
        self.norm()
        torch.matmul(f["z"], q["w2"], out=self.logits)
        self.loss()  # self.logits now holds their gradient
        torch.matmul(self.logits, q["w2"].t(), out=self.dz)
        torch.matmul(f["z"].t(), self.logits, out=gr["w2"])
        self.norm_grad()
        dy = self.norm_grad.outputs["grad_y"]
        torch.matmul(self.x.t(), dy, out=gr["w1"])
        self.dx.addmm_(dy, q["w1"].t())
        self.embed_grad()
        return self.loss.outputs["loss"].sum()

    def update(self, rate):
        for k, v in self.params.items():
            v.sub_(self.grads[k], alpha=rate)


def vocabulary_parallel_lookup(table, ids, P):
    """The lookup with the table's rows split over P ranks."""
    per = (table.shape[0] + P - 1) // P
    parts = [hc.embedding(table[r * per:(r + 1) * per], ids, scale=DIM ** 0.5, first_id=r * per)["out"] for r in range(P)]
    return hc.allreduce(parts)


def run(P=4, steps=20, tokens=512, rate=0.5):
    """Returns the losses of all steps and the ranks."""
    ranks = [Rank(r, tokens) for r in range(P)]
    for r in ranks:
        r.bind(P * tokens)
    losses = []
    for _ in range(steps):
        losses.append(sum(r.gradients() for r in ranks))
        hc.allreduce([r.grads_flat for r in ranks])  # in place
        for r in ranks:
            r.update(rate)
    return [float(v) for v in losses], ranks


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, ranks = run(a.ranks, a.steps)
    for i, v in enumerate(losses):
        print("step %2d  loss %.5f" % (i, v))
    whole = hc.embedding(ranks[0].params["table"], ranks[0].ids, scale=DIM ** 0.5)["out"]
    split = vocabulary_parallel_lookup(ranks[0].params["table"], ranks[0].ids, a.ranks)
    print("vocabulary split over %d ranks: %s" % (a.ranks, "the same lookup" if all(torch.equal(whole, s) for s in split)
                                                   else "DIFFERENT"))


if __name__ == "__main__":
    main()
