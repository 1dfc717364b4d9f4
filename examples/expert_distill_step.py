"""Data-parallel training of a small routed model against a teacher's top
logits, on p simulated ranks of one GPU.

Every rank holds its own tokens and a copy of the weights.  A step is

  route            gate of the rank's tokens: chosen experts, combine weights,
                   per-expert counts and probability sums
  allreduce        counts (int32) and probability sums (fp32) over the ranks
  distill_step     loss and gradient of the rank's student logits
  (or, with --shards: the ranks hold vocabulary shards of the student head,
   distill_parts, all_gather, distill_join, distill_grad)
  route_grad       balance loss, gradient of the gate's logits
  allreduce        weight gradients over the ranks

so that every rank ends with the same weights.  Run it as
  python examples/expert_distill_step.py [--ranks 4] [--steps 20] [--shards]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_reduce_reduction_amd as sim  # noqa: E402

HIDDEN, EXPERTS, TOPK, VOCAB, TEACHER_TOPK = 64, 16, 4, 1000, 8
TEMPERATURE, BALANCE = 2.0, 0.02


def make_weights(seed: int, device):
    """Gate, one output vector per expert, student head."""
    g = torch.Generator().manual_seed(seed)
    return {"gate": (0.3 * torch.randn(HIDDEN, EXPERTS, generator=g)).to(device),
            "experts": (0.3 * torch.randn(EXPERTS, HIDDEN, generator=g)).to(device),
            "head": (0.2 * torch.randn(HIDDEN, VOCAB, generator=g)).to(device)}


def make_batch(rank: int, tokens: int, device):
    """A rank's tokens, which of them count, and their teacher's top logits."""
    g = torch.Generator().manual_seed(1000 + rank)
    x = torch.randn(tokens, HIDDEN, generator=g)
    keep = torch.rand(tokens, generator=g) < 0.9  # the rest is padding
    truth = torch.randn(HIDDEN, VOCAB, generator=torch.Generator().manual_seed(7))
    top = (x @ truth).topk(TEACHER_TOPK, dim=1)
    ids = torch.where(keep[:, None], top.indices.int(), -1)
    return {"x": x.to(device), "keep": keep.to(device), "ids": ids.to(device), "teacher": top.values.to(device)}


def whole_rows(w, y, batch, scale):
    """Student logits of all of a rank's rows: loss of each row, gradients of the head and of y."""
    loss, d = sim.distill_step(y @ w["head"], batch["ids"], batch["teacher"], temperature=TEMPERATURE,
                               row_scale=batch["keep"].float(), coef=scale)
    return loss, y.t() @ d, d @ w["head"].t()


def vocabulary_shards(w, y, batch, scale, p):
    """The same with the head's columns cut into p shards (16-byte aligned statistics, any shard width)."""
    cut = [r * VOCAB // p for r in range(p + 1)]
    heads = [w["head"][:, a:b] for a, b in zip(cut, cut[1:])]
    logits = [y @ h for h in heads]
    kw = dict(temperature=TEMPERATURE, vocab=VOCAB)
    ids, teacher = batch["ids"], batch["teacher"]
    parts = [sim.distill_parts(z, ids, teacher, first=a, **kw) for z, a in zip(logits, cut)]
    gathered = [torch.empty((p,) + parts[0].shape, device=y.device) for _ in range(p)]
    sim.all_gather(parts, gathered)
    grads, loss = [], None
    for r in range(p):  # every shard's owner joins for itself
        loss, norm = sim.distill_join(gathered[r], ids, teacher, **kw)
        grads.append(sim.distill_grad(logits[r], ids, teacher, norm, row_scale=batch["keep"].float(), coef=scale,
                                      first=cut[r], out=logits[r], **kw))
    return loss, torch.cat([y.t() @ d for d in grads], 1), sum(d @ h.t() for d, h in zip(grads, heads))


def gradients(weights, batches, shards: bool):
    """One forward and backward pass over all ranks: (distillation loss, balance loss, gradients of each rank, the
    same on all of them)."""
    p = len(batches)
    gate = [b["x"] @ w["gate"] for w, b in zip(weights, batches)]
    routed = [sim.route(z, TOPK, keep=b["keep"]) for z, b in zip(gate, batches)]
    counts = sim.allreduce([r[2] for r in routed])  # in place: what every rank's tokens chose together
    sums = sim.allreduce([r[3] for r in routed])
    rows = sim.allreduce([b["keep"].sum().float().reshape(1) for b in batches])  # tokens that count
    grads, losses, balance = [], [], None
    for r, (w, b) in enumerate(zip(weights, batches)):
        chosen, mix = routed[r][:2]
        at = chosen.clamp(min=0).long()
        y = b["x"] + (mix[:, :, None] * w["experts"][at]).sum(1)
        scale = 1.0 / float(rows[r])
        loss, dhead, dy = vocabulary_shards(w, y, b, scale, p) if shards else whole_rows(w, y, b, scale)
        dmix = (dy[:, None, :] * w["experts"][at]).sum(2)
        balance, dgate = sim.route_grad(gate[r], chosen, dmix, counts[r], sums[r], BALANCE, keep=b["keep"])
        dexperts = torch.zeros_like(w["experts"]).index_add_(0, at.reshape(-1),
                                                             (mix[:, :, None] * dy[:, None, :]).reshape(-1, HIDDEN))
        grads.append({"gate": b["x"].t() @ dgate, "experts": dexperts, "head": dhead})
        losses.append(loss.sum().reshape(1) * scale)
    for name in grads[0]:
        for g, total in zip(grads, sim.allreduce([g[name].contiguous() for g in grads])):
            g[name] = total
    return sim.allreduce(losses)[0], balance, grads


def train(ranks: int = 4, tokens: int = 256, steps: int = 20, rate: float = 0.5, shards: bool = False, log=print):
    device = torch.device("cuda:0")
    sim.sim_init(0)
    weights = [make_weights(0, device) for _ in range(ranks)]
    batches = [make_batch(r, tokens, device) for r in range(ranks)]
    history = []
    for step in range(steps):
        loss, balance, grads = gradients(weights, batches, shards)
        for w, g in zip(weights, grads):
            for name in w:
                w[name] -= rate * g[name]
        history.append((float(loss), float(balance)))
        log(f"step {step:3d}: distillation loss {history[-1][0]:.4f}, balance loss {history[-1][1]:.5f}")
    return history, weights


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=256, help="per rank")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--shards", action="store_true", help="cut the vocabulary into one shard per rank")
    a = ap.parse_args()
    train(a.ranks, a.tokens, a.steps, shards=a.shards)


if __name__ == "__main__":
    main()
