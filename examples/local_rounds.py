"""SparseLoCo rounds of a small language model, every stage by this library's operators.

Each peer takes local steps from the shared weights (embedding lookup, a hidden layer, token
log-probabilities and their gradients, the embedding table's gradient by sorted tokens, the
hidden matrix stepped by its orthogonalised momentum), compresses its pseudo-gradient (weights
before minus after, with error feedback), and all peers' records are averaged into the shared
weights.  A validator scores every peer's own update by what it does to the held-out loss.

The peers are emulated in turn on one GPU; the data are synthetic (a sparse random Markov chain).

    python examples/local_rounds.py [--rounds 4] [--peers 4] [--local-steps 8]
"""
from __future__ import annotations

import argparse
import json
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import compressed_pseudo_gradient_gb300 as spl  # noqa: E402

VOCAB, WIDTH, HIDDEN = 2000, 128, 256
BATCH = 1024


class Chain:
    """Token pairs of a Markov chain: each token has 4 likely successors."""

    def __init__(self, gen):
        self.gen = gen
        self.next = torch.randint(0, VOCAB, (VOCAB, 4), generator=gen, device=gen.device)

    def pairs(self, n=BATCH):
        at = torch.rand(n, generator=self.gen, device=self.gen.device).pow(2).mul(VOCAB).long()
        choice = torch.randint(0, 4, (n,), generator=self.gen, device=self.gen.device)
        return at, self.next[at, choice]


def new_weights(gen):
    dev = gen.device
    return {"table": torch.randn(VOCAB, WIDTH, generator=gen, device=dev) * 0.02,
            "hidden": torch.randn(HIDDEN, WIDTH, generator=gen, device=dev) / math.sqrt(WIDTH),
            "head": torch.randn(VOCAB, HIDDEN, generator=gen, device=dev) * 0.01}


def forward(w, tokens, targets):
    x = spl.embedding(tokens, w["table"], scale=math.sqrt(WIDTH))
    h = torch.tanh(x @ w["hidden"].t())
    logits = h @ w["head"].t()
    return x, h, logits, spl.token_logprobs(logits, targets)


def held_out_loss(w, tokens, targets):
    return -forward(w, tokens, targets)[3].logp.double().mean().item()


def local_step(w, state, tokens, targets, lr):
    """One local step in place: SGD on the two vocabulary-sized matrices, orthogonalised momentum
    on the hidden one."""
    x, h, logits, r = forward(w, tokens, targets)
    d_logp = torch.full((tokens.numel(),), -1.0 / tokens.numel(), device=x.device)
    d_logits = spl.token_logprobs_grad(logits, targets, r.lse, d_logp, out=logits)
    d_head = d_logits.t() @ h
    d_pre = (d_logits @ w["head"]).mul_(1 - h * h)
    d_table = spl.embedding_grad(tokens, d_pre @ w["hidden"], VOCAB, scale=math.sqrt(WIDTH))
    step = spl.orthogonalize(d_pre.t() @ x, momentum=state["momentum"], mu=0.9)
    w["hidden"].add_(step.float(), alpha=-0.1 * lr)
    w["head"].add_(d_head, alpha=-40.0 * lr)
    w["table"].add_(d_table, alpha=-1.0 * lr)


def run(rounds=4, peers=4, local_steps=8, lr=0.5, outer_lr=0.7, beta=0.95, seed=0, device="cuda:0",
        report=print):
    gen = torch.Generator(device=device).manual_seed(seed)
    chain = Chain(gen)
    shared = new_weights(gen)
    names = list(shared)
    held = chain.pairs(4 * BATCH)
    states = [{"momentum": torch.zeros_like(shared["hidden"]),
               "ef": [torch.zeros_like(shared[n]) for n in names]} for _ in range(peers)]
    chunks = [spl.num_chunks(shared[n].numel()) for n in names]
    losses = [held_out_loss(shared, *held)]
    for rnd in range(rounds):
        sent = []
        for st in states:
            w = {n: t.clone() for n, t in shared.items()}
            for _ in range(local_steps):
                local_step(w, st, *chain.pairs(), lr)
            deltas = [shared[n] - w[n] for n in names]
            sent.append(spl.ef_compress_multi(deltas, st["ef"], beta))
        scores, first = [], 0
        trial = [{n: t.clone() for n, t in shared.items()} for _ in sent]
        for n, c in zip(names, chunks):
            size = shared[n].numel()
            records = [(p[first:first + c], s[first:first + c]) for p, s in sent]
            for t, (p, s) in zip(trial, records):      # each peer's update alone, for its score
                spl.decode_aggregate([p], [s], size, theta=t[n].view(-1), lr=outer_lr)
            spl.decode_aggregate([p for p, _ in records], [s for _, s in records], size,
                                 theta=shared[n].view(-1), lr=outer_lr)
            first += c
        for t in trial:
            scores.append(losses[-1] - held_out_loss(t, *held))
        losses.append(held_out_loss(shared, *held))
        report(json.dumps({"round": rnd, "held_out_loss": round(losses[-1], 4),
                           "loss_scores": [round(s, 4) for s in scores]}))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=4)
    ap.add_argument("--peers", type=int, default=4)
    ap.add_argument("--local-steps", type=int, default=8)
    a = ap.parse_args()
    run(a.rounds, a.peers, a.local_steps)
