"""A tied-weight language model trained over logical ranks: the operators
between two gradient syncs.

    ids -> embedding -> RMS norm (input kept in 8 bits) -> output layer + loss
    loss -> output layer's gradients -> norm's -> embedding's, onto the same
    weight's gradient -> all ranks' mean, clipping and AdamW

The model predicts the next token from the current one.  Its tokens follow a
fixed random successor table most of the time, so the loss has a known bottom.

    python examples/tied_lm.py [--steps 60] [--ranks 4]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gradient_sync_rcc_gb300 import rcc  # noqa: E402

DEV = "cuda:0"


class TiedLM:
    """Master weights in fp32; the output layer reads a bf16 copy."""

    def __init__(self, vocab, dim, tokens, ranks, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.vocab, self.dim, self.tokens, self.ranks = vocab, dim, tokens, ranks
        self.table = torch.randn(vocab, dim, generator=g, device=DEV) / math.sqrt(dim)
        self.norm = torch.ones(dim, device=DEV)
        # each rank's gradients, and the optimizer's state (held here: ParamSets
        # keeps addresses alone)
        self.dtable = [torch.empty_like(self.table) for _ in range(ranks)]
        self.dnorm = [torch.empty_like(self.norm) for _ in range(ranks)]
        self.tensors = [
            dict(grads=grads, params=[p], exp_avg=[torch.zeros_like(p)],
                 exp_avg_sq=[torch.zeros_like(p)])
            for p, grads in ((self.table, self.dtable), (self.norm, self.dnorm))]
        self.sets = rcc.ParamSets(self.tensors)
        # scratch that every micro-batch uses again
        need = max(rcc.linear_ce_workspace(tokens, vocab, dim),
                   rcc.linear_ce_workspace(tokens, vocab, dim, True, torch.float32),
                   rcc.embedding_backward_workspace(tokens, vocab, dim),
                   rcc.rmsnorm_backward_workspace(tokens, dim))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=DEV)
        self.kept = rcc.Kept(tokens, dim, DEV)

    def forward_backward(self, rank, ids, labels, w16, loss_scale):
        """One rank's micro-batch: its loss for each token, and its gradients."""
        ws, scale = self.workspace, math.sqrt(self.dim)
        counted = (labels >= 0).float()
        h = rcc.embedding_forward(self.table, ids, scale=scale, out_dtype=torch.bfloat16)
        y, kept = rcc.rmsnorm_forward(h, self.norm, keep=self.kept)
        loss, lse = rcc.linear_ce_forward(y, w16, labels, workspace=ws)
        dloss = counted * (loss_scale / counted.sum().clamp_min(1))
        dy, _ = rcc.linear_ce_backward(y, w16, labels, lse, dloss, dw=self.dtable[rank],
                                       workspace=ws)
        dh, _ = rcc.rmsnorm_backward(dy, kept, self.norm, dweight=self.dnorm[rank], workspace=ws)
        rcc.embedding_backward(dh, ids, self.dtable[rank], scale=scale, accumulate=True,
                               workspace=ws)
        return loss, counted

    def step(self, comm, batches, cfg, state):
        """A training step over all ranks' (ids, labels); the mean loss, the report."""
        w16 = self.table.to(torch.bfloat16)
        total = torch.zeros((), device=DEV)
        count = torch.zeros((), device=DEV)
        for r, (ids, labels) in enumerate(batches):
            loss, counted = self.forward_backward(r, ids, labels, w16, state.scale)
            total += loss.sum()
            count += counted.sum()
        report = rcc.grad_sync_adamw(comm, self.sets, cfg, state)
        return float(total / count), report


def batch(g, follow, vocab, tokens, noise=0.1):
    """Tokens whose successor is follow[token], but for a share of `noise`;
    some positions are padding, which neither embeds nor counts."""
    ids = torch.randint(vocab, (tokens,), generator=g, device=DEV)
    labels = follow[ids]
    stray = torch.rand(tokens, generator=g, device=DEV) < noise
    labels = torch.where(stray, torch.randint(vocab, (tokens,), generator=g, device=DEV), labels)
    padding = torch.rand(tokens, generator=g, device=DEV) < 0.05
    return torch.where(padding, -1, ids), torch.where(padding, -1, labels)


def train(steps=60, ranks=4, vocab=1000, dim=128, tokens=1024, lr=1e-2, seed=1, say=print):
    """Trains; returns the loss of each step and the final optimizer state."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    follow = torch.randperm(vocab, generator=g, device=DEV)
    model = TiedLM(vocab, dim, tokens, ranks)
    cfg = rcc.adamw_cfg(lr=lr, weight_decay=0.0, max_grad_norm=1.0)
    state = rcc.optim_state(scale=1024.0)
    comm = rcc.register(device=0, num_ranks=ranks, dtype=rcc.F32)
    losses = []
    try:
        for i in range(steps):
            loss, report = model.step(comm, [batch(g, follow, vocab, tokens)
                                             for _ in range(ranks)], cfg, state)
            losses.append(loss)
            if i % 10 == 0 or i == steps - 1:
                say("step %3d  loss %.3f  gradient norm %.3f  skipped %d"
                    % (i, loss, report.grad_norm, report.skipped))
    finally:
        rcc.finish(comm)
    return losses, state


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    train(a.steps, a.ranks)
