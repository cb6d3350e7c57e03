"""A small decoder trained for a step with the operators together: embedding,
residual RMS norms, rotary positions, output layer, gradients of two ranks brought
together, and AdamW with 8-bit states whose copies are the next step's weights.

Its matrix products, attention and activation are torch's.  Against automatic
differentiation of the same model in 64 bits.
"""
import math
import os
import re

import pytest
import torch

import test_gpu_adamw as adam
import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV, session

pytestmark = pytest.mark.gpu

U, F32, BF16, E4M3 = defs.U, defs.F32, defs.BF16, torch.float8_e4m3fn
VOCAB, DIM, HEADS, KEYS, LAYERS, EPS = 300, 128, 4, 2, 2, 1e-6
HEAD = DIM // HEADS


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids):
        ctx.ids, ctx.shape = ids, table.shape
        return rcc.embedding_forward(table, ids, scale=math.sqrt(DIM))

    @staticmethod
    def backward(ctx, dout):
        return rcc.embedding_backward(dout.contiguous(), ctx.ids,
                                      torch.empty(ctx.shape, device=DEV),
                                      scale=math.sqrt(DIM)), None


class Norm(torch.autograd.Function):
    """(y, h) of h = x + residual, or of x alone."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        ctx.weight, ctx.added = weight, residual is not None
        if residual is None:
            y, ctx.kept = rcc.rmsnorm_forward(x, weight, keep=True)
            return y, x.clone()
        y, h, ctx.kept = rcc.add_rmsnorm_forward(x, residual, weight, keep=True)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        dx, dw = rcc.add_rmsnorm_backward(dy.contiguous(), dh.contiguous(), ctx.kept, ctx.weight)
        return dx, dx if ctx.added else None, dw


class Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, turns, positions):
        ctx.turns, ctx.positions = turns, positions
        return rcc.rotary_forward(q, k, turns, positions)

    @staticmethod
    def backward(ctx, dq, dk):
        return *rcc.rotary_backward(dq.contiguous(), dk.contiguous(), ctx.turns,
                                    ctx.positions), None, None


class Loss(torch.autograd.Function):
    """The mean of the counted tokens' losses."""

    @staticmethod
    def forward(ctx, x, table, w16, labels):
        ctx.x16, ctx.w16, ctx.labels = x.to(BF16), w16, labels
        loss, ctx.lse = rcc.linear_ce_forward(ctx.x16, w16, labels)
        ctx.share = (labels >= 0).float() / (labels >= 0).sum()
        return (loss * ctx.share).sum()

    @staticmethod
    def backward(ctx, d):
        dx, dw = rcc.linear_ce_backward(ctx.x16, ctx.w16, ctx.labels, ctx.lse,
                                        ctx.share * d, grad_dtype=F32)
        return dx, dw, None, None


def weights(g):
    w = {"table": defs.randn(g, VOCAB, DIM, scale=1 / math.sqrt(DIM)),
         "norm0": 1.0 + defs.randn(g, DIM, scale=0.1)}
    for i in range(LAYERS):
        w["qkv%d" % i] = defs.randn(g, DIM, (HEADS + 2 * KEYS) * HEAD, scale=1 / math.sqrt(DIM))
        w["out%d" % i] = defs.randn(g, DIM, DIM, scale=1 / math.sqrt(DIM))
        w["up%d" % i] = defs.randn(g, DIM, 2 * DIM, scale=1 / math.sqrt(DIM))
        w["down%d" % i] = defs.randn(g, 2 * DIM, DIM, scale=1 / math.sqrt(2 * DIM))
        w["norma%d" % i], w["normb%d" % i] = (1.0 + defs.randn(g, DIM, scale=0.1)
                                              for _ in range(2))
    return w


def forward(w, ids, labels, positions, mask, embed, norm, rotary, loss):
    y, h = norm(embed(w["table"], ids), None, w["norm0"])
    for i in range(LAYERS):
        q, k, v = (y @ w["qkv%d" % i]).unflatten(1, (-1, HEAD)).split((HEADS, KEYS, KEYS), 1)
        q, k = rotary(q, k)
        k, v = (t.repeat_interleave(HEADS // KEYS, 1) for t in (k, v))
        s = torch.einsum("thd,shd->hts", q, k) / math.sqrt(HEAD)
        p = torch.softmax(s.masked_fill(~mask, -math.inf), 2)
        o = torch.einsum("hts,shd->thd", p, v).flatten(1)
        y, h = norm(o @ w["out%d" % i], h, w["norma%d" % i])
        y, h = norm(torch.tanh(y @ w["up%d" % i]) @ w["down%d" % i], h, w["normb%d" % i])
    return loss(y, w["table"], labels)


def with_operators(w, w16, turns, ids, labels, positions, mask):
    return forward(w, ids, labels, positions, mask, Embed.apply, Norm.apply,
                   lambda q, k: Rotary.apply(q, k, turns, positions),
                   lambda y, table, labels: Loss.apply(y, table, w16, labels))


def in_64_bits(w, ids, labels, positions, mask):
    f = 10000.0 ** (-torch.arange(0, HEAD, 2, device=DEV).double() / HEAD)
    angle = positions.double()[:, None, None] * f
    c, s = torch.cos(angle), torch.sin(angle)

    def turn(x):
        a, b = x[:, :, :HEAD // 2], x[:, :, HEAD // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], 2)

    def norm(x, residual, weight):
        h = x if residual is None else x + residual
        return h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * weight, h

    def loss(y, table, labels):
        each = torch.nn.functional.cross_entropy(y @ table.t(), labels, ignore_index=-1)
        return each
    return forward(w, ids, labels, positions, mask,
                   lambda table, ids: torch.where((ids >= 0)[:, None],
                                                  table[ids.clamp_min(0)] * math.sqrt(DIM), 0.0),
                   norm, lambda q, k: (turn(q), turn(k)), loss)


def batch(g, lengths):
    """Documents one behind the other, some positions padding."""
    tokens = sum(lengths)
    ids = torch.randint(VOCAB, (tokens,), generator=g, device=DEV)
    labels = torch.randint(VOCAB, (tokens,), generator=g, device=DEV)
    doc = torch.repeat_interleave(torch.arange(len(lengths), device=DEV),
                                  torch.tensor(lengths, device=DEV))
    positions = torch.cat([torch.arange(n, device=DEV) for n in lengths])
    padding = torch.rand(tokens, generator=g, device=DEV) < 0.05
    at = torch.arange(tokens, device=DEV)
    mask = (doc[:, None] == doc) & (at[:, None] >= at)
    return (torch.where(padding, -1, ids), torch.where(padding, -1, labels), positions, mask)


def test_two_ranks_and_a_step_of_adamw():
    """Five norms read their inputs in 8 bits in the backward pass, 1/254 of a
    group's largest value off at most, in random directions; a value's size is a
    third to a quarter of that, so each perturbs the gradients that pass it by
    less than 1%, and the output layer's bf16 by less than 1% again."""
    g = defs.gen(101)
    w = {k: v.requires_grad_() for k, v in weights(g).items()}
    w16 = w["table"].detach().to(BF16)
    turns = rcc.rotary_turns(HEAD, device=DEV)
    batches = [batch(g, (40, 1, 90)), batch(g, (131,))]
    grads, exact = [], []
    for b in batches:
        loss = with_operators(w, w16, turns, *b)
        grads.append(dict(zip(w, torch.autograd.grad(loss, list(w.values())))))
        w64 = {k: v.detach().double().requires_grad_() for k, v in w.items()}
        want = in_64_bits(w64, *b)
        exact.append(dict(zip(w64, torch.autograd.grad(want, list(w64.values())))))
        assert abs(float(loss.detach()) - float(want.detach())) < 0.01 * float(want.detach())
        for k in w:
            off = float((grads[-1][k].double() - exact[-1][k]).norm() / exact[-1][k].norm())
            assert off < 0.06, (k, off)
    mean = {k: torch.empty_like(v) for k, v in w.items()}
    with session(2) as comm:
        for k in w:
            rcc.reduce(comm, [r[k] for r in grads], mean[k], 0, "mean")
        torch.cuda.synchronize()
    param = {k: v.detach() for k, v in w.items()}
    tensors = [dict(param=param[k], grad=mean[k]) | (dict(copy=w16) if k == "table" else {})
               for k in w]
    plan = rcc.AdamWPlan(tensors, states=E4M3, seed=11)
    flat = [{k: v.view(-1) for k, v in t.items()} for t in plan.tensors]
    before = adam.clone(flat)
    rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=1.0, **adam.CFG))
    r = rcc.adamw_report(plan)
    norm = math.sqrt(sum(float(v.double().square().sum()) for v in mean.values()))
    assert r.skipped == 0 and abs(r.grad_norm - norm) <= 1e-12 * norm
    now = adam.Powers(adam.CFG["betas"], 0).next()
    adam.same(flat, [adam.expected(t, i, adam.CFG, 1.0, 0, 11, r.clip_coef, now)
                     for i, t in enumerate(before)])
    assert torch.equal(w16, param["table"].to(BF16))
    # the next step's forward pass, on the new weights and their copy
    loss = with_operators(w, w16, turns, *batches[0])
    want = in_64_bits({k: v.double() for k, v in param.items()}, *batches[0])
    assert abs(float(loss.detach()) - float(want)) < 0.01 * float(want)


def test_one_token_at_a_time():
    """Decoding: the rows of a prompt one by one give what they give together."""
    g = defs.gen(102)
    q, k = defs.randn(g, 9, HEADS, HEAD, dtype=BF16), defs.randn(g, 9, KEYS, HEAD, dtype=BF16)
    x, r = defs.randn(g, 9, DIM, dtype=BF16), defs.randn(g, 9, DIM, dtype=BF16)
    weight = 1.0 + defs.randn(g, DIM, scale=0.1)
    turns = rcc.rotary_turns(HEAD, scaling=("parts", 8.0, 64, 1.0, 4.0), device=DEV)
    q2, k2 = rcc.rotary_forward(q, k, turns, offset=1000)
    y, h = rcc.add_rmsnorm_forward(x, r, weight)
    y8, _ = rcc.add_rmsnorm_forward(x, r, weight, out_dtype=E4M3)
    for i in range(9):
        a, b = rcc.rotary_forward(q[i:i + 1], k[i:i + 1], turns, offset=1000 + i)
        assert torch.equal(a, q2[i:i + 1]) and torch.equal(b, k2[i:i + 1])
        yi, hi = rcc.add_rmsnorm_forward(x[i:i + 1], r[i:i + 1], weight)
        assert torch.equal(yi, y[i:i + 1]) and torch.equal(hi, h[i:i + 1])
        ei, _ = rcc.add_rmsnorm_forward(x[i:i + 1], r[i:i + 1], weight, out_dtype=E4M3)
        assert torch.equal(ei.values.view(torch.uint8), y8.values[i:i + 1].view(torch.uint8))
        assert torch.equal(ei.scales, y8.scales[i:i + 1])


def test_the_documented_calls_run(capsys):
    """The front page's example of these operators, as written."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    block = [b for b in re.findall(r"```python\n(.*?)```", open(path).read(), re.S)
             if "adamw_step" in b]
    assert len(block) == 1
    scope = {}
    exec(compile(block[0], "README.md", "exec"), scope)
    total = scope["dnorm"].double().square().sum() + \
        scope["plan"].tensors[0]["grad"].double().square().sum()
    # printed with 16 digits; the norm is good to 2^-40
    assert abs(float(capsys.readouterr().out) - math.sqrt(float(total))) < 1e-11 * math.sqrt(float(total))
    assert torch.equal(scope["w16"], scope["weight"].to(BF16))
    assert torch.isfinite(scope["dx"]).all() and torch.isfinite(scope["dq"]).all()
