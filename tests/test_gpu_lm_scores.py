"""The output layer's special values, against 64 bits: large scores, certain
tokens, masked vocabulary entries, padding tokens that hold anything."""
import math

import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U, F32, BF16 = defs.U, defs.F32, defs.BF16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def exact_scores(tokens, vocab, steps):
    """x and w with one column that is not zero: a score is one product of two
    bf16 numbers, which fp32 holds exactly.  w takes the values 1 - i / 256."""
    x = torch.zeros(tokens, 8, device=DEV)
    x[:, 0] = torch.linspace(30.0, 2000.0, tokens, device=DEV) if tokens > 1 else 1000.0
    w = torch.zeros(vocab, 8, device=DEV)
    w[:, 0] = 1.0 - torch.arange(vocab, device=DEV) % steps / 256.0
    return x.to(BF16), w.to(BF16)


# ---------------------------------------------------------------- certain tokens

@pytest.mark.parametrize("tokens", [1, 100, 300])
@pytest.mark.parametrize("vocab", [20, 400])
def test_a_certain_token_has_no_loss(tokens, vocab):
    """Scores m >= 30 of the label and 0 of all others: the others' share, below
    400 e^-30 = 4e-11, is less than half a unit of the 1 it is added to, so the
    sum is 1 and the loss 0; in no case less."""
    x, _ = exact_scores(tokens, vocab, 1)
    w = torch.zeros(vocab, 8, device=DEV, dtype=BF16)
    w[vocab // 2, 0] = 1.0
    labels = torch.full((tokens,), vocab // 2, device=DEV)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    assert float(loss.min()) >= 0.0 and float(loss.max()) <= 1e-9
    assert torch.equal(lse, x[:, 0].float())


@pytest.mark.parametrize("tokens", [1, 100, 300])
def test_loss_of_large_exact_scores(tokens):
    """The bound of the sum of exponentials alone: no rounding of a score, and
    none that grows with a score's size."""
    vocab = 20
    x, w = exact_scores(tokens, vocab, 3)
    labels = torch.arange(tokens, device=DEV) % vocab
    loss, _ = rcc.linear_ce_forward(x, w, labels)
    z = x[:, 0].double()[:, None] * w[:, 0].double()
    lse = torch.logsumexp(z, 1)
    want = lse - z.gather(1, labels[:, None])[:, 0]
    far = (z - lse[:, None]).abs().amax(1)
    # vocab additions, the exponentials' last bits and their arguments', the final sum
    near = torch.where((z - lse[:, None]).abs() < 40, (z - lse[:, None]).abs(), 0.0).amax(1)
    defs.within(loss, want, (vocab + 16 + 4 * near) * U + 2 * U * far)


@pytest.mark.parametrize("tokens", [1, 40, 130])
def test_gradient_of_large_exact_scores(tokens):
    """dz = exp(z - lse) - [label] of scores near 1,000 and an lse that fp32
    holds exactly, read off dw: every token alike, so dw = tokens dz x."""
    vocab = 12
    x, w = exact_scores(1, vocab, 3)
    x = x.expand(tokens, 8).contiguous()
    labels = torch.zeros(tokens, dtype=torch.int64, device=DEV)
    dloss = torch.ones(tokens, device=DEV)
    z = x[0, 0].double() * w[:, 0].double()
    for at in range(12):
        lse = torch.full((tokens,), 1000.5 + at * 0.0625, device=DEV)
        _, dw = rcc.linear_ce_backward(x, w, labels, lse, dloss, grad_dtype=F32, need_dx=False)
        p = torch.exp(z - float(lse[0]))
        one = torch.zeros_like(p)
        one[0] = 1.0
        want = (p - one) * tokens * 1000.0
        far = (z - float(lse[0])).abs()
        # p: its argument's roundings and its own; dz in three parts: 2^-23 of it;
        # truncating additions of three products a token
        size = p * (8 + 4 * far) * U + 2 * U * (p - one).abs()
        bound = (size + ((p - one).abs() + size) * U * (2 + 2 * (3 * tokens + 16))) * tokens * 1000.0
        defs.within(dw[:, 0], want, bound + 2.0 ** -100)


# ---------------------------------------------------------------- masked entries

LOWEST = torch.finfo(BF16).min


@pytest.mark.parametrize("mask", [-math.inf, LOWEST])
@pytest.mark.parametrize("tokens", [1, 60, 200])
@pytest.mark.parametrize("vocab,first,last", [(257, 256, 257), (640, 128, 256), (640, 0, 384),
                                              (5000, 16, 4990)])
def test_masked_entries_do_not_count(tokens, vocab, first, last, mask):
    """Entries whose score is minus infinity, or the type's lowest value, have no
    part in the loss, also where a whole tile of scores holds nothing else."""
    x, w, _, dloss = defs.ce_inputs(21, tokens, vocab, 72)
    x[:, 0] = 1.0
    w[first:last] = 0.0
    w[first:last, 0] = mask
    keep = torch.ones(vocab, dtype=torch.bool, device=DEV)
    keep[first:last] = False
    kept = torch.nonzero(keep)[:, 0]
    at = torch.arange(tokens, device=DEV) * 7 % kept.numel()
    want, bound = defs.ce_64(x, w[kept], at, dloss)
    loss, lse = rcc.linear_ce_forward(x, w, kept[at])
    defs.within(lse, want["lse"], bound["lse"] + vocab * U)
    defs.within(loss, want["loss"], bound["loss"] + vocab * U)
    for kind in (BF16, F32):
        _, dw = rcc.linear_ce_backward(x, w, kept[at], lse, dloss, grad_dtype=kind, need_dx=False)
        assert not dw[~keep].any()
        defs.within(dw[kept], want["dw"], bound["dw", kind])


# ---------------------------------------------------------------- padding tokens

@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tokens,vocab,dim,extra", [(3, 300, 72, 0), (100, 2049, 200, 8),
                                                    (200, 700, 1000, 0), (640, 1500, 512, 8)])
def test_what_padding_tokens_hold_reaches_nothing(tokens, vocab, dim, extra, bad):
    """Padding adds to no gradient, whatever stands in its row of x and its dloss:
    the bits are those of rows of zeros."""
    x, w, labels, dloss = defs.ce_inputs(22, tokens, vocab, dim)
    labels[0] = -1
    padding = (labels < 0) | (labels >= vocab)
    x[padding] = 0.0
    clean = x.clone()
    x[padding] = bad
    dirty = dloss.clone()
    dirty[padding] = bad
    if extra:
        x = defs.strided(x, extra)
    loss0, lse0 = rcc.linear_ce_forward(clean, w, labels)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    assert torch.equal(loss, loss0) and torch.equal(lse[~padding], lse0[~padding])
    for kind in (BF16, F32):
        dx0, dw0 = rcc.linear_ce_backward(clean, w, labels, lse0, dloss, grad_dtype=kind)
        dx, dw = rcc.linear_ce_backward(x, w, labels, lse, dirty, grad_dtype=kind)
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
        base = torch.ones_like(dw)
        only = rcc.linear_ce_backward(x, w, labels, lse, dirty, dw=base.clone(), need_dx=False,
                                      accumulate=True)[1]
        assert torch.equal(only, rcc.linear_ce_backward(clean, w, labels, lse0, dloss,
                                                        dw=base.clone(), need_dx=False,
                                                        accumulate=True)[1])
