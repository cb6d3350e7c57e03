"""Language-model operators on the GPU against their definitions in 64 bits.

Tolerances are worst-case rounding bounds of the formulas, element by element:
u = 2^-24 is the unit of one fp32 rounding; one of bf16, with its 8 significant
bits, costs at most 2^-8 of the value.  A sum of n terms in any order is off by at
most n u sum|term|; on the tensor cores an addition may truncate (2 u each).
"""
import math

import numpy as np
import pytest
import torch

from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV, Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def half_ulp(v, dtype):
    """What rounding v once to dtype may cost (bf16; fp32 is in the other terms)."""
    return v.abs() * 2.0 ** -8 + 2.0 ** -133 if dtype == BF16 else 0.0


def within(got, want, bound):
    err = (got.double() - want).abs()
    assert bool(torch.all(err <= bound)), \
        "off by up to %g where %g is allowed" % (float((err - bound).max()), float(bound.max()))


def skewed_ids(g, tokens, vocab, dtype=torch.int64, padding=0.1):
    u = torch.rand(tokens, generator=g, device=DEV, dtype=torch.float64)
    ids = ((vocab + 1.0) ** u).long().clamp_(1, vocab) - 1
    if padding:
        ids[torch.rand(tokens, generator=g, device=DEV) < padding] = -1
    return ids.to(dtype)


def strided(t, extra):
    """The same rows, `extra` elements further apart."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ------------------------------------------------------------------- embedding

@pytest.mark.parametrize("table_type,out_type", [(F32, F32), (F32, BF16), (BF16, BF16),
                                                 (BF16, F32)])
@pytest.mark.parametrize("tokens,vocab,dim,extra", [(1, 1, 1, 0), (7, 50, 64, 0), (5, 33, 7, 3),
                                                    (130, 1000, 2056, 8), (9, 20, 4096, 1)])
def test_embedding_forward(table_type, out_type, tokens, vocab, dim, extra):
    g = gen(1)
    table = strided(randn(g, vocab, dim, dtype=table_type), extra) if extra else \
        randn(g, vocab, dim, dtype=table_type)
    ids = skewed_ids(g, tokens, vocab)
    if tokens > 4:
        ids[1], ids[2], ids[3] = vocab, -100, vocab - 1
    for index in (torch.int64, torch.int32):
        out = Guarded(tokens * dim, out_type)
        rcc.embedding_forward(table, ids.to(index), scale=1.7, out=out.t.view(tokens, dim))
        inside = (ids >= 0) & (ids < vocab)
        want = table[ids.clamp(0, vocab - 1)].float() * torch.tensor(1.7, device=DEV)
        want = torch.where(inside[:, None], want, 0.0).to(out_type)
        assert torch.equal(out.t.view(tokens, dim), want)   # one product, rounded once
        assert out.guards_intact()


def embedding_grad_64(dout, ids, vocab, scale, base):
    want = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=DEV) if base is None \
        else base.double()
    size = torch.zeros_like(want) if base is None else base.double().abs()
    hit = torch.nonzero((ids >= 0) & (ids < vocab))[:, 0]
    want.index_add_(0, ids[hit].long(), dout[hit].double(), alpha=scale)
    size.index_add_(0, ids[hit].long(), dout[hit].double().abs(), alpha=scale)
    count = torch.bincount(ids[hit].long(), minlength=vocab).double()
    return want, (count[:, None] + 4) * U * size


@pytest.mark.parametrize("dout_type,grad_type", [(F32, F32), (BF16, F32), (BF16, BF16),
                                                 (F32, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,vocab,dim,extra", [
    (1, 1, 1, 0), (1, 40, 64, 0), (31, 3, 8, 0), (33, 1, 72, 0),       # one row takes everything
    (700, 511, 40, 8), (700, 512, 9, 2),                               # one digit, two digits
    (4097, 5000, 264, 0), (9000, 300000, 16, 0),                       # windows; three digits
    (70000, 97, 8, 0)])                                                # long runs, wide windows
def test_embedding_backward(dout_type, grad_type, accumulate, tokens, vocab, dim, extra):
    g = gen(2)
    dout = randn(g, tokens, dim, dtype=dout_type)
    if extra:
        dout = strided(dout, extra)
    ids = skewed_ids(g, tokens, vocab, torch.int32 if tokens % 2 else torch.int64)
    if tokens > 4:
        ids[0], ids[2] = vocab, vocab - 1
    base = randn(g, vocab, dim, dtype=grad_type)
    out = Guarded(vocab * dim, grad_type, fill=base.reshape(-1))
    dtable = out.t.view(vocab, dim)
    rcc.embedding_backward(dout, ids, dtable, scale=0.75, accumulate=accumulate)
    want, bound = embedding_grad_64(dout, ids, vocab, 0.75, base if accumulate else None)
    within(dtable, want, bound + half_ulp(want, grad_type))
    assert out.guards_intact()
    present = torch.zeros(vocab, dtype=torch.bool, device=DEV)
    present[ids[(ids >= 0) & (ids < vocab)].long()] = True
    rest = base if accumulate else torch.zeros_like(base)
    assert torch.equal(dtable[~present], rest[~present])
    # the same bits again, whatever the workspace held
    again = base.clone()
    need = rcc.embedding_backward_workspace(tokens, vocab, dim)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    rcc.embedding_backward(dout, ids, again, scale=0.75, accumulate=accumulate, workspace=ws)
    assert torch.equal(again, dtable)


def test_embedding_backward_all_padding_and_no_tokens():
    base = randn(gen(3), 10, 24)
    for ids in (torch.full((6,), -1, device=DEV), torch.full((6,), 10, device=DEV),
                torch.empty(0, dtype=torch.int64, device=DEV)):
        dout = torch.full((ids.numel(), 24), float("nan"), device=DEV)
        kept = rcc.embedding_backward(dout, ids, base.clone(), accumulate=True)
        assert torch.equal(kept, base)
        assert not rcc.embedding_backward(dout, ids, base.clone()).any()
    assert rcc.embedding_forward(base, torch.empty(0, dtype=torch.int32, device=DEV)).shape == (0, 24)


def test_embedding_gradient_is_the_forward_pass_transposed():
    """<dout, E(W)> is linear in W: its difference along D is <dW, D>."""
    g = gen(4)
    ids = skewed_ids(g, 300, 60)
    dout, table, along = randn(g, 300, 40), randn(g, 60, 40), randn(g, 60, 40)
    dtable = rcc.embedding_backward(dout, ids, torch.empty_like(table), scale=3.0)
    f = [float((rcc.embedding_forward(table + s * along, ids, scale=3.0).double()
                * dout.double()).sum()) for s in (1, -1)]
    got = float((dtable.double() * along.double()).sum())
    size = float((dtable.double().abs() * (along.abs() + table.abs()).double()).sum()) + \
        3.0 * float(dout.double().abs().sum()) * 8
    assert abs((f[0] - f[1]) / 2 - got) <= 300 * U * size


# -------------------------------------------------------------------- RMS norm

def kept_reference(x):
    """The 8-bit form in numpy's fp32, operation for operation."""
    x = x.float().cpu().numpy()
    t, d = x.shape
    g = -(-d // 128)
    pad = np.zeros((t, g * 128), np.float32)
    pad[:, :d] = x
    pad = pad.reshape(t, g, 128)
    a = np.abs(pad).max(2)
    small = a < np.float32(2.0 ** -120)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(small, np.float32(0), np.float32(127) * (np.float32(1) / a))
    q = np.rint(pad * inv[:, :, None]).astype(np.int8)
    return q.reshape(t, g * 128), np.where(small, np.float32(0), a * np.float32(1.0 / 127))


NORM_SHAPES = [(1, 1, 0), (3, 8, 0), (5, 127, 3), (9, 129, 0), (17, 256, 8), (4, 500, 4),
               (6, 1000, 0), (3, 1024, 0), (2, 2050, 6), (310, 4096, 0), (5, 8192, 0),
               (2, 16384, 0), (2, 32768, 0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,dim,extra", NORM_SHAPES)
def test_rmsnorm(dtype, tokens, dim, extra):
    g = gen(5)
    x = randn(g, tokens, dim, dtype=dtype, scale=3.0)
    x[:, dim // 2] *= 40
    if tokens > 2:
        x[1] = 0                       # a row of nothing
        x[2] *= 2.0 ** -124            # below what the 8-bit form holds
    if extra:
        x = strided(x, extra)
    weight = 1.0 + randn(g, dim, scale=0.2)
    eps = 1e-5
    out = Guarded(tokens * dim, dtype)
    y, kept = rcc.rmsnorm_forward(x, weight, eps=eps, keep=True, out=out.t.view(tokens, dim))
    x64, w64 = x.double(), weight.double()
    want = x64 / (x64.square().mean(1, keepdim=True) + np.float32(eps)).sqrt() * w64
    # the sum of squares passes through at most 8 * 4 + 10 + 32 additions and halves in the root
    within(y, want, 48 * U * want.abs() + 2.0 ** -149 + half_ulp(want, dtype))
    assert out.guards_intact()
    assert torch.equal(rcc.rmsnorm_forward(x, weight, eps=eps), y)
    q, s = kept_reference(x)
    assert np.array_equal(kept.values.cpu().numpy(), q)
    assert np.array_equal(kept.scales.cpu().numpy(), s)

    dy = randn(g, tokens, dim, dtype=dtype)
    if extra:
        dy = strided(dy, extra)
    grad = Guarded(tokens * dim, dtype)
    dweight = Guarded(dim, F32)
    rcc.rmsnorm_backward(dy, kept, weight, eps=eps, dx=grad.t.view(tokens, dim),
                         dweight=dweight.t)
    x64 = torch.from_numpy(q.astype(np.float64)).to(DEV).view(tokens, -1, 128) * \
        torch.from_numpy(s.astype(np.float64)).to(DEV)[:, :, None]
    x64 = x64.view(tokens, -1)[:, :dim]
    r = 1 / (x64.square().mean(1, keepdim=True) + np.float32(eps)).sqrt()
    n, d = x64 * r, dy.double() * w64
    want = r * (d - n * (d * n).mean(1, keepdim=True))
    size = r * (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True))
    # two such sums, three roots' worth of r, and a few products
    within(grad.t.view(tokens, dim), want, 256 * U * size + 2.0 ** -149 + half_ulp(want, dtype))
    terms = dy.double() * n
    within(dweight.t, terms.sum(0), (tokens + 64) * U * terms.abs().sum(0) + 2.0 ** -140)
    assert grad.guards_intact() and dweight.guards_intact()
    base = randn(g, dim)
    dx2, added = rcc.rmsnorm_backward(dy, kept, weight, eps=eps, dweight=base.clone(),
                                      accumulate=True)
    assert torch.equal(dx2, grad.t.view(tokens, dim))
    assert torch.equal(added, base + dweight.t)


def test_rmsnorm_gradient_against_differences():
    """Central differences of the norm itself, in 64 bits, at the kept input."""
    g = gen(6)
    tokens, dim = 4, 300
    weight = 1.0 + randn(g, dim, scale=0.2)
    _, kept = rcc.rmsnorm_forward(randn(g, tokens, dim), weight, keep=True)
    dy = randn(g, tokens, dim)
    dx, dweight = rcc.rmsnorm_backward(dy, kept, weight)
    at, w = kept.dequantize().double(), weight.double()

    def f(x, w):
        return float((dy.double() * x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * w).sum())

    h = 1e-5
    for _ in range(3):
        along, aw = randn(g, tokens, dim).double(), randn(g, dim).double()
        diff = (f(at + h * along, w + h * aw) - f(at - h * along, w - h * aw)) / (2 * h)
        got = float((dx.double() * along).sum() + (dweight.double() * aw).sum())
        size = float((dx.double().abs() * along.abs()).sum() +
                     (dweight.double().abs() * aw.abs()).sum())
        assert abs(diff - got) <= 1e-5 * size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rmsnorm_keeps_what_is_not_finite(dtype, bad):
    """A NaN or infinity makes its group's scale NaN, and its row's gradient."""
    g = gen(7)
    x = randn(g, 3, 300, dtype=dtype)
    x[1, 140] = bad
    weight = torch.ones(300, device=DEV)
    y, kept = rcc.rmsnorm_forward(x, weight, keep=True)
    assert torch.isnan(kept.scales).tolist() == [[False] * 3, [False, True, False], [False] * 3]
    assert not torch.isfinite(y[1]).all() and torch.isfinite(y[[0, 2]]).all()
    dx, dweight = rcc.rmsnorm_backward(torch.ones_like(x), kept, weight)
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[[0, 2]]).all()
    assert torch.isnan(dweight).all()


def test_rmsnorm_no_tokens():
    weight = torch.ones(40, device=DEV)
    y, kept = rcc.rmsnorm_forward(torch.empty(0, 40, device=DEV), weight, keep=True)
    assert y.shape == (0, 40)
    base = torch.ones(40, device=DEV)
    dx, dw = rcc.rmsnorm_backward(y, kept, weight, dweight=base.clone(), accumulate=True)
    assert dx.shape == (0, 40) and torch.equal(dw, base)
    assert not rcc.rmsnorm_backward(y, kept, weight, dweight=base.clone())[1].any()


# ----------------------------------------------------- output layer, cross entropy

def ce_64(x, w, labels, dloss):
    """Values in 64 bits and the worst-case bounds of each output."""
    x, w, labels = x.double(), w.double(), labels.long()
    dim, vocab = x.shape[1], w.shape[0]
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    hit = (labels >= 0) & (labels < vocab)
    at = torch.where(hit, labels, 0)
    loss = torch.where(hit, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    # additions that truncate: 2 u each, dim of them, of partial sums at most |x| |w|
    ez = 2 * U * dim * (x.abs() @ w.abs().t()) + U * z.abs()
    # the sum of exponentials: relative vocab u, each exponential a few ulp and its
    # argument's rounding (|z - lse| log2e u, taken with the row's largest)
    far = (z - lse[:, None]).abs().amax(1)
    elog = (vocab + 16 + 4 * far) * U
    elz = ez.amax(1) + elog + 4 * U * lse.abs()
    eloss = torch.where(hit, 2 * elz + 2 * U * loss.abs(), 0.0)
    p = torch.exp(z - lse[:, None])
    f = torch.where(hit, dloss.double(), 0.0)[:, None]
    one = torch.zeros_like(p)
    one[torch.nonzero(hit)[:, 0], labels[hit]] = 1.0
    dz = f * (p - one)
    edz = f.abs() * (p * (ez + elz[:, None] + (8 + 4 * far)[:, None] * U) + 2 * U * (p - one).abs())
    out = {"z": z, "lse": lse, "loss": loss, "dx": dz @ w, "dw": dz.t() @ x}
    bound = {"lse": elz, "loss": eloss}
    for kind, step in ((F32, 2.0 ** -23), (BF16, 2.0 ** -8)):
        e = edz * (1 + step) + step * dz.abs()
        for name, left, err, right, n in (("dx", dz, e, w, vocab),
                                          ("dw", dz.t(), e.t(), x, x.shape[0])):
            b = err @ right.abs() + 2 * U * (2 * n + 64) * ((left.abs() + err) @ right.abs())
            bound[name, kind] = b + half_ulp(out[name], kind) + 2.0 ** -140
    return out, bound


CE_SHAPES = [(1, 1, 8), (1, 5, 64), (3, 300, 72), (2, 1000, 136), (128, 256, 64), (129, 257, 128),
             (100, 2049, 200), (200, 700, 1000), (257, 513, 64), (300, 4000, 256), (640, 1500, 512)]


def ce_inputs(seed, tokens, vocab, dim, index=torch.int64):
    g = gen(seed)
    w = randn(g, vocab, dim, scale=2.0 / math.sqrt(dim))
    labels = skewed_ids(g, tokens, vocab, padding=0.1 if tokens > 1 else 0)
    x = randn(g, tokens, dim) + 2.0 * w[labels.clamp_min(0)]
    if tokens > 3:
        labels[1], labels[2] = vocab, -100
    dloss = torch.rand(tokens, generator=g, device=DEV) + 0.5
    return x.to(BF16), w.to(BF16), labels.to(index), dloss


@pytest.mark.parametrize("tokens,vocab,dim", CE_SHAPES)
@pytest.mark.parametrize("extra", [0, 8])
def test_linear_ce(tokens, vocab, dim, extra):
    x, w, labels, dloss = ce_inputs(8, tokens, vocab, dim,
                                    torch.int32 if vocab % 2 else torch.int64)
    if extra:
        x, w = strided(x, extra), strided(w, extra)
    want, bound = ce_64(x, w, labels, dloss)
    loss, lse = Guarded(tokens, F32), Guarded(tokens, F32)
    rcc.linear_ce_forward(x, w, labels, loss=loss.t, lse=lse.t)
    within(lse.t, want["lse"], bound["lse"])
    within(loss.t, want["loss"], bound["loss"])
    assert loss.guards_intact() and lse.guards_intact()
    for kind in (BF16, F32):
        dx, dw = Guarded(tokens * dim, kind), Guarded(vocab * dim, kind)
        rcc.linear_ce_backward(x, w, labels, lse.t, dloss, dx=dx.t.view(tokens, dim),
                               dw=dw.t.view(vocab, dim))
        within(dx.t.view(tokens, dim), want["dx"], bound["dx", kind])
        within(dw.t.view(vocab, dim), want["dw"], bound["dw", kind])
        assert dx.guards_intact() and dw.guards_intact()
        # one of the two alone, added to what is there, a workspace of ones: the same bits
        ws = torch.full((rcc.linear_ce_workspace(tokens, vocab, dim, True, kind),), 0xFF,
                        dtype=torch.uint8, device=DEV)
        only, none = rcc.linear_ce_backward(x, w, labels, lse.t, dloss, grad_dtype=kind,
                                            need_dw=False, workspace=ws)
        assert none is None and torch.equal(only, dx.t.view(tokens, dim))
        base = torch.ones(vocab, dim, dtype=kind, device=DEV)
        none, added = rcc.linear_ce_backward(x, w, labels, lse.t, dloss, dw=base.clone(),
                                             need_dx=False, accumulate=True)
        assert none is None
        within(added, want["dw"] + 1.0, bound["dw", kind] + 2 * U + half_ulp(want["dw"] + 1, kind))


def test_linear_ce_vocabulary_in_pieces():
    """More dz than the workspace holds at a time; outputs 16 bytes into a sector."""
    tokens, vocab, dim = 1810, 150100, 72
    x, w, labels, dloss = ce_inputs(16, tokens, vocab, dim)
    want, bound = ce_64(x, w, labels, dloss)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    within(lse, want["lse"], bound["lse"])
    within(loss, want["loss"], bound["loss"])
    for kind, bytes_each in ((BF16, 2), (F32, 6)):
        assert rcc.linear_ce_workspace(tokens, vocab, dim, True, kind) < tokens * vocab * bytes_each
        pad = 16 // torch.empty(0, dtype=kind).element_size()
        dx = torch.empty(tokens * dim + pad, dtype=kind, device=DEV)[pad:].view(tokens, dim)
        dw = torch.empty(vocab * dim + pad, dtype=kind, device=DEV)[pad:].view(vocab, dim)
        rcc.linear_ce_backward(x, w, labels, lse, dloss, dx=dx, dw=dw)
        within(dx, want["dx"], bound["dx", kind])
        within(dw, want["dw"], bound["dw", kind])
        dw.fill_(1.0)
        rcc.linear_ce_backward(x, w, labels, lse, dloss, dw=dw, need_dx=False, accumulate=True)
        within(dw, want["dw"] + 1.0, bound["dw", kind] + 2 * U + half_ulp(want["dw"] + 1, kind))


def test_linear_ce_gradient_against_differences():
    """Central differences of the loss in 64 bits."""
    x, w, labels, dloss = ce_inputs(9, 40, 300, 64)
    _, lse = rcc.linear_ce_forward(x, w, labels)
    dx, dw = rcc.linear_ce_backward(x, w, labels, lse, dloss, grad_dtype=F32)
    hit = (labels >= 0) & (labels < 300)

    def f(x, w):
        z = x @ w.t()
        e = torch.logsumexp(z, 1) - z.gather(1, labels.clamp(0, 299)[:, None])[:, 0]
        return float((e * dloss.double())[hit].sum())

    g, h = gen(10), 1e-5
    for _ in range(3):
        ax, aw = randn(g, 40, 64).double(), randn(g, 300, 64).double()
        diff = (f(x.double() + h * ax, w.double() + h * aw)
                - f(x.double() - h * ax, w.double() - h * aw)) / (2 * h)
        got = float((dx.double() * ax).sum() + (dw.double() * aw).sum())
        size = float((dx.double().abs() * ax.abs()).sum() + (dw.double().abs() * aw.abs()).sum())
        assert abs(diff - got) <= 1e-5 * size


def test_linear_ce_every_label_padding():
    x, w, labels, dloss = ce_inputs(11, 150, 400, 64)
    labels.fill_(-1)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    assert not loss.any() and torch.isfinite(lse).all()
    for kind in (BF16, F32):
        dx, dw = rcc.linear_ce_backward(x, w, labels, lse, dloss, grad_dtype=kind)
        assert not dx.any() and not dw.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_linear_ce_what_is_not_finite_reaches_its_row(bad):
    x, w, labels, dloss = ce_inputs(12, 140, 600, 64)
    labels.clamp_(0, 599)
    x[5, 3] = bad
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    rest = torch.arange(140, device=DEV) != 5
    assert not torch.isfinite(loss[5]) and torch.isfinite(loss[rest]).all()
    dx, dw = rcc.linear_ce_backward(x, w, labels, lse, dloss)
    assert torch.isnan(dx[5]).all() and torch.isfinite(dx[rest]).all()
    assert torch.isnan(dw).all()


def test_linear_ce_large_scores_do_not_overflow():
    x, w, labels, dloss = ce_inputs(13, 130, 500, 64)
    x, w = (x.float() * 60).to(BF16), (w.float() * 60).to(BF16)   # scores of several thousand
    want, bound = ce_64(x, w, labels, dloss)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    within(lse, want["lse"], bound["lse"])
    within(loss, want["loss"], bound["loss"])
    dx, dw = rcc.linear_ce_backward(x, w, labels, lse, dloss)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_linear_ce_no_tokens():
    w = randn(gen(14), 30, 16, dtype=BF16)
    x = torch.empty(0, 16, dtype=BF16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse = rcc.linear_ce_forward(x, w, none)
    assert loss.shape == lse.shape == (0,)
    dx, dw = rcc.linear_ce_backward(x, w, none, lse, loss)
    assert dx.shape == (0, 16) and not dw.any()
    base = torch.ones(30, 16, dtype=BF16, device=DEV)
    _, dw = rcc.linear_ce_backward(x, w, none, lse, loss, dw=base.clone(), accumulate=True)
    assert torch.equal(dw, base)


# --------------------------------------------------------------------- streams, graphs

def test_operators_on_a_side_stream_and_in_a_graph():
    """On another stream than the current one, and replayed from a CUDA graph
    on new inputs: the bits of the plain calls."""
    g = gen(15)
    vocab, dim, tokens = 700, 128, 300
    table, weight = randn(g, vocab, dim, scale=0.3), 1.0 + randn(g, dim, scale=0.1)
    ids = skewed_ids(g, tokens, vocab)
    w16 = table.to(BF16)
    dloss = torch.full((tokens,), 1.0 / tokens, device=DEV)

    def step(stream=None):
        h = rcc.embedding_forward(table, ids, out_dtype=BF16, stream=stream)
        y, kept = rcc.rmsnorm_forward(h, weight, keep=True, stream=stream)
        loss, lse = rcc.linear_ce_forward(y, w16, ids, stream=stream)
        dy, dw = rcc.linear_ce_backward(y, w16, ids, lse, dloss, dx=torch.empty_like(y),
                                        dw=torch.empty_like(w16), stream=stream)
        dh, dweight = rcc.rmsnorm_backward(dy, kept, weight, stream=stream)
        rcc.embedding_backward(dh, ids, dw, accumulate=True, stream=stream)
        return loss, dw, dweight

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    ids.copy_(ids.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))
