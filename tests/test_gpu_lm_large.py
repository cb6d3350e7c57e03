"""The language-model operators on matrices of more than 2^31 elements: offsets
that pass 32 bits.  Rows at both ends are compared with the definitions."""
import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U, F32, BF16 = defs.U, defs.F32, defs.BF16
ROWS, DIM = 530000, 4096   # 2.17e9 elements


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    assert ROWS * DIM > 1 << 31
    yield
    torch.cuda.empty_cache()


def large(seed, scale=1.0):
    """Random at both ends, a pattern of few values between."""
    t = torch.full((ROWS, DIM), 0.25, dtype=BF16, device=DEV)
    g = defs.gen(seed)
    for part in (t[:600], t[-600:]):
        part.copy_(defs.randn(g, 600, DIM, scale=scale))
    return t


def test_embedding():
    table = large(41)
    ids = torch.tensor([0, ROWS - 1, ROWS - 300, 5, ROWS, -1, ROWS - 1], device=DEV)
    out = rcc.embedding_forward(table, ids, out_dtype=F32)
    for i, at in enumerate(ids.tolist()):
        want = table[at].float() if 0 <= at < ROWS else torch.zeros(DIM, device=DEV)
        assert torch.equal(out[i], want)
    before = table[-300:].clone()
    dout = defs.randn(defs.gen(42), ids.numel(), DIM)
    rcc.embedding_backward(dout, ids, table, accumulate=True)
    want, bound = defs.embedding_grad_64(dout, ids - (ROWS - 300), 300, 1.0, before)
    defs.within(table[-300:], want, bound + defs.half_ulp(want, BF16))
    rcc.embedding_backward(dout, ids, table)
    assert not table[6:-300].any() and not table[-299:-1].any()
    want, bound = defs.embedding_grad_64(dout, ids - (ROWS - 300), 300, 1.0, None)
    defs.within(table[-300:], want, bound + defs.half_ulp(want, BF16))


def test_rmsnorm():
    x, weight = large(43), 1.0 + defs.randn(defs.gen(44), DIM, scale=0.2)
    y, kept = rcc.rmsnorm_forward(x, weight, keep=True)
    dx, _ = rcc.rmsnorm_backward(x, kept, weight)
    for rows in (slice(0, 500), slice(ROWS - 500, ROWS)):
        ys, ks = rcc.rmsnorm_forward(x[rows], weight, keep=True)   # a row's bits are its own
        assert torch.equal(y[rows], ys)
        assert torch.equal(kept.values[rows], ks.values)
        assert torch.equal(kept.scales[rows], ks.scales)
        assert torch.equal(dx[rows], rcc.rmsnorm_backward(x[rows], ks, weight)[0])


def test_output_layer_of_a_large_vocabulary():
    w = large(45, scale=2.0 / DIM ** 0.5)
    w[600:-600] = 0.0
    ends = torch.cat([torch.arange(600, device=DEV), torch.arange(ROWS - 600, ROWS, device=DEV)])
    x = defs.randn(defs.gen(46), 5, DIM, dtype=BF16)
    labels = torch.tensor([ROWS - 1, 3, -1, ROWS - 555, ROWS], device=DEV)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    # the 528,800 rows of zeros have scores of 0
    z = torch.cat([x.double() @ w[ends].double().t(), torch.zeros(5, 1, device=DEV).double()], 1)
    z_all = torch.cat([z[:, :-1], z[:, -1:] + torch.tensor(float(ROWS - 1200)).log()], 1)
    want = torch.logsumexp(z_all, 1)
    # every sum of exponentials: at most ROWS additions, most of them within 256 columns, then
    # a few thousand pairs; scores as in ce_64
    bound = 2 * U * DIM * (x.abs().double() @ w[ends].abs().double().t()).amax(1) + 8192 * U
    defs.within(lse, want, bound + 4 * U * want.abs())
    _, dw = rcc.linear_ce_backward(x, w, labels, lse, torch.ones(5, device=DEV), need_dx=False)
    dz = torch.exp(z[:, :-1] - want[:, None])
    for t, at in ((0, ROWS - 1), (1, 3), (3, ROWS - 555)):
        dz[t, int(torch.nonzero(ends == at))] -= 1.0
    dz[labels < 0] = 0.0
    dz[labels >= ROWS] = 0.0
    exact = dz.t() @ x.double()
    # dz is rounded to bf16, and so is the result; its own error is that of lse and the scores
    size = dz.abs().t() @ x.abs().double()
    defs.within(dw[ends], exact, (2.0 ** -8 + float(bound.max()) * 2 + 1e-5) * size * 1.01
                + defs.half_ulp(exact, BF16) + 1e-9)


def test_output_layer_of_many_tokens():
    x = large(47)
    w = defs.randn(defs.gen(48), 300, DIM, dtype=BF16, scale=2.0 / DIM ** 0.5)
    labels = torch.full((ROWS,), -1, device=DEV)
    labels[-500:] = torch.arange(500, device=DEV) % 300
    dloss = torch.ones(ROWS, device=DEV)
    loss, lse = rcc.linear_ce_forward(x, w, labels)
    dx, dw = rcc.linear_ce_backward(x, w, labels, lse, dloss)
    assert not loss[:-500].any() and not dx[:-500].any()
    want, bound = defs.ce_64(x[-500:], w, labels[-500:], dloss[-500:])
    defs.within(loss[-500:], want["loss"], bound["loss"])
    defs.within(lse[-500:], want["lse"], bound["lse"])
    defs.within(dx[-500:], want["dx"], bound["dx", BF16])
    defs.within(dw, want["dw"], bound["dw", BF16])
    z = x[:500].double() @ w.double().t()
    far = (z - torch.logsumexp(z, 1)[:, None]).abs().amax(1)
    ez = 2 * U * DIM * (x[:500].abs().double() @ w.abs().double().t()).amax(1)
    defs.within(lse[:500], torch.logsumexp(z, 1), ez + (316 + 4 * far) * U + 4 * U * lse[:500].abs())
