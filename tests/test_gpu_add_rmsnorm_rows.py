"""The residual norm's backward pass over many rows that are on no boundary: blocks
copy rows ahead into the stages that rows before them were read from.  dx and dweight
against 64 bits (the bounds of test_gpu_add_rmsnorm.py), and the same bits each time.
"""
import numpy as np
import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U, F32, BF16 = defs.U, defs.F32, defs.BF16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def unaligned(t, offset, extra):
    tokens, dim = t.shape
    wide = torch.full((offset + tokens * (dim + extra),), float("nan"), dtype=t.dtype, device=DEV)
    rows = wide[offset:].view(tokens, dim + extra)[:, :dim]
    rows.copy_(t)
    return rows


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,tokens", [(513, 9000), (1001, 9000), (2047, 6000), (4095, 5000),
                                        (8191, 3000), (12289, 1500), (16383, 1000), (20001, 700)])
def test_many_rows(dtype, dim, tokens):
    g = defs.gen(301)
    x = defs.randn(g, tokens, dim, dtype=dtype)
    weight = 1.0 + defs.randn(g, dim, scale=0.2)
    _, kept = rcc.rmsnorm_forward(x, weight, eps=EPS, keep=True)
    # each row's dh has a size of its own: a row with another one's is far off
    dy, dh = defs.randn(g, tokens, dim, dtype=dtype), defs.randn(g, tokens, dim)
    dh = (dh * (1.0 + 100.0 * torch.rand(tokens, 1, generator=g, device=DEV))).to(dtype)
    first = None
    for offset, extra in ((1, 0), (3, 1), (1, 0), (0, 3)):
        place = unaligned(dh, offset, extra)
        dx, dweight = rcc.add_rmsnorm_backward(unaligned(dy, offset, extra), place, kept, weight,
                                               eps=EPS)
        if first is None:
            first = dx, dweight
        assert torch.equal(dx, first[0]) and torch.equal(dweight, first[1])
    dx, dweight = first
    s64 = kept.scales.double()[:, :, None] * kept.values.double().view(tokens, -1, 128)
    x64, w64 = s64.view(tokens, -1)[:, :dim], weight.double()
    rr = 1 / (x64.square().mean(1, keepdim=True) + np.float32(EPS)).sqrt()
    n, d = x64 * rr, dy.double() * w64
    want = dh.double() + rr * (d - n * (d * n).mean(1, keepdim=True))
    size = rr * (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True))
    # the norm's own bound, one more addition, one rounding
    defs.within(dx, want, 256 * U * size + U * want.abs() + 2.0 ** -149 + defs.half_ulp(want, dtype))
    terms = dy.double() * n
    defs.within(dweight, terms.sum(0), (tokens + 64) * U * terms.abs().sum(0) + 2.0 ** -140)
    # in place of dh
    place = dh.clone()
    got, _ = rcc.add_rmsnorm_backward(unaligned(dy, 1, 1), place, kept, weight, eps=EPS, dx=place)
    assert got.data_ptr() == place.data_ptr() and torch.equal(got, dx)
