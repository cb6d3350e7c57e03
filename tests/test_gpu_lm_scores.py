"""The output layer's special values, against 64 bits: masked vocabulary entries."""
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


# ---------------------------------------------------------------- masked entries

@pytest.mark.parametrize("mask", [-math.inf])
@pytest.mark.parametrize("tokens", [1, 60, 200])
@pytest.mark.parametrize("vocab,first,last", [(257, 256, 257), (640, 128, 256), (640, 0, 384),
                                              (5000, 16, 4990)])
def test_masked_entries_do_not_count(tokens, vocab, first, last, mask):
    """Entries whose score is minus infinity have no part in the loss, also where
    a whole tile of scores holds nothing else."""
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
