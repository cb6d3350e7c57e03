"""The language-model operators at sizes that give a block several tiles, rows
several slabs and runs several windows, against their definitions in 64 bits
(the checks and bounds of test_gpu_lm.py)."""
import pytest
import torch

import test_gpu_lm as defs

pytestmark = pytest.mark.gpu

F32, BF16 = defs.F32, defs.BF16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


# few tokens: tiles wider than 128 columns, and two a block; many: several
# accumulators a tile, and several tiles a pair
@pytest.mark.parametrize("tokens,vocab,dim", [(1, 32768, 64), (100, 50021, 136), (128, 100003, 72),
                                              (600, 20000, 1032), (1500, 9001, 520)])
@pytest.mark.parametrize("extra", [0, 8])
def test_linear_ce(tokens, vocab, dim, extra):
    defs.test_linear_ce(tokens, vocab, dim, extra)


# whole blocks to a row, several slabs, runs over many windows
@pytest.mark.parametrize("dout_type,grad_type", [(F32, F32), (BF16, F32), (BF16, BF16),
                                                 (F32, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,vocab,dim,extra", [(4097, 60, 520, 0), (4097, 3, 2056, 8),
                                                    (4097, 60, 1001, 0), (6000, 9000, 4100, 3),
                                                    (200, 50, 2500, 0)])
def test_embedding_backward(dout_type, grad_type, accumulate, tokens, vocab, dim, extra):
    defs.test_embedding_backward(dout_type, grad_type, accumulate, tokens, vocab, dim, extra)


# blocks that take many rows one after the other
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,dim,extra", [(20000, 136, 0), (5000, 1024, 8), (3000, 4096, 0),
                                              (6000, 1001, 0), (2500, 4095, 2), (700, 16384, 0),
                                              (500, 32760, 0)])
def test_rmsnorm(dtype, tokens, dim, extra):
    defs.test_rmsnorm(dtype, tokens, dim, extra)
