"""The gradients' norm of an AdamW step, of many elements: good to 2^-40, as documented,
where the errors of the sums all point one way (equal gradients that are no short
binary fractions), and where they do not.
"""
from fractions import Fraction
import math

import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = defs.F32, defs.BF16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def norm_of(grad):
    n = grad.numel()
    plan = rcc.AdamWPlan([dict(param=torch.zeros(n, device=DEV), grad=grad)], states=E4M3)
    rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=1.0))
    r = rcc.adamw_report(plan)
    assert r.skipped == 0 and r.nonfinite == 0
    return r.grad_norm


def root(x):
    """The square root of a Fraction, good to a double."""
    shift = 200
    return math.isqrt(int(x * (1 << (2 * shift)))) / (1 << shift)


@pytest.mark.parametrize("kind,offset", [(F32, 0), (BF16, 0), (F32, 1), (BF16, 1)])
@pytest.mark.parametrize("n", [100_000, 30_000_000, 400_000_000])
def test_equal_gradients(kind, offset, n):
    for value in (0.1, 0.7071, 1e-7):
        grad = torch.full((n + offset,), value, dtype=kind, device=DEV)[offset:]
        want = root(n * Fraction(float(grad[0])) ** 2)
        assert abs(norm_of(grad) - want) <= 2.0 ** -40 * want, (value, norm_of(grad) / want - 1)


@pytest.mark.parametrize("kind", [F32, BF16])
def test_gradients_of_many_sizes(kind):
    """Compared with sums of exact squares, in fp64 pieces of 4,096 (good to 2^-44)."""
    g = defs.gen(401)
    n = 200_000_000 // 4096 * 4096
    grad = (defs.randn(g, n) * torch.exp(4.0 * defs.randn(g, n // 4096)).repeat_interleave(4096)).to(kind)
    pieces = torch.cat([part.double().square().view(-1, 4096).sum(1)
                        for part in grad.view(-1).split(1 << 24)])
    want = math.sqrt(math.fsum(pieces.cpu().tolist()))
    assert abs(norm_of(grad) - want) <= 2.0 ** -40 * want
