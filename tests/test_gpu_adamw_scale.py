"""Loss scales whose inverse fp32 does not have: the factor of the gradients would be
infinite (NaN where they are zero) or nothing at all.  They are refused; the largest and
smallest that are not give the step they should."""
import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, E4M3 = defs.F32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("states", [F32, E4M3])
def test_scales(states):
    n = 300
    param = torch.ones(n, device=DEV)
    grad = torch.zeros(n, device=DEV)
    plan = rcc.AdamWPlan([dict(param=param, grad=grad)], states=states)
    cfg = rcc.adamw_cfg(lr=1e-3, weight_decay=0.0, max_grad_norm=0.0)
    for scale in (2.0 ** -129, 1e-45, 1e-300, 2.0 ** 127, 1e39, 1e300):
        with pytest.raises(rcc.RccError):
            rcc.adamw_step(plan, cfg, scale)
    assert rcc.adamw_report(plan).step == 0
    assert torch.equal(param, torch.ones_like(param))
    for k, scale in enumerate((2.0 ** -127, 2.0 ** 126)):
        grad.fill_(scale if scale > 1 else 2.0 ** -126)
        rcc.adamw_step(plan, cfg, scale)
        r = rcc.adamw_report(plan)
        assert r.step == k + 1 and r.skipped == 0
        want = float(grad[0]) / scale * n ** 0.5
        assert abs(r.grad_norm - want) <= 2.0 ** -40 * want
        # the gradient is 2 and then 1: Adam's first steps are lr times about 1
        assert bool(((1.0 - param) > 0.0009 * (k + 1)).all()) and bool((param > 0.997).all())
