"""adamw_report waits for the plan's last step, whichever stream it ran on."""
import pytest
import torch

from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

DELAY = 200000000   # cycles, about 100 ms: the step behind it is still to come


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    rcc.adamw_step(made(), rcc.adamw_cfg())   # the first launch loads the kernels, and waits
    torch.cuda.synchronize()


def made():
    param, grad = torch.ones(1000, device=DEV), torch.ones(1000, device=DEV)
    plan = rcc.AdamWPlan([dict(param=param, grad=grad)])
    torch.cuda.synchronize()
    return plan


@pytest.mark.parametrize("form", ["stream", "handle", "current"])
def test_a_step_on_another_stream(form):
    plan, side = made(), torch.cuda.Stream()
    for k in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(DELAY)
            if form == "current":
                rcc.adamw_step(plan, rcc.adamw_cfg())
        if form != "current":
            rcc.adamw_step(plan, rcc.adamw_cfg(), stream=side if form == "stream" else side.cuda_stream)
        assert not side.query()
        r = rcc.adamw_report(plan)
        assert r.step == k + 1 and abs(r.grad_norm - 1000 ** 0.5) < 1e-9


def test_a_step_on_the_default_stream_and_a_report_on_another():
    plan, side = made(), torch.cuda.Stream()
    torch.cuda._sleep(DELAY)
    rcc.adamw_step(plan, rcc.adamw_cfg())
    assert rcc.adamw_report(plan, stream=side).step == 1
    # and a plan that no step has run of
    assert rcc.adamw_report(made(), stream=side).step == 0


def test_replays_on_the_reporting_stream():
    plan = made()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rcc.adamw_step(plan, rcc.adamw_cfg())
    assert rcc.adamw_report(plan).step == 0
    torch.cuda._sleep(DELAY)
    graph.replay()
    graph.replay()
    assert rcc.adamw_report(plan).step == 2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
        graph.replay()
    assert rcc.adamw_report(plan, stream=side).step == 3
