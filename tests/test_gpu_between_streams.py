"""The `stream` argument of the residual norm, rotary positions and AdamW: calls on
a stream that is not the current one, with outputs and workspaces left out."""
import threading

import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16, E4M3 = defs.BF16, torch.float8_e4m3fn
TOKENS, DIM, HEADS = 900, 520, 5
DELAY = 20000000   # cycles, about 10 ms: everything queued behind it is still to come


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Step:
    """All calls; `after` runs behind each of them."""

    def __init__(self, seed):
        g = defs.gen(seed)
        self.x, self.r = (defs.randn(g, TOKENS, DIM, dtype=BF16) for _ in range(2))
        self.weight = 1.0 + defs.randn(g, DIM, scale=0.1)
        self.turns = rcc.rotary_turns(104, device=DEV)
        self.param, self.start = (torch.empty(DIM, device=DEV) for _ in range(2))
        self.start.copy_(defs.randn(g, DIM))
        self.grad = torch.zeros(DIM, device=DEV)
        torch.cuda.synchronize()

    def run(self, stream=None, after=lambda: None):
        y, h, kept = rcc.add_rmsnorm_forward(self.x, self.r, self.weight, keep=True, stream=stream)
        after()
        y8, _ = rcc.add_rmsnorm_forward(self.x, self.r, self.weight, out_dtype=E4M3, stream=stream)
        after()
        q, k = y.view(TOKENS, HEADS, DIM // HEADS), h.view(TOKENS, HEADS, DIM // HEADS)
        q, k = rcc.rotary_forward(q, k, self.turns, stream=stream)
        after()
        dq, dk = rcc.rotary_backward(q, k, self.turns, stream=stream)
        after()
        dx, dweight = rcc.add_rmsnorm_backward(dq.view(TOKENS, DIM), dk.view(TOKENS, DIM), kept,
                                               self.weight, dweight=self.grad, stream=stream)
        after()
        return y, h, kept.data, y8.values.view(torch.uint8), y8.scales, q, k, dq, dk, dx, dweight


SIZES = [TOKENS * DIM * 2, TOKENS * DIM, TOKENS * 5 * 132, TOKENS * 5 * 4, DIM * 4,
         rcc.rmsnorm_backward_workspace(TOKENS, DIM)]


def overwrite():
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in SIZES * 2]
    del held


@pytest.mark.parametrize("form", ["object", "address"])
def test_released_blocks_are_not_given_out_while_in_use(form):
    step = Step(121)
    want = [t.clone() for t in step.run()]
    step.grad.fill_(-1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    got = step.run(side if form == "object" else side.cuda_stream, after=overwrite)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_are_not_blocks_that_the_current_stream_still_writes():
    step = Step(122)
    want = [t.clone() for t in step.run()]
    step.grad.fill_(-1.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    overwrite()
    side = torch.cuda.Stream()
    got = step.run(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", [0, 1])
def test_adamw_on_a_stream(name):
    """A plan made and stepped on a side stream, and one on the default stream by
    its names while another is current: the same bits."""
    g = defs.gen(123)
    param, grad = defs.randn(g, 70001), defs.randn(g, 70001, dtype=BF16)
    cfg = rcc.adamw_cfg(max_grad_norm=1.0)
    plans = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, current in ((None, None), (side, None), (side.cuda_stream, None), (name, side)):
        p = param.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            plan = rcc.AdamWPlan([dict(param=p, grad=grad)], states=E4M3, stream=stream)
            for _ in range(3):
                rcc.adamw_step(plan, cfg, stream=stream)
            assert rcc.adamw_report(plan, stream=stream).step == 3
            assert torch.cuda.current_stream() == (current or torch.cuda.default_stream())
        plans.append((plan, p))
    torch.cuda.synchronize()
    first, p0 = plans[0]
    for plan, p in plans[1:]:
        assert torch.equal(p, p0)
        for k in ("exp_avg", "exp_avg_sq"):
            assert torch.equal(plan.tensors[0][k].view(torch.uint8),
                               first.tensors[0][k].view(torch.uint8))


def test_a_plan_is_not_made_while_capturing():
    p, g = torch.zeros(300, device=DEV), torch.zeros(300, device=DEV)
    plan = rcc.AdamWPlan([dict(param=p, grad=g)])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        with pytest.raises(rcc.RccError, match="capturing"):
            rcc.AdamWPlan([dict(param=p, grad=g, exp_avg=torch.empty_like(p),
                                exp_avg_sq=torch.empty_like(p))])
        rcc.adamw_step(plan, rcc.adamw_cfg())
    graph.replay()
    assert rcc.adamw_report(plan).step == 1


def test_calls_of_several_threads():
    """Threads with streams and plans of their own, at once."""
    g = defs.gen(124)
    work = []
    for i in range(4):
        n = 50000 + 777 * i
        work.append(dict(param=defs.randn(g, n), grad=defs.randn(g, n, dtype=BF16)))
    step = Step(125)
    cfg = rcc.adamw_cfg(max_grad_norm=1.0)

    def run(i, param, stream, out):
        plan = rcc.AdamWPlan([dict(param=param, grad=work[i]["grad"])], states=E4M3, seed=i,
                             stream=stream)
        for _ in range(20):
            rcc.adamw_step(plan, cfg, stream=stream)
            y, h = rcc.add_rmsnorm_forward(step.x, step.r, step.weight, stream=stream)
        q, _ = rcc.rotary_forward(y.view(TOKENS, HEADS, -1), None, step.turns, stream=stream)
        out[i] = (plan, y, h, q, rcc.adamw_report(plan, stream=stream).step)

    want, got = {}, {}
    alone = [w["param"].clone() for w in work]
    together = [w["param"].clone() for w in work]
    for i, p in enumerate(alone):
        run(i, p, None, want)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i, p, torch.cuda.Stream(), got))
               for i, p in enumerate(together)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 4
    for i in range(4):
        assert got[i][4] == want[i][4] == 20 and torch.equal(alone[i], together[i])
        assert all(torch.equal(a, b) for a, b in zip(got[i][1:4], want[i][1:4]))


def test_graphs_of_two_plans_in_turn():
    g = defs.gen(126)
    cfg = rcc.adamw_cfg(max_grad_norm=1.0)
    params = [defs.randn(g, 9000), defs.randn(g, 300)]
    grads = [defs.randn(g, p.numel()) for p in params]
    plain = [p.clone() for p in params]
    plans = [rcc.AdamWPlan([dict(param=p, grad=d)], states=E4M3) for p, d in zip(params, grads)]
    others = [rcc.AdamWPlan([dict(param=p, grad=d)], states=E4M3) for p, d in zip(plain, grads)]
    graphs = []
    torch.cuda.synchronize()
    for plan in plans:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rcc.adamw_step(plan, cfg)
        graphs.append(graph)
    for _ in range(5):
        for graph, other in zip(graphs, others):
            graph.replay()
            rcc.adamw_step(other, cfg)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(params, plain))
    assert [rcc.adamw_report(p).step for p in plans] == [5, 5]


@pytest.mark.parametrize("states", [torch.float32, E4M3])
@pytest.mark.parametrize("other", ["stream", "default", "handle"])
def test_a_plan_is_dropped_while_a_step_runs_on_another_stream(states, other):
    """Its workspace, and the states that it made, are not given out before the step
    is through."""
    n = 3 << 20   # blocks of their own in the allocator
    g = defs.gen(127)
    param, grad = defs.randn(g, n), defs.randn(g, n)
    want = param.clone()
    alone = rcc.AdamWPlan([dict(param=want, grad=grad)], states=states)
    rcc.adamw_step(alone, rcc.adamw_cfg())
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    made_on, run_on = (one, torch.cuda.default_stream()) if other == "default" else \
        (torch.cuda.default_stream(), two)
    plan = rcc.AdamWPlan([dict(param=param, grad=grad)], states=states, stream=made_on)
    held = [plan.workspace] + [plan.tensors[0][k] for k in ("exp_avg", "exp_avg_sq")]
    places = [(v.data_ptr(), v.data_ptr() + v.nbytes, v.nbytes) for v in held]
    del held
    torch.cuda.synchronize()
    with torch.cuda.stream(run_on):
        torch.cuda._sleep(DELAY)
    rcc.adamw_step(plan, rcc.adamw_cfg(),
                   stream=run_on.cuda_stream if other == "handle" else run_on)
    del plan
    with torch.cuda.stream(made_on):
        new = [torch.empty(size, dtype=torch.uint8, device=DEV) for _, _, size in places * 2]
    assert not run_on.query()   # the step is still to come
    for v in new:
        assert all(v.data_ptr() + v.nbytes <= lo or v.data_ptr() >= hi for lo, hi, _ in places)
    torch.cuda.synchronize()
    assert torch.equal(param, want)
