"""The language-model operators' `stream` argument: calls on a stream that is
not the current one, with outputs and workspaces left out."""
import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = defs.F32, defs.BF16
VOCAB, DIM, TOKENS = 2500, 520, 900
DELAY = 20000000   # cycles, about 10 ms: everything queued behind it is still to come


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Step:
    """All six calls; `after` runs behind each of them."""

    def __init__(self, seed):
        g = defs.gen(seed)
        self.table = defs.randn(g, VOCAB, DIM, scale=0.3)
        self.weight = 1.0 + defs.randn(g, DIM, scale=0.1)
        self.ids = defs.skewed_ids(g, TOKENS, VOCAB)
        self.w16 = self.table.to(BF16)
        self.dloss = torch.full((TOKENS,), 1.0 / TOKENS, device=DEV)
        self.dtable = torch.empty(VOCAB, DIM, device=DEV)
        torch.cuda.synchronize()

    def run(self, stream=None, after=lambda: None):
        h = rcc.embedding_forward(self.table, self.ids, out_dtype=BF16, stream=stream)
        after()
        y, kept = rcc.rmsnorm_forward(h, self.weight, keep=True, stream=stream)
        after()
        loss, lse = rcc.linear_ce_forward(y, self.w16, self.ids, stream=stream)
        after()
        dy, dw = rcc.linear_ce_backward(y, self.w16, self.ids, lse, self.dloss, grad_dtype=F32,
                                        stream=stream)
        after()
        dh, dweight = rcc.rmsnorm_backward(dy, kept, self.weight, stream=stream)
        after()
        rcc.embedding_backward(dh, self.ids, self.dtable, stream=stream)
        after()
        return h, y, kept.data, loss, lse, dy, dw, dh, dweight, self.dtable


# every size that a call may take from the allocator
SIZES = sorted({TOKENS * DIM * 2, TOKENS * DIM * 4, VOCAB * DIM * 2, VOCAB * DIM * 4, TOKENS * 4,
                DIM * 4, TOKENS * 5 * 132})


def workspaces():
    return [rcc.embedding_backward_workspace(TOKENS, VOCAB, DIM),
            rcc.rmsnorm_backward_workspace(TOKENS, DIM),
            rcc.linear_ce_workspace(TOKENS, VOCAB, DIM),
            rcc.linear_ce_workspace(TOKENS, VOCAB, DIM, True, F32)]


def overwrite():
    """Takes and fills blocks of every size on the current stream."""
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in SIZES + workspaces()]
    del held


@pytest.mark.parametrize("form", ["object", "address"])
def test_released_workspaces_are_not_given_out_while_in_use(form):
    """The calls wait on `side` behind a delay; meanwhile the current stream
    allocates and overwrites whatever the allocator gives it."""
    step = Step(31)
    want = [t.clone() for t in step.run()]
    step.dtable.fill_(-1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    got = step.run(side if form == "object" else side.cuda_stream, after=overwrite)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_are_not_blocks_that_the_current_stream_still_writes():
    """Blocks are released while the current stream still has writes to them
    queued; the calls on `side` run at once."""
    step = Step(32)
    want = [t.clone() for t in step.run()]
    step.dtable.fill_(-1.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    overwrite()
    side = torch.cuda.Stream()
    got = step.run(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_do_not_share_a_workspace():
    steps = [Step(33), Step(34)]
    want = [[t.clone() for t in s.run()] for s in steps]
    for s in steps:
        s.dtable.fill_(-1.0)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in steps]
    for side in sides:
        with torch.cuda.stream(side):
            torch.cuda._sleep(DELAY)
    got = [s.run(side) for s, side in zip(steps, sides)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_the_default_streams_names():
    """0 and 1 name the default stream, also while another one is current."""
    step = Step(35)
    want = [t.clone() for t in step.run()]
    side = torch.cuda.Stream()
    for name in (0, 1, torch.cuda.default_stream()):
        step.dtable.fill_(-1.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = step.run(name)
            assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_refusal_leaves_the_current_stream():
    step, side = Step(36), torch.cuda.Stream()
    with pytest.raises(rcc.RccError):   # librcc refuses, with the stream already current
        rcc.rmsnorm_forward(step.table, step.weight, eps=-1.0, stream=side)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
