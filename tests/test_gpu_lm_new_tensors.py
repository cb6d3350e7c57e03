"""Tensors that the language-model operators make for a caller are seen by dispatch
modes and profilers, as torch's own are, and filled where deterministic runs ask for it."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TOKENS, DIM = 4, 256


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def calls():
    """Each call with the number of tensors that it makes, workspaces among them."""
    x = torch.randn(TOKENS, DIM, device=DEV)
    b, w = x.bfloat16(), torch.ones(DIM, device=DEV)
    ids = torch.zeros(TOKENS, dtype=torch.int64, device=DEV)
    _, kept = rcc.rmsnorm_forward(x, w, keep=True)
    turns = rcc.rotary_turns(64, device=DEV)
    q = x.view(TOKENS, 2, 128)
    _, lse = rcc.linear_ce_forward(b, b, ids)
    ones, table = torch.ones(TOKENS, device=DEV), torch.zeros(8, DIM, device=DEV)
    return [
        (1, lambda: rcc.embedding_forward(x, ids)),
        (1, lambda: rcc.embedding_backward(x, ids, table)),
        (1, lambda: rcc.rmsnorm_forward(x, w)),
        (2, lambda: rcc.rmsnorm_forward(x, w, keep=True)),
        (3, lambda: rcc.rmsnorm_backward(x, kept, w)),
        (3, lambda: rcc.add_rmsnorm_forward(x, x, w, keep=True)),
        (4, lambda: rcc.add_rmsnorm_forward(x, x, w, keep=True, out_dtype=torch.float8_e4m3fn)),
        (3, lambda: rcc.add_rmsnorm_backward(x, x, kept, w)),
        (2, lambda: rcc.rotary_forward(q, q, turns)),
        (3, lambda: rcc.linear_ce_forward(b, b, ids)),
        (3, lambda: rcc.linear_ce_backward(b, b, ids, lse, ones)),
    ]


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.made.append(out)
        return out


def test_dispatch_modes_see_them():
    for i, (many, call) in enumerate(calls()):
        with Seen() as seen:
            got = call()
        assert len(seen.made) == many, i
        got = [t for t in (got if isinstance(got, tuple) else (got,)) if isinstance(t, torch.Tensor)]
        made = {t.data_ptr() for t in seen.made}
        assert i == 1 or all(t.data_ptr() in made for t in got), i
        with Seen() as seen:      # and nothing once it is gone
            pass
        call()
        assert not seen.made


def test_profilers_see_them():
    many, call = calls()[6]
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        call()
    made = [e for e in prof.events() if e.name == "aten::empty"]
    assert len(made) >= many


def test_deterministic_runs_fill_them():
    """New memory is filled (with NaN, or the largest number) in front of the call: an
    operation more for each tensor, and the same results."""
    many, call = calls()[4]
    want = call()
    torch.use_deterministic_algorithms(True)
    try:
        with Seen() as seen:
            got = call()
    finally:
        torch.use_deterministic_algorithms(False)
    assert len(seen.made) == many
    assert all(torch.equal(a, b) for a, b in zip(got, want))
