"""The tied-weight language model of examples/tied_lm.py: it learns its
successor table over several ranks, its tied gradient is the sum of both ends',
and a non-finite gradient skips the step."""
import importlib.util
import os
import re

import pytest
import torch

from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location(
        "tied_lm", os.path.join(ROOT, "examples", "tied_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_it_learns(example):
    losses, state = example.train(steps=60, ranks=2, say=lambda *a: None)
    # a uniform guess costs ln 1000 = 6.9
    assert losses[0] > 6.0 and losses[-1] < 0.5 * losses[0]
    assert state.step == 60


def test_the_tied_gradient_is_the_sum_of_both_ends(example):
    """Against automatic differentiation of the same model in 64 bits.  What
    separates the two: the activations are bf16 (2^-8), and the norm's backward
    pass reads its input in 8 bits, half a step of a group's largest value off
    (1/254 of it, here up to 4 times a value's size).  Each perturbs every term
    of the gradient by a few per cent at most, in random directions."""
    model = example.TiedLM(300, 64, 200, 1, seed=3)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    follow = torch.randperm(300, generator=g, device=DEV)
    ids, labels = example.batch(g, follow, 300, 200)
    loss, counted = model.forward_backward(0, ids, labels, model.table.bfloat16(), 1.0)
    table = model.table.double().requires_grad_()
    norm = model.norm.double().requires_grad_()
    h = torch.where((ids >= 0)[:, None], table[ids.clamp_min(0)] * 8.0, 0.0)
    y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * norm
    z = y @ table.t()
    each = torch.logsumexp(z, 1) - z.gather(1, labels.clamp_min(0)[:, None])[:, 0]
    want = (each * counted.double()).sum() / counted.sum()
    want.backward()
    assert abs(float((loss * counted).sum() / counted.sum() - want.detach())) < 0.02
    for got, exact in ((model.dtable[0], table.grad), (model.dnorm[0], norm.grad)):
        assert float((got.double() - exact).norm() / exact.norm()) < 0.03


def test_an_infinite_weight_skips_the_step(example):
    model = example.TiedLM(100, 64, 50, 2, seed=5)
    model.table[7, 3] = float("inf")
    before = model.table.clone()
    state = rcc.optim_state(scale=1024.0)
    ids = torch.arange(50, device=DEV)
    comm = rcc.register(0, 2, rcc.F32)
    try:
        _, report = model.step(comm, [(ids, (ids + 1) % 100)] * 2, rcc.adamw_cfg(), state)
    finally:
        rcc.finish(comm)
    assert report.skipped == 1 and report.nonfinite > 0 and state.step == 0
    assert state.scale == 512.0 and torch.equal(model.table, before)


def test_the_documented_calls_run():
    """The front page's example of the operators, as written."""
    text = open(os.path.join(ROOT, "README.md")).read()
    block = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "linear_ce" in b]
    assert len(block) == 1
    scope = {}
    exec(compile(block[0], "README.md", "exec"), scope)
    assert scope["dtable"].dtype == scope["dnorm"].dtype == torch.float32
    assert all(torch.isfinite(scope[n]).all() for n in ("loss", "dtable", "dnorm"))
    # 1,024 products of fp32: 2,048 roundings of 2^-24 of sum |y w|, near 20
    z = scope["y"].double() @ scope["w16"].double().t()
    want = torch.logsumexp(z, 1) - z.gather(1, scope["labels"][:, None])[:, 0]
    assert float((scope["loss"] - want).abs().max()) < 2.5e-3
