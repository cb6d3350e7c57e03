"""The residual RMS norm, rotary positions and AdamW on more than 2^31 elements:
offsets that pass 32 bits.  Both ends are compared with the definitions."""
import pytest
import torch

import test_gpu_adamw as adam
import test_gpu_lm as defs
import test_gpu_rotary as rotary
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = defs.F32, defs.BF16, torch.float8_e4m3fn
ROWS, DIM = 530000, 4096   # 2.17e9 elements


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    assert ROWS * DIM > 1 << 31
    yield
    torch.cuda.empty_cache()


def large(seed):
    t = torch.full((ROWS, DIM), 0.25, dtype=BF16, device=DEV)
    g = defs.gen(seed)
    for part in (t[:600], t[-600:]):
        part.copy_(defs.randn(g, 600, DIM))
    return t


def test_residual_norm():
    x, r, weight = large(111), large(112), 1.0 + defs.randn(defs.gen(113), DIM, scale=0.2)
    y, h, kept = rcc.add_rmsnorm_forward(x, r, weight, keep=True)
    y8, _ = rcc.add_rmsnorm_forward(x, r, weight, out_dtype=E4M3)
    dx, _ = rcc.add_rmsnorm_backward(x, r, kept, weight)
    for rows in (slice(0, 500), slice(ROWS - 500, ROWS)):   # a row's bits are its own
        ys, hs, ks = rcc.add_rmsnorm_forward(x[rows], r[rows], weight, keep=True)
        es, _ = rcc.add_rmsnorm_forward(x[rows], r[rows], weight, out_dtype=E4M3)
        assert torch.equal(y[rows], ys) and torch.equal(h[rows], hs)
        assert torch.equal(kept.values[rows], ks.values)
        assert torch.equal(kept.scales[rows], ks.scales)
        assert torch.equal(y8.values[rows].view(torch.uint8), es.values.view(torch.uint8))
        assert torch.equal(y8.scales[rows], es.scales)
        assert torch.equal(dx[rows], rcc.add_rmsnorm_backward(x[rows], r[rows], ks, weight)[0])


@pytest.mark.parametrize("heads_first", [False, True])
def test_rotary(heads_first):
    flat = large(114)
    q = flat.view(32, ROWS, 128).transpose(0, 1) if heads_first else flat.view(ROWS, 32, 128)
    turns = rcc.rotary_turns(128, device=DEV)
    ends = [slice(0, 300), slice(ROWS - 300, ROWS)]
    before = [q[s].clone() for s in ends]
    out = torch.empty_like(flat).view(ROWS, 32, 128)
    rcc.rotary_forward(q, None, turns, offset=7, q_out=out)
    rcc.rotary_forward(q, None, turns, offset=7, q_out=q)
    for s, b in zip(ends, before):
        rotary.check(out[s], b, turns, range(7 + s.start, 7 + s.stop))
        assert torch.equal(q[s], out[s])


@pytest.mark.parametrize("states", [F32, E4M3])
def test_adamw(states):
    n = (1 << 31) + 70001
    ends = [slice(0, 12288), slice(n // 4096 * 4096 - 8192, n)]
    t = {"param": torch.zeros(n, device=DEV), "grad": torch.zeros(n, dtype=BF16, device=DEV),
         "copy": torch.ones(n, dtype=BF16, device=DEV)}
    g = defs.gen(115)
    for s in ends:
        t["param"][s] = defs.randn(g, s.stop - s.start, scale=0.02)
        t["grad"][s] = defs.randn(g, s.stop - s.start, dtype=BF16)
    plan = rcc.AdamWPlan([dict(param=t["param"][:100].clone(), grad=t["grad"][:100].clone()), t],
                         states=states, seed=77)
    t = plan.tensors[1]
    powers = adam.Powers(adam.CFG["betas"], 0)
    for step in range(2):
        parts = []
        for s in ends:
            part = {k: v[s.start // 128:-(-s.stop // 128)].clone() if k.endswith("scale") else
                    adam.bits(v[s]).clone().view(v.dtype) for k, v in t.items()}
            parts.append(part)
        now = powers.next()
        want = [adam.expected(p, 1, adam.CFG, 1.0, step, 77, 1.0, now, start=s.start)
                for p, s in zip(parts, ends)]
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=0.0, **adam.CFG))
        got = [{k: v[s.start // 128:-(-s.stop // 128)] if k.endswith("scale") else v[s]
                for k, v in t.items()} for s in ends]
        adam.same(got, want)
    norm = float(sum(t["grad"][s].double().square().sum() for s in ends).sqrt())
    small = float(plan.tensors[0]["grad"].double().square().sum())
    r = rcc.adamw_report(plan)
    assert abs(r.grad_norm ** 2 - norm ** 2 - small) <= 1e-10 * norm ** 2
    middle = slice(1 << 20, (1 << 20) + 1000)
    assert not t["param"][middle].any() and not t["copy"][middle].any()
