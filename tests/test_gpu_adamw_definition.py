"""AdamW with 8-bit states against its definition in fp32, operation for operation:
parameters, copies, held bytes and scales are its bits, over many steps that begin
once and go on from the definition's own states.
"""
import math

import pytest
import torch

import test_gpu_adamw as adamw
import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = defs.F32, defs.BF16, torch.float8_e4m3fn
CFG = adamw.CFG


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def f32(v):
    return torch.tensor(v, dtype=F32, device=DEV)


def hold(x, numbers, root):
    """The bytes and scales of x (fp32): the documented 32-bit operations.  `numbers`:
    [groups, 128]."""
    n = x.numel()
    v = adamw.groups(x)
    top = v.abs().amax(1).view(torch.int32)
    # the smallest power of two with max <= 448 s: 448 is 1.75 2^8
    scale = (((top + 0x1FFFFF) & 0x7F800000) - (8 << 23)).view(F32)
    scale = torch.where(top.view(F32) < 2.0 ** -100, 0.0, scale)
    inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
    y = v.abs() * inverse[:, None]
    low = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)
    bits = ((y + low).view(torch.int32) + numbers * 16) & -0x100000
    w = (bits.view(F32) - low).clamp(max=448.0)
    if root:
        w = torch.where(y > 0, w.clamp(min=2.0 ** -9), 0.0)
    w = torch.copysign(w, v).view(-1)[:n].to(E4M3)
    return w.view(torch.uint8), scale


def step_of(t, numbers, cfg, scale, coef, powers):
    """One step of a tensor in place: every line one operation rounded to fp32."""
    n = t["param"].numel()
    b1, b2 = cfg["betas"]
    g = t["grad"].float() * f32(1.0 / scale)
    g = g * f32(coef)
    wide = lambda k: t[k].view(E4M3).float() * t[k + "_scale"].repeat_interleave(128)[:n]  # noqa: E731
    m, u = wide("exp_avg"), wide("exp_avg_sq")
    m = f32(b1) * m + f32(1 - b1) * g
    v = f32(b2) * (u * u) + f32(1 - b2) * (g * g)
    u = torch.sqrt(v)
    size, root = f32(cfg["lr"] / (1 - powers[0])), f32(1 / math.sqrt(1 - powers[1]))
    p = t["param"] * f32(1 - cfg["lr"] * cfg["weight_decay"])
    p = p - size * (m / (u * root + f32(cfg["eps"])))
    t["param"] = p
    if "copy" in t:
        t["copy"] = p.to(BF16)
    t["exp_avg"], t["exp_avg_scale"] = hold(m, numbers, False)
    t["exp_avg_sq"], t["exp_avg_sq_scale"] = hold(u, numbers, True)


def raw(v):
    return v.contiguous().view(torch.uint8)


def follow(tensors, steps, limit, scale, seed=0x12345678, first=40, **more):
    """Steps of a plan and of the definition, side by side."""
    own = [dict(t) for t in adamw.clone(tensors)]
    settings = CFG | more
    plan = rcc.AdamWPlan(tensors, seed=seed, step=first, betas=settings["betas"])
    powers = adamw.Powers(settings["betas"], first)
    cfg = rcc.adamw_cfg(max_grad_norm=limit, **settings)
    for k in range(steps):
        rcc.adamw_step(plan, cfg, scale)
        r = rcc.adamw_report(plan)
        norm = math.sqrt(sum(float(t["grad"].double().square().sum()) for t in own)) / scale
        assert abs(r.grad_norm - norm) <= 1e-12 * norm and (r.clip_coef < 1) == (0 < limit < norm)
        now = powers.next()
        for i, t in enumerate(own):
            numbers = adamw.numbers_of(t["param"].numel(), i, seed, first + k)
            step_of(t, adamw.groups(numbers).int(), settings, scale, r.clip_coef, now)
        for i, (got, want) in enumerate(zip(tensors, own)):
            for key, v in want.items():
                wrong = raw(got[key]) != raw(v)
                assert not wrong.any(), (k, i, key, int(wrong.sum()), v.numel())
        for t, o in zip(tensors, own):   # other gradients, the same for both
            new = (t["grad"].float().roll(1) * -0.7).to(t["grad"].dtype)
            t["grad"].copy_(new)
            o["grad"] = new


def heavy(g, t):
    """Gradients of groups of very different sizes, rows without any, single large ones."""
    n = t["grad"].numel()
    size = torch.exp(2.0 * defs.randn(g, -(-n // 128)))
    size *= torch.rand(size.numel(), generator=g, device=DEV) > 0.1
    grad = t["grad"].float() * size.repeat_interleave(128)[:n]
    grad[:: 97] *= 50.0
    t["grad"].copy_(grad.to(t["grad"].dtype))
    return t


@pytest.mark.parametrize("kinds,offset,limit,scale", [
    ((F32,), 0, 1.0, 1024.0), ((BF16,), 0, 0.7, 3.0), ((F32, BF16), 0, 0.0, 1.0),
    ((F32,), 1, 0.7, 3.0), ((BF16,), 1, 0.0, 1.0), ((F32, BF16), 8, 1.0, 1024.0)])
def test_bits_of_many_steps(kinds, offset, limit, scale):
    g = defs.gen(201)
    tensors = [heavy(g, adamw.make(g, n, kinds[i % len(kinds)], True, i % 2 == 0, offset=offset))
               for i, n in enumerate(adamw.SIZES)]
    follow(tensors, 12, limit, scale)


@pytest.mark.parametrize("kind", [F32, BF16])
def test_bits_of_a_thousand_tensors(kind):
    """1,024 tensors of 1 to 40,000 elements and one of four million, as parts of flat
    buffers (zeros between them), which the definition steps over as a whole."""
    g = defs.gen(202)
    sizes = [1 + (i * i * 977) % 40000 for i in range(1024)] + [1 << 22]
    many = [-(-n // 128) for n in sizes]
    first = [sum(many[:i]) for i in range(len(many))]
    owner = torch.repeat_interleave(torch.arange(len(many)), torch.tensor(many)).to(DEV)
    inside = torch.arange(sum(many), device=DEV) - torch.tensor(first, device=DEV)[owner]
    at = inside[:, None] * 128 + torch.arange(128, device=DEV)
    live = (at < torch.tensor(sizes, device=DEV)[owner][:, None]).view(-1)
    flat = heavy(g, adamw.make(g, 128 * sum(many), kind, True, True))
    for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
        adamw.bits(flat[k])[~live] = 0
    tensors = []
    for n, f, m in zip(sizes, first, many):
        t = {k: v[f:f + m] if "scale" in k else v[128 * f:128 * f + n] for k, v in flat.items()}
        tensors.append(t)
    own = adamw.clone([flat])[0]
    seed, step, scale = 77, 5, 1024.0
    plan = rcc.AdamWPlan(tensors, seed=seed, step=step, betas=CFG["betas"])
    powers = adamw.Powers(CFG["betas"], step)
    for _ in range(10):
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=1.0, **CFG), scale)
        r = rcc.adamw_report(plan)
        assert 0 < r.clip_coef < 1
        key = adamw.stir(torch.tensor(seed, device=DEV) ^ adamw.stir(torch.tensor(step, device=DEV)))
        key = adamw.stir((key + owner * 0x9E3779B9) & adamw.WORD)[:, None]
        h = adamw.stir((adamw.stir(key ^ (at // 4096)) + at % 4096 // 2) & adamw.WORD)
        numbers = torch.where(at % 2 == 0, h & 0xFFFF, h >> 16).int()
        step_of(own, numbers, CFG, scale, r.clip_coef, powers.next())
        for k, v in own.items():
            wrong = raw(flat[k]) != raw(v)
            assert not wrong.any(), (step, k, int(wrong.sum()))
        step += 1


def test_bits_of_extreme_values():
    """Moments and gradients near both ends of what fp32 has."""
    g = defs.gen(203)
    t = adamw.make(g, 128 * 40, F32, True, True)
    for i in range(40):
        t["grad"][128 * i:128 * (i + 1)] *= 2.0 ** (-140 + 6 * i)
    follow([t], 12, 0.0, 1.0)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("more", [dict(eps=1e-15), dict(eps=1e-20), dict(eps=2.0), dict(lr=1e-25),
                                  dict(lr=0.0), dict(betas=(0.0, 0.99999)), dict(betas=(0.9, 0.0)),
                                  dict(weight_decay=0.0)])
def test_bits_of_other_settings(offset, more):
    """Denominators, step sizes and moments on both sides of the range that is taken two
    at a time; first steps, where the corrections are largest."""
    g = defs.gen(204)
    tensors = [heavy(g, adamw.make(g, n, F32, True, True, offset=offset)) for n in (5000, 300, 4096)]
    tensors[0]["grad"][1000:3000] *= 2.0 ** 12
    tensors[0]["grad"][2000:4000:7] *= 2.0 ** 10
    follow(tensors, 6, 0.0, 1.0, first=0, **more)
