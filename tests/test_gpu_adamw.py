"""AdamW over many tensors, states in fp32 and in 8 bits, on the GPU.

With fp32 states the definition is restated here operation for operation, and
compared bit for bit.  With 8-bit states it is restated in 64 bits with the worst
rounding of each operation: what is held must lie between what the ends of that
interval are held as, by the same rounding numbers.  The norm is compared in 64
bits; where the gradients are clipped, the coefficient is that of the reported norm.
"""
import ctypes as C
import math

import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV, GUARD_BYTE, session

pytestmark = pytest.mark.gpu

U, F32, BF16, E4M3 = defs.U, defs.F32, defs.BF16, torch.float8_e4m3fn
WORD = 0xFFFFFFFF
CFG = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


# --------------------------------------------------------------- the definition

def stir(x):
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & WORD
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & WORD
    return x ^ (x >> 16)


def numbers_of(n, tensor, seed, step, start=0):
    """The 16 bits of the elements [start, start + n) of tensor `tensor`."""
    i = torch.arange(start, start + n, device=DEV)
    key = stir(torch.tensor(seed, device=DEV) ^ stir(torch.tensor(step & WORD, device=DEV)))
    key = stir((key + tensor * 0x9E3779B9) & WORD)
    h = stir((stir(key ^ (i // 4096)) + i % 4096 // 2) & WORD)
    return torch.where(i % 2 == 0, h & 0xFFFF, h >> 16)


def groups(x):
    n = x.numel()
    padded = torch.zeros(-(-n // 128) * 128, device=DEV, dtype=x.dtype)
    padded[:n] = x
    return padded.view(-1, 128)


def power_for(x):
    """The scales of x's groups: the smallest powers of two with max <= 448 s."""
    top = groups(x).abs().amax(1).double()
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)))
    return torch.where(top < 2.0 ** -100, 0.0, scale)


def rounded(x, scale, numbers, root):
    """What x / scale is held as, by the definition of the grid: rises with x."""
    n = x.numel()
    v, scale = groups(x).double(), scale[:, None].double()
    y = torch.where(scale > 0, v.abs() / torch.where(scale > 0, scale, 1.0), 0.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    w = (torch.floor(y / step + groups(numbers).double() / 65536) * step).clamp_max(448.0)
    if root:
        w = torch.where(y > 0, w.clamp_min(2.0 ** -9), 0.0)
    return torch.copysign(w, v).view(-1)[:n]


def held(x, numbers, root):
    """The bits and scales of a state to begin with."""
    scale = power_for(x)
    w = rounded(x, scale, numbers, root)
    return w.float().to(E4M3).view(torch.uint8), scale.float()


def const(v):
    """A number that the step takes in fp32."""
    return float(torch.tensor(v, dtype=F32))


def expected(t, tensor, cfg, scale, step, seed, coef, powers, start=0):
    """New param, states and scales of one tensor (or a part of it, from element
    `start` on).  fp32 states: the documented operations.  8 bits: each as what is
    the least and the most it may be."""
    b1, b2 = cfg["betas"]
    f = lambda v: torch.tensor(v, dtype=F32, device=DEV)  # noqa: E731
    n = t["param"].numel()
    size, root = const(cfg["lr"] / (1 - powers[0])), const(1 / math.sqrt(1 - powers[1]))
    decay, eps = const(1 - cfg["lr"] * cfg["weight_decay"]), const(cfg["eps"])
    if t["exp_avg"].dtype != E4M3:
        g = t["grad"].float() * f(1.0 / scale)
        g = g * f(coef)
        m = f(b1) * t["exp_avg"] + f(1 - b1) * g
        v = f(b2) * t["exp_avg_sq"] + f(1 - b2) * (g * g)
        p = t["param"] * f(decay) - f(size) * (m / (torch.sqrt(v) * f(root) + f(eps)))
        out = {"param": p, "exp_avg": m, "exp_avg_sq": v}
        return out | ({"copy": p.to(BF16)} if "copy" in t else {})
    # in 64 bits.  The gradient, its factor and the products each cost U: m is off
    # by 6 U of its two terms; v, all positive, by 6 U, sqrt(v) by half of that and
    # 2^-23 of the root itself
    g = t["grad"].double() * const(coef / scale)
    m0 = t["exp_avg"].double() * t["exp_avg_scale"].double().repeat_interleave(128)[:n]
    u0 = t["exp_avg_sq"].double() * t["exp_avg_sq_scale"].double().repeat_interleave(128)[:n]
    m = const(b1) * m0 + const(1 - b1) * g
    dm = 6 * U * (const(b1) * m0.abs() + const(1 - b1) * g.abs()) + 2.0 ** -149
    u = (const(b2) * u0 * u0 + const(1 - b2) * g * g).sqrt()
    du = 6 * U * u + 2.0 ** -70      # the root of the smallest fp32 numbers
    denom = u * root + eps
    # denominator: u's error, a product and a sum; its inverse 2 U; a product
    dp = size * (dm / denom + 14 * U * m.abs() / denom) * (1 + 16 * U)
    p = t["param"].double() * decay - size * m / denom
    dp = dp + 2 * U * (t["param"].double().abs() + p.abs()) + 2.0 ** -140
    numbers = numbers_of(n, tensor, seed, step, start)
    out = {"param": (p - dp, p + dp)}
    if "copy" in t:
        out["copy"] = ((p - dp).float().to(BF16).double(), (p + dp).float().to(BF16).double())
    for k, x, dx, is_root in (("exp_avg", m, dm, False), ("exp_avg_sq", u, du, True)):
        lo, hi = ((x - dx).clamp_min(0) if is_root else x - dx), x + dx
        near = torch.minimum(lo.abs(), hi.abs()) if not is_root else lo
        near = torch.where(lo * hi < 0, 0.0, near)
        scales = [power_for(v) for v in (near, torch.maximum(lo.abs(), hi.abs()))]
        out[k + "_scale"] = tuple(scales)
        out[k] = (lo, hi, numbers, is_root)
    return out


def bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def same(tensors, want):
    for i, (t, w) in enumerate(zip(tensors, want)):
        for k, v in w.items():
            got = t[k]
            if isinstance(v, torch.Tensor):
                assert torch.equal(got, v), (i, k, int((got != v).sum()), got.numel())
                continue
            if len(v) == 4:      # held values, with the scale that the group has
                lo, hi, numbers, is_root = v
                # the sum with 2^-6 of a small value is rounded to fp32
                s = t[k + "_scale"].double()
                slack = (s * 2.0 ** -29).repeat_interleave(128)[:got.numel()]
                lo = (lo - slack).clamp_min(0) if is_root else lo - slack
                v = tuple(rounded(x, s, numbers, is_root) for x in (lo, hi + slack))
            wrong = ~((got.double() >= v[0]) & (got.double() <= v[1]))
            assert not wrong.any(), (i, k, int(wrong.sum()), got.numel(), got[wrong][:4],
                                     v[0][wrong][:4], v[1][wrong][:4])


class Powers:
    """The products of the betas, as the status has them."""

    def __init__(self, betas, step):
        self.betas, self.now = betas, [b ** step for b in betas]

    def next(self):
        self.now = [p * b for p, b in zip(self.now, self.betas)]
        return self.now


# ------------------------------------------------------------------------ inputs

def make(g, n, grad_type, eight, copy, fresh=False, offset=0):
    """A tensor of n elements with states of a run under way; `offset` elements
    off the buffers' boundaries."""
    def place(v):
        room = torch.zeros(v.numel() + offset, device=DEV, dtype=torch.uint8 if v.dtype == E4M3
                           else v.dtype)
        room = room.view(E4M3) if v.dtype == E4M3 else room
        bits(room)[offset:] = bits(v)
        return room[offset:]
    t = {"param": place(defs.randn(g, n, scale=0.02)),
         "grad": place(defs.randn(g, n, dtype=grad_type, scale=1.0))}
    if copy:
        t["copy"] = place(torch.zeros(n, device=DEV, dtype=BF16))
    if fresh:
        return t
    m = defs.randn(g, n, scale=3e-4)
    u = defs.randn(g, n, scale=3e-4).add_(1e-3).abs_()
    if not eight:
        return t | {"exp_avg": place(m), "exp_avg_sq": place(u * u)}
    numbers = torch.zeros(n, dtype=torch.int64, device=DEV)
    for k, v, root in (("exp_avg", m, False), ("exp_avg_sq", u, True)):
        q, s = held(v, numbers, root)
        t[k], t[k + "_scale"] = place(q.view(E4M3)), place(s)
    return t


SIZES = [1, 2, 7, 127, 128, 129, 255, 1000, 4095, 4096, 4097, 8192, 20001, 300000]


def clone(tensors):
    return [{k: bits(v).clone().view(v.dtype) if v.dtype == E4M3 else v.clone()
             for k, v in t.items()} for t in tensors]


# ------------------------------------------------------------------------- tests

@pytest.mark.parametrize("grad_type", [F32, BF16])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 4, 8, 16])
def test_steps(grad_type, eight, copy, offset):
    g = defs.gen(81)
    tensors = [make(g, n, grad_type, eight, copy, offset=offset) for n in SIZES]
    for t in tensors[3:6]:
        t["grad"].zero_()
    seed, step, scale = 0xDEADBEEF, 41, 1024.0
    plan = rcc.AdamWPlan(tensors, seed=seed, step=step, betas=CFG["betas"])
    powers = Powers(CFG["betas"], step)
    cfg = rcc.adamw_cfg(max_grad_norm=0.0, **CFG)
    for k in range(3):
        now = powers.next()
        want = [expected(t, i, CFG, scale, step + k, seed, 1.0, now)
                for i, t in enumerate(tensors)]
        rcc.adamw_step(plan, cfg, scale)
        same(tensors, want)
        r = rcc.adamw_report(plan)
        assert (r.step, r.skipped, r.nonfinite, r.clip_coef) == (step + k + 1, 0, 0, 1.0)
        norm = math.sqrt(sum(float(t["grad"].double().square().sum()) for t in tensors)) / scale
        assert abs(r.grad_norm - norm) <= 1e-12 * norm
        assert float(plan.grad_norm) == r.grad_norm
        assert [r.beta1_power, r.beta2_power] == now
        for t in tensors:
            t["grad"].mul_(-0.3)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("scale", [1.0, 3.0, 65536.0])
def test_clipping(eight, scale):
    g = defs.gen(82)
    tensors = [make(g, n, F32, eight, False) for n in (5000, 300)]
    plan = rcc.AdamWPlan(tensors, seed=5, step=0)
    norm = math.sqrt(sum(float(t["grad"].double().square().sum()) for t in tensors)) / scale
    powers = Powers(CFG["betas"], 0)
    for k, limit in enumerate((0.5 * norm, norm * (1 - 1e-6), 2 * norm)):
        now = powers.next()
        before = clone(tensors)
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=limit, **CFG), scale)
        r = rcc.adamw_report(plan)
        assert abs(r.grad_norm - norm) <= 1e-12 * norm
        coef = torch.tensor(limit / r.grad_norm if r.grad_norm > limit else 1.0,
                            dtype=torch.float64).float().item()
        assert r.clip_coef == coef and (coef < 1.0) == (limit < norm)
        same(tensors, [expected(t, i, CFG, scale, k, 5, coef, now)
                       for i, t in enumerate(before)])


@pytest.mark.parametrize("grad_type", [F32, BF16])
def test_the_update_of_grad_sync(grad_type):
    """fp32 states: the same bits as rcc_grad_sync_adamw's of one rank."""
    g = defs.gen(83)
    tensors = [make(g, n, grad_type, False, True, fresh=True) for n in (1000, 4099, 70000)]
    other = [dict(grads=[t["grad"].float()], params=[t["param"].clone()],
                  exp_avg=[torch.zeros_like(t["param"])],
                  exp_avg_sq=[torch.zeros_like(t["param"])]) for t in tensors]
    plan = rcc.AdamWPlan(tensors)
    cfg = rcc.adamw_cfg(max_grad_norm=0.0, **CFG)
    state = rcc.optim_state(scale=256.0)
    with session(1) as comm:
        for _ in range(4):
            rcc.adamw_step(plan, cfg, 256.0)
            rcc.grad_sync_adamw(comm, rcc.ParamSets(other), cfg, state)
        torch.cuda.synchronize()
    for t, o in zip(plan.tensors, other):
        assert torch.equal(t["param"], o["params"][0])
        assert torch.equal(t["exp_avg"], o["exp_avg"][0])
        assert torch.equal(t["exp_avg_sq"], o["exp_avg_sq"][0])
        assert torch.equal(t["copy"], t["param"].to(BF16))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_gradient_that_is_not_finite_skips_the_step(eight, bad):
    g = defs.gen(84)
    tensors = [make(g, n, kind, eight, True) for n, kind in ((5000, F32), (131, BF16), (9000, BF16))]
    plan = rcc.AdamWPlan(tensors, step=3)
    good = tensors[1]["grad"].clone()
    tensors[1]["grad"][130] = bad
    tensors[2]["grad"][4096:4100] = bad
    before = clone(tensors)
    cfg = rcc.adamw_cfg(**CFG)
    rcc.adamw_step(plan, cfg)
    r = rcc.adamw_report(plan)
    assert (r.skipped, r.nonfinite, r.step) == (1, 5, 3)
    for t, b in zip(tensors, before):
        assert all(torch.equal(bits(t[k]).view(torch.uint8), bits(b[k]).view(torch.uint8)) for k in t)
    tensors[1]["grad"].copy_(good)
    tensors[2]["grad"][4096:4100] = 1.0
    rcc.adamw_step(plan, cfg)
    r = rcc.adamw_report(plan)
    assert (r.skipped, r.nonfinite, r.step) == (0, 0, 4)


def test_norms_of_any_size():
    """Squares that fp32 cannot hold count; a group of zeros does not."""
    for kind in (F32, BF16):
        for value in (1e30, 1e-30, 1e-38, 3e38, 1e-3):
            n = 10000
            t = make(defs.gen(85), n, kind, False, False)
            t["grad"].zero_()
            t["grad"][::7] = value
            plan = rcc.AdamWPlan([t])
            rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=1.0, **CFG))
            r = rcc.adamw_report(plan)
            want = float(t["grad"].double().norm())
            assert r.skipped == 0 and abs(r.grad_norm - want) <= 1e-12 * want
        # large and small together: the small ones are not lost beside each other
        t["grad"].fill_(1e-4)
        t["grad"][5] = 1.0
        plan = rcc.AdamWPlan([t])
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=1.0, **CFG))
        want = float(t["grad"].double().norm())
        assert abs(rcc.adamw_report(plan).grad_norm - want) <= 1e-12 * want
        t["grad"].zero_()
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=1.0, **CFG))
        assert rcc.adamw_report(plan).grad_norm == 0.0


def test_guards():
    """A step writes its buffers and nothing beside them."""
    g = defs.gen(86)
    for eight in (False, True):
        for n in (1, 129, 4097, 10000):
            for offset in (0, 3):
                rooms, t = {}, {}
                for k, v in make(g, n, BF16, eight, True).items():
                    size = v.element_size()
                    raw = torch.full((4096 + (offset + v.numel()) * size + 4096,), GUARD_BYTE,
                                     dtype=torch.uint8, device=DEV)
                    lo = 4096 + offset * size
                    part = raw[lo:lo + v.numel() * size]
                    part.copy_(v.view(torch.uint8))
                    rooms[k], t[k] = (raw, lo, part.numel()), part.view(v.dtype)
                plan = rcc.AdamWPlan([t])
                grad = t["grad"].clone()
                rcc.adamw_step(plan, rcc.adamw_cfg(**CFG))
                torch.cuda.synchronize()
                for k, (raw, lo, size) in rooms.items():
                    assert bool((raw[:lo] == GUARD_BYTE).all()), k
                    assert bool((raw[lo + size:] == GUARD_BYTE).all()), k
                assert torch.equal(t["grad"], grad)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kinds", [(F32, BF16, BF16), (BF16, BF16, BF16), (F32, F32, F32)])
def test_many_pieces(eight, kinds):
    """Blocks take whole pieces and edges of several tensors, of one or both types."""
    g = defs.gen(91)
    sizes = [2048 * 700, 5, 2048, 4096 * 300 + 17, 100, 2049, 6144, 4096, 2047] * 2
    tensors = [make(g, n, kinds[i % 3], eight, i % 2 == 1, offset=2 if i == 6 else 0)
               for i, n in enumerate(sizes)]
    plan = rcc.AdamWPlan(tensors, seed=3, step=1)
    powers = Powers(CFG["betas"], 1)
    for k in range(2):
        now = powers.next()
        want = [expected(t, i, CFG, 1.0, 1 + k, 3, 1.0, now) for i, t in enumerate(tensors)]
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=0.0, **CFG))
        same(tensors, want)


def test_thousands_of_tensors():
    g = defs.gen(87)
    sizes = [1 + (i * i * 31) % 700 for i in range(2500)]
    tensors = [make(g, n, BF16 if i % 3 else F32, False, i % 2 == 0) for i, n in enumerate(sizes)]
    plan = rcc.AdamWPlan(tensors, step=1)
    powers = Powers(CFG["betas"], 1).next()
    want = [expected(t, i, CFG, 1.0, 1, 0, 1.0, powers) for i, t in enumerate(tensors)]
    rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=0.0, **CFG))
    same(tensors, want)


@pytest.mark.parametrize("beta2,steps", [(0.999, 400), (0.95, 20)])
def test_held_moments_follow_small_changes(beta2, steps):
    """Without gradients sqrt(v) falls by a factor of sqrt(beta2) a step, far less
    than a step of the grid: rounded to nearest it would stay.  Each rounding is
    right on average, with a variance of at most a quarter of a step squared
    (a step is at most 1/8 of a value, here up to 2^-4 of a scale off), so the
    mean over n elements and the steps is within 8 standard deviations of
    sqrt(steps / n) / 16 of a value; a chance of 16 bits is 2^-17 of a step off."""
    n = 1 << 18
    g = defs.gen(88)
    t = make(g, n, BF16, True, False)
    u0 = torch.rand(n, generator=g, device=DEV) + 1.0
    zero = torch.zeros(n, dtype=torch.int64, device=DEV)
    q, s = held(u0, zero, True)
    t["exp_avg_sq"], t["exp_avg_sq_scale"] = q.view(E4M3), s
    t["grad"].zero_()
    plan = rcc.AdamWPlan([t], seed=9)
    start = (t["exp_avg_sq"].double() * s.double().repeat_interleave(128)).mean()
    cfg = rcc.adamw_cfg(betas=(0.9, beta2), max_grad_norm=0.0, lr=0.0, weight_decay=0.0)
    param = t["param"].clone()
    for _ in range(steps):
        rcc.adamw_step(plan, cfg)
    end = (t["exp_avg_sq"].double() *
           t["exp_avg_sq_scale"].double().repeat_interleave(128)).mean()
    want = beta2 ** (steps / 2)
    assert abs(float(end / start) - want) <= 8 * math.sqrt(steps / n) / 16 + steps * 2.0 ** -20
    assert torch.equal(t["param"], param)


def test_small_and_extreme_moments():
    """Next to nothing is held as zeros, a root above zero is not, the largest fp32
    saturates."""
    n = 512
    t = {"param": torch.zeros(n, device=DEV), "grad": torch.zeros(n, device=DEV)}
    t["grad"][:128] = 1e-32            # moments below 2^-100
    t["grad"][128:256] = 1e-12
    t["grad"][128] = 1.0               # 2^-40 of the largest: below the grid
    t["grad"][256:384] = 3e38
    plan = rcc.AdamWPlan([t], states=E4M3)
    rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=0.0, lr=1e-3, weight_decay=0.0))
    t = plan.tensors[0]
    u = t["exp_avg_sq"].float()
    assert not u[:128].any() and t["exp_avg_sq_scale"][0] == 0 and t["exp_avg_scale"][0] == 0
    assert bool((u[129:256] == 2.0 ** -9).all()) and 224 < float(u[128]) <= 448
    assert bool(torch.isfinite(t["exp_avg_scale"]).all()) and not u[384:].any()
    assert bool((u[256:384] == 448).all())       # v overflows: sqrt(v) is held as the largest
    assert bool(torch.isfinite(t["param"]).all())


def test_captured_steps_and_resuming():
    """Replays are steps; states saved with their step go on with the same bits."""
    g = defs.gen(89)
    tensors = [make(g, n, BF16, True, True) for n in (5000, 70000)]
    twin, third = clone(tensors), clone(tensors)
    cfg = rcc.adamw_cfg(**CFG)
    plan = rcc.AdamWPlan(tensors, seed=7, step=10)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rcc.adamw_step(plan, cfg, 8.0)
    for _ in range(4):
        graph.replay()
    other = rcc.AdamWPlan(twin, seed=7, step=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        rcc.adamw_step(other, cfg, 8.0, stream=side)
    side.synchronize()
    assert rcc.adamw_report(plan).step == 14 and rcc.adamw_report(other, stream=side).step == 14

    def equal(a, b):
        assert all(torch.equal(bits(x[k]).view(torch.uint8), bits(y[k]).view(torch.uint8))
                   for x, y in zip(a, b) for k in x)
    equal(tensors, twin)
    first = rcc.AdamWPlan(third, seed=7, step=10)
    for _ in range(2):
        rcc.adamw_step(first, cfg, 8.0)
    saved = clone(first.tensors)
    step = rcc.adamw_report(first).step
    del first
    second = rcc.AdamWPlan(saved, seed=7, step=step, betas=CFG["betas"])
    for _ in range(2):
        rcc.adamw_step(second, cfg, 8.0)
    equal(saved, tensors)


def test_shared_gradients_and_fresh_states():
    """Tensors may read one gradient; states that are left out begin as zeros."""
    g = defs.gen(90)
    grad = defs.randn(g, 3000, scale=0.1)
    p = defs.randn(g, 3000)
    for states in (F32, E4M3):
        plan = rcc.AdamWPlan([dict(param=p.clone(), grad=grad), dict(param=p.clone(), grad=grad)],
                             states=states)
        assert plan.tensors[0]["exp_avg"].dtype == states
        before = clone(plan.tensors)
        rcc.adamw_step(plan, rcc.adamw_cfg(max_grad_norm=0.0, **CFG))
        now = Powers(CFG["betas"], 0).next()
        same(plan.tensors, [expected(t, i, CFG, 1.0, 0, 0, 1.0, now) for i, t in enumerate(before)])
        assert torch.equal(plan.tensors[0]["param"], plan.tensors[1]["param"])


def test_refusals_on_the_gpu():
    p, g = torch.zeros(300, device=DEV), torch.zeros(300, device=DEV)
    with pytest.raises(rcc.RccError):
        rcc.AdamWPlan([dict(param=p, grad=p)])
    with pytest.raises(rcc.RccError):
        rcc.AdamWPlan([dict(param=p, grad=g), dict(param=p[100:], grad=g[100:])])
    with pytest.raises(rcc.RccError):
        rcc.AdamWPlan([dict(param=p, grad=g)], step=-1)
    with pytest.raises(ValueError):
        rcc.AdamWPlan([dict(param=p, grad=g, copy=torch.zeros(300, dtype=BF16))])
    plan = rcc.AdamWPlan([dict(param=p, grad=g)])
    for bad in (dict(replicas=2), dict(flags=rcc.ADAMW_GRAPH), dict(lr=-1.0), dict(eps=0.0),
                dict(eps=1e-60), dict(betas=(1.0, 0.9)), dict(max_grad_norm=float("nan"))):
        with pytest.raises(rcc.RccError):
            rcc.adamw_step(plan, rcc.adamw_cfg(**bad))
    for scale in (0.0, float("inf"), -1.0):
        with pytest.raises(rcc.RccError):
            rcc.adamw_step(plan, rcc.adamw_cfg(), scale)
    rcc.adamw_step(plan, rcc.adamw_cfg())
    assert rcc.adamw_report(plan).step == 1
    handle = plan.handle
    del plan
    cfg = rcc.adamw_cfg()
    assert rcc.raw("rcc_adamw_step", handle, C.byref(cfg), 1.0, None) == rcc.ERR_MISSING_REGISTRATION


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("n", [100, 5000, 3000000])
def test_what_the_kernels_just_ahead_wrote(eight, n):
    """A step reads gradients, parameters and states that the work right ahead of it
    on the stream wrote, skipped steps between: the bits of a plan that waits."""
    g = defs.gen(92)
    tensors = [make(g, n, BF16, eight, True), make(g, 77, BF16, eight, True)]
    twin = clone(tensors)
    plan, other = rcc.AdamWPlan(tensors, seed=1), rcc.AdamWPlan(twin, seed=1)
    cfg = rcc.adamw_cfg(max_grad_norm=1.0)
    draws = [[defs.randn(g, t["grad"].numel(), dtype=BF16) for t in tensors] for _ in range(5)]
    draws[3][1][5] = float("nan")

    def before(tensors, k):
        for t, d in zip(tensors, draws[k % 5]):
            t["grad"].copy_(d)
            t["param"].mul_(0.999)
            bits(t["exp_avg"]).copy_(bits(t["exp_avg"]).clone())
    torch.cuda.synchronize()
    for k in range(40):
        before(tensors, k)
        rcc.adamw_step(plan, cfg)
    for k in range(40):
        before(twin, k)
        torch.cuda.synchronize()
        rcc.adamw_step(other, cfg)
        torch.cuda.synchronize()
    assert rcc.adamw_report(plan).step == rcc.adamw_report(other).step == 32
    for a, b in zip(tensors, twin):
        assert all(torch.equal(bits(a[k]).view(torch.uint8), bits(b[k]).view(torch.uint8)) for k in a)
