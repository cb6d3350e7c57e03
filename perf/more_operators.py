"""Cases of the operators between a language model's matrix products and at the
end of its training step: the residual addition with its RMS norm (output in the
input's type or in 8 bits, input kept in 8 bits for the backward pass), rotary
positions, and AdamW over many tensors with states in 8 bits or in 32.

`run` computes an operator in its plain form (elementary torch operations in 32
bits, rounded once at the end; angles and long sums in 64) or, where `own` is
true, through this repository's entry points.  `exact` restates the definitions
in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda:0"
EPS = 1e-6           # of the norm
COLUMNS = 128        # columns, or elements of a tensor, that share one scale
TINY = 2.0 ** -120   # a norm's group below this is held as zeros
NOTHING = 2.0 ** -100   # and so is an optimizer state's
E4M3 = torch.float8_e4m3fn
TOP = 448.0          # the largest e4m3 value
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# the optimizer's settings, as a training run has them
LR, BETAS, ADAM_EPS, DECAY, SCALE = 1e-3, (0.9, 0.999), 1e-8, 0.01, 1024.0
TAKEN = 100          # steps taken before
BLOCK = 4096         # elements whose rounding numbers share one key
WHOLE = 0xFFFFFFFF
MOST_ELEMENTS = 400000000   # of a drawn optimizer step


# ------------------------------------------------------------------- cases

def listed():
    return [
        # decoding: a few sequences' tokens, nothing kept
        {"name": "residual_few", "op": "residual", "tokens": 8, "dim": 4096, "act": "bf16",
         "eight": False},
        # a prompt on its way into 8-bit matrix products
        {"name": "residual_eight_batch", "op": "residual", "tokens": 16384, "dim": 4096,
         "act": "bf16", "eight": True},
        # a training micro-batch: forward, sum kept in 8 bits, backward
        {"name": "residual_step_batch", "op": "residual_step", "tokens": 16384, "dim": 4096,
         "act": "bf16", "eight": False},
        # a small fp32 model of odd sizes
        {"name": "residual_step_odd", "op": "residual_step", "tokens": 1023, "dim": 1000,
         "act": "f32", "eight": False},
        # decoding far into long contexts: one token of each sequence, shared key heads
        {"name": "rotary_few", "op": "rotary", "tokens": 8, "heads": 32, "key_heads": 8,
         "head_dim": 128, "turned": 128, "layout": "half", "scaling": "parts", "act": "bf16",
         "far": True},
        # a training micro-batch of packed documents: queries and keys, then their gradients
        {"name": "rotary_step_batch", "op": "rotary_step", "tokens": 16384, "heads": 32,
         "key_heads": 8, "head_dim": 128, "turned": 128, "layout": "half", "scaling": "none",
         "act": "bf16", "far": False},
        # neighbouring pairs, a part of an odd head, fp32
        {"name": "rotary_part_odd", "op": "rotary", "tokens": 2049, "heads": 12, "key_heads": 12,
         "head_dim": 80, "turned": 20, "layout": "interleaved", "scaling": "linear",
         "act": "f32", "far": False},
        # a small model's two tensors: a table of 1,000 x 128 and a norm
        {"name": "adamw_few", "op": "adamw", "tensors": 2, "least": 128, "most": 128000,
         "grad": "f32", "states": "f32", "copy": True, "clip": True},
        # tied table of 50,021 x 2,048 in one tensor, fp32 gradients, 8-bit states
        {"name": "adamw_one_eight", "op": "adamw", "tensors": 1, "least": 102443008,
         "most": 102443008, "grad": "f32", "states": "e4m3", "copy": False, "clip": True},
        # a model of 1,024 tensors, bf16 gradients and copies, 8-bit states
        {"name": "adamw_many_eight", "op": "adamw", "tensors": 1024, "least": 1024,
         "most": 4194304, "grad": "bf16", "states": "e4m3", "copy": True, "clip": True},
        # the same with fp32 gradients and states, not clipped
        {"name": "adamw_many_full", "op": "adamw", "tensors": 1024, "least": 1024,
         "most": 4194304, "grad": "f32", "states": "f32", "copy": False, "clip": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["residual", "residual_step", "rotary", "rotary_step", "adamw", "adamw"])
    act = rng.choice(["f32", "bf16"])
    if op in ("residual", "residual_step"):
        step = rng.choice([1, 8, 128])
        return {"op": op, "tokens": _log_uniform(rng, 1, 16384),
                "dim": max(64, _log_uniform(rng, 64, 8192) // step * step),
                "act": act, "eight": rng.random() < 0.5}
    if op in ("rotary", "rotary_step"):
        head_dim = rng.choice([64, 80, 96, 128, 256])
        key_heads = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log_uniform(rng, 1, 8192),
                "heads": key_heads * rng.choice([1, 2, 4]), "key_heads": key_heads,
                "head_dim": head_dim,
                "turned": rng.choice([head_dim, head_dim // 2, head_dim // 4]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "parts"]), "act": act,
                "far": rng.random() < 0.5}
    while True:
        tensors = _log_uniform(rng, 1, 1024)
        most = _log_uniform(rng, 1024, 50000000)
        case = {"op": op, "tensors": tensors, "least": _log_uniform(rng, 1, most), "most": most,
                "grad": act, "states": rng.choice(["f32", "e4m3"]), "copy": rng.random() < 0.5,
                "clip": rng.random() < 0.5}
        if sum(_sizes(case)) <= MOST_ELEMENTS:
            return case


def _sizes(case):
    """The tensors' elements: log-uniform, the largest and the smallest among them."""
    rng = random.Random(case["tensors"] * 1000003 + case["most"])
    n = [_log_uniform(rng, case["least"], case["most"]) for _ in range(case["tensors"])]
    n[0] = case["most"]
    if len(n) > 1:
        n[-1] = case["least"]
    return n


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _prepare_residual(case, g):
    t, dim, act = case["tokens"], case["dim"], TYPES[case["act"]]
    # a residual stream: a few columns far larger than the others; a layer's output to add
    stream = _randn(g, t, dim)
    stream *= torch.exp(0.5 * _randn(g, dim))
    stream[:, torch.randint(dim, (max(1, dim // 512),), generator=g, device=DEVICE)] *= 30.0
    return {"case": case, "residual": stream.to(act), "x": _randn(g, t, dim).mul_(0.3).to(act),
            "weight": 1.0 + 0.1 * _randn(g, dim),
            "dy": _randn(g, t, dim).mul_(1e-2).to(act),
            "dh": _randn(g, t, dim).mul_(1e-2).to(act)}


def _scaling(case):
    """How a context is stretched to longer ones."""
    return {"none": None, "linear": ("linear", 4.0), "base": ("base", 8.0),
            "parts": ("parts", 8.0, 8192, 1.0, 4.0)}[case["scaling"]]


def _prepare_rotary(case, g):
    t, hd, act = case["tokens"], case["head_dim"], TYPES[case["act"]]
    s = {"case": case}
    for name, heads in (("q", case["heads"]), ("k", case["key_heads"])):
        s[name] = _randn(g, t, heads, hd, dtype=act)
        s["d" + name] = _randn(g, t, heads, hd).mul_(1e-2).to(act)
    if case["far"]:     # tokens of contexts of up to a million
        s["positions"] = torch.randint(1 << 20, (t,), generator=g, device=DEVICE)
    else:               # documents one behind the other, each from 0
        starts = torch.rand(t, generator=g, device=DEVICE) < 1.0 / 700
        at = torch.arange(t, device=DEVICE)
        s["positions"] = (at - torch.cummax(torch.where(starts, at, 0), 0).values).int()
    if own:
        from gradient_sync_rcc_gb300 import rcc
        s["turns"] = rcc.rotary_turns(case["turned"], 10000.0, _scaling(case), device=DEVICE)
    return s


def _prepare_adamw(case, g, seed):
    """Flat buffers, each tensor on a boundary of 128 elements (zeros between)."""
    sizes = _sizes(case)
    groups = [-(-n // COLUMNS) for n in sizes]
    first = [0]
    for n in groups:
        first.append(first[-1] + n)
    total = first[-1]
    group = torch.arange(total, device=DEVICE)
    begin = torch.tensor(first[:-1], device=DEVICE)
    owner = torch.searchsorted(begin, group, right=True) - 1
    inside = group - begin[owner]           # a group's number within its tensor
    elements = torch.arange(COLUMNS, device=DEVICE)
    live = (inside[:, None] * COLUMNS + elements
            < torch.tensor(sizes, device=DEVICE)[owner][:, None])
    size = torch.exp(_randn(g, total, 1))   # how large a group's gradients are
    size *= torch.rand(total, 1, generator=g, device=DEVICE) > 0.05   # rows without any
    s = {"case": case, "seed": seed & WHOLE, "owner": owner, "inside": inside,
         "param": _randn(g, total, COLUMNS).mul_(0.02).mul_(live),
         "grad": (_randn(g, total, COLUMNS) * (1e-3 * SCALE) * size * live)
         .to(TYPES[case["grad"]])}
    avg = _randn(g, total, COLUMNS).mul_(3e-4).mul_(size).mul_(live)
    root = (_randn(g, total, COLUMNS).mul_(0.3).add_(1.0).abs_().mul_(1e-3)).mul_(size).mul_(live)
    if case["states"] == "f32":
        s["exp_avg"], s["exp_avg_sq"] = avg, root * root
    else:
        for name, v in (("exp_avg", avg), ("exp_avg_sq", root)):
            scale = _power(v.abs().amax(1))
            s[name] = (v / torch.where(scale > 0, scale, 1.0)[:, None]).to(E4M3)
            s[name + "_scale"] = scale
    if case["copy"]:
        s["copy"] = torch.zeros(total, COLUMNS, device=DEVICE, dtype=torch.bfloat16)
    s["step"] = torch.full((), TAKEN, device=DEVICE, dtype=torch.int64)
    if own:
        from gradient_sync_rcc_gb300 import rcc
        tensors = []
        for n, at, many in zip(sizes, first, groups):
            t = {k: s[k].view(-1)[at * COLUMNS:at * COLUMNS + n]
                 for k in ("param", "grad", "exp_avg", "exp_avg_sq", "copy") if k in s}
            for k in ("exp_avg_scale", "exp_avg_sq_scale"):
                if k in s:
                    t[k] = s[k][at:at + many]
            tensors.append(t)
        s["plan"] = rcc.AdamWPlan(tensors, seed=s["seed"], step=TAKEN, betas=BETAS)
        s["cfg"] = rcc.adamw_cfg(lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY,
                                 max_grad_norm=1.0 if case["clip"] else 0.0)
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"].startswith("residual"):
        return _prepare_residual(case, g)
    if case["op"].startswith("rotary"):
        return _prepare_rotary(case, g)
    return _prepare_adamw(case, g, seed)


# ------------------------------------------------------- plain: residual norm

def _grouped(x):
    """[tokens, groups of columns, 128], zeros past the row."""
    t, dim = x.shape
    many = -(-dim // COLUMNS)
    padded = torch.zeros(t, many * COLUMNS, device=x.device)
    padded[:, :dim] = x
    return padded.view(t, many, COLUMNS)


def _plain_kept(x):
    """What is left of x once it has been held in 8 bits: whole numbers in
    [-127, 127] and one scale for each group of columns."""
    v = _grouped(x.float())
    top = v.abs().amax(2, keepdim=True)
    small = top < TINY
    q = torch.round(v * torch.where(small, 0.0, 127.0 * (1.0 / top)))
    v = q * torch.where(small, 0.0, top * (1.0 / 127.0))
    return v.view(x.shape[0], -1)[:, :x.shape[1]]


def _plain_eight(y):
    """e4m3 values and one scale for each group of columns."""
    v = _grouped(y)
    top = v.abs().amax(2, keepdim=True)
    small = top < TINY
    v = v * torch.where(small, 0.0, TOP * (1.0 / top))
    v = v.clamp(-TOP, TOP).view(y.shape[0], -1)[:, :y.shape[1]].to(E4M3)
    return v.contiguous(), torch.where(small, 0.0, top * (1.0 / TOP))[:, :, 0]


def _plain_residual(s):
    act = s["x"].dtype
    h = (s["x"].float() + s["residual"].float()).to(act)
    v = h.float()
    r = torch.rsqrt(torch.mean(v * v, 1, keepdim=True) + EPS)
    y = v * r * s["weight"]
    out = {"h": h}
    if s["case"]["eight"]:
        out["y"], out["scales"] = _plain_eight(y)
    else:
        out["y"] = y.to(act)
    if s["case"]["op"] == "residual":
        return out
    v, dy = _plain_kept(h), s["dy"].float()
    r = torch.rsqrt(torch.mean(v * v, 1, keepdim=True) + EPS)
    n, d = v * r, dy * s["weight"]
    dx = s["dh"].float() + r * (d - n * torch.mean(d * n, 1, keepdim=True))
    out["dx"], out["dweight"] = dx.to(act), torch.sum(dy * n, 0)
    return out


# --------------------------------------------------------------- plain: rotary

def _frequencies(case):
    """Radians a position, in 64 bits."""
    n, scaling = case["turned"], _scaling(case)
    base = 10000.0
    if case["scaling"] == "base":     # the slowest pair slows down by the factor
        base *= scaling[1] ** (n / (n - 2))
    f = base ** (-torch.arange(0, n, 2, device=DEVICE, dtype=torch.float64) / n)
    if case["scaling"] == "linear":
        f = f / scaling[1]
    if case["scaling"] == "parts":    # by the turns within the length trained on
        _, factor, length, low, high = scaling
        keep = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f


def _plain_turned(x, cos, sin, case):
    n, v = case["turned"], x.float()
    out = v.clone()
    if case["layout"] == "half":
        a, b = v[:, :, :n // 2], v[:, :, n // 2:n]
        out[:, :, :n // 2], out[:, :, n // 2:n] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = v[:, :, 0:n:2], v[:, :, 1:n:2]
        out[:, :, 0:n:2], out[:, :, 1:n:2] = a * cos - b * sin, a * sin + b * cos
    return out.to(x.dtype)


def _plain_rotary(s):
    case = s["case"]
    angle = s["positions"].double()[:, None] * _frequencies(case)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {n: _plain_turned(s[n], cos, sin, case) for n in ("q", "k")}
    if case["op"] == "rotary_step":
        out |= {n: _plain_turned(s[n], cos, -sin, case) for n in ("dq", "dk")}
    return out


# ---------------------------------------------------------------- plain: AdamW

def _power(top):
    """The smallest power of two s with top <= 448 s; 0 for next to nothing."""
    bits = top.view(torch.int32)
    s = (((bits + 0x1FFFFF) & 0x7F800000) - (8 << 23)).view(torch.float32)
    return torch.where(top < NOTHING, 0.0, s)


def _mix(x):
    """32 bits of x (in 64) stirred: shifts, and products with fractions of roots."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & WHOLE
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & WHOLE
    return x ^ (x >> 16)


def _rounding_numbers(s):
    """16 bits for each element: by seed, step, tensor, block of 4,096 and pair."""
    key = _mix(s["seed"] ^ _mix(s["step"] & WHOLE))
    key = _mix((key + s["owner"] * 0x9E3779B9) & WHOLE)
    key = _mix(key ^ (s["inside"] // (BLOCK // COLUMNS)))
    pair = torch.arange(COLUMNS // 2, device=DEVICE)
    pair = (s["inside"] % (BLOCK // COLUMNS) * (COLUMNS // 2))[:, None] + pair
    h = _mix((key[:, None] + pair) & WHOLE)
    return torch.stack((h & 0xFFFF, h >> 16), 2).view(-1, COLUMNS).int()


def _plain_hold(v, numbers, least):
    """e4m3 values v stands for, rounded up or down by the numbers, and scales."""
    scale = _power(v.abs().amax(1))
    y = v.abs() * torch.where(scale > 0, 1.0 / scale, 0.0)[:, None]
    low = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)
    bits = ((y + low).view(torch.int32) + numbers * 16) & -0x100000
    w = (bits.view(torch.float32) - low).clamp(max=TOP)
    if least:      # what is not zero stays so: it is divided by
        w = torch.where(y > 0, w.clamp(min=2.0 ** -9), 0.0)
    return torch.copysign(w, v).to(E4M3), scale


def _plain_adamw(s):
    case, (b1, b2) = s["case"], BETAS
    g = s["grad"].float() * (1.0 / SCALE)
    norm = torch.sqrt(torch.sum(g.double().square()))
    ok = torch.isfinite(norm)
    coef = torch.where(norm > 1.0, 1.0 / norm, 1.0).float() if case["clip"] else 1.0
    t = (s["step"] + 1).double()
    size = (LR / (1.0 - b1 ** t)).float()
    root = (1.0 / torch.sqrt(1.0 - b2 ** t)).float()
    g = g * coef
    eight = case["states"] == "e4m3"
    m, v = s["exp_avg"].float(), s["exp_avg_sq"].float()
    if eight:
        m, v = m * s["exp_avg_scale"][:, None], v * s["exp_avg_sq_scale"][:, None]
        v = v * v
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    u = torch.sqrt(v)
    p = s["param"] * (1.0 - LR * DECAY) - size * (m / (u * root + ADAM_EPS))
    new = {"param": p}
    if case["copy"]:
        new["copy"] = p.to(torch.bfloat16)
    if eight:
        numbers = _rounding_numbers(s)
        new["exp_avg"], new["exp_avg_scale"] = _plain_hold(m, numbers, False)
        new["exp_avg_sq"], new["exp_avg_sq_scale"] = _plain_hold(u, numbers, True)
    else:
        new["exp_avg"], new["exp_avg_sq"] = m, v
    for name in new:
        old = s[name].view(torch.uint8) if s[name].dtype == E4M3 else s[name]
        old.copy_(torch.where(ok, new[name].view(old.dtype), old))
    s["step"] += ok
    return {"norm": norm} | {name: s[name] for name in new}


# --------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"residual": _plain_residual, "residual_step": _plain_residual,
                "rotary": _plain_rotary, "rotary_step": _plain_rotary,
                "adamw": _plain_adamw}[op](s)
    from gradient_sync_rcc_gb300 import rcc
    if op.startswith("residual"):
        kept = None
        out = rcc.add_rmsnorm_forward(s["x"], s["residual"], s["weight"], eps=EPS,
                                      out_dtype=E4M3 if case["eight"] else None,
                                      keep=op == "residual_step")
        if op == "residual_step":
            y, h, kept = out
        else:
            y, h = out
        got = {"h": h, "y": y}
        if case["eight"]:
            got = {"h": h, "y": y.values, "scales": y.scales}
        if kept is not None:
            got["dx"], got["dweight"] = rcc.add_rmsnorm_backward(s["dy"], s["dh"], kept,
                                                                 s["weight"], eps=EPS)
        return got
    if op.startswith("rotary"):
        got = {}
        got["q"], got["k"] = rcc.rotary_forward(s["q"], s["k"], s["turns"], s["positions"],
                                                layout=case["layout"])
        if op == "rotary_step":
            got["dq"], got["dk"] = rcc.rotary_backward(s["dq"], s["dk"], s["turns"],
                                                       s["positions"], layout=case["layout"])
        return got
    rcc.adamw_step(s["plan"], s["cfg"], scale=SCALE)
    names = ("param", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "copy")
    return {"norm": s["plan"].grad_norm} | {name: s[name] for name in names if name in s}


# -------------------------------------------------------------------- work

def _size(kind):
    return {"f32": 4, "bf16": 2}[kind]


def work(case):
    op = case["op"]
    if op.startswith("residual"):
        t, d = case["tokens"], case["dim"]
        e, many = _size(case["act"]), -(-d // COLUMNS)
        moved = t * d * 3 * e + d * 4 + (t * (d + 4 * many) if case["eight"] else t * d * e)
        if op == "residual":
            return {"bytes": moved, "flops": 5 * t * d}
        # the 8-bit form and its scales written, then read; dy and dh read, dx written
        return {"bytes": moved + t * d * 3 * e + 2 * t * (d + 4 * many) + d * 8,
                "flops": 22 * t * d}
    if op.startswith("rotary"):
        n = case["tokens"] * (case["heads"] + case["key_heads"]) * case["head_dim"]
        times = 2 if op == "rotary_step" else 1
        return {"bytes": times * 2 * n * _size(case["act"])
                + case["tokens"] * (8 if case["far"] else 4),
                "flops": times * 3 * n * case["turned"] // case["head_dim"]}
    n = sum(_sizes(case))
    states = 16 * n if case["states"] == "f32" else 4 * n + 16 * n // COLUMNS
    return {"bytes": n * (_size(case["grad"]) + 8 + (2 if case["copy"] else 0)) + states,
            "flops": 18 * n}


# ------------------------------------------------------------------- exact

def _exact_parts(x):
    """Pieces of 128 columns, the last one shorter."""
    return [x[:, at:at + COLUMNS] for at in range(0, x.shape[1], COLUMNS)]


def _exact_residual(case, s):
    h64 = s["x"].double() + s["residual"].double()
    h, weight = h64.to(s["x"].dtype).double(), s["weight"].double()
    rms = (h.square().sum(1, keepdim=True) / case["dim"] + EPS).sqrt()
    y = h / rms * weight
    out = {"h": h64, "y": y}
    if case["eight"]:
        values, scales = [], []
        for part in _exact_parts(y):
            top = part.abs().max(1, keepdim=True).values
            scale = torch.where(top < TINY, 0.0, top / TOP)
            values.append(_exact_e4m3(part / torch.where(scale > 0, scale, 1.0), 0.5))
            scales.append(scale)
        out["y"], out["scales"] = torch.cat(values, 1), torch.cat(scales, 1)
    if case["op"] == "residual":
        return out
    kept = []
    for part in _exact_parts(h.float()):
        # whole numbers by the definition's own 32-bit operations: bf16 values lie on borders
        top = part.abs().max(1, keepdim=True).values
        whole = torch.round(part * (127.0 * torch.where(top < TINY, 0.0, 1.0 / top)))
        kept.append(whole.double() * torch.where(top < TINY, 0.0, top * (1.0 / 127.0)).double())
    x, dy = torch.cat(kept, 1), s["dy"].double()
    rms = (x.square().sum(1, keepdim=True) / case["dim"] + EPS).sqrt()
    back = dy * weight
    along = (back * x).sum(1, keepdim=True) / case["dim"] / rms.square()
    out["dx"] = s["dh"].double() + (back - x * along) / rms
    out["dweight"] = (dy * x / rms).sum(0)
    return out


def _exact_e4m3(v, up):
    """v on the grid of e4m3: away from zero where the rest of a step is 1 - up or
    more (for a half: ties to even)."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3.0)
    n = torch.round(a / step) if isinstance(up, float) else torch.floor(a / step + up)
    return torch.copysign((n * step).clamp_max(TOP), v)


def _exact_rotary(case, s):
    n = case["turned"]
    i = torch.arange(n // 2, device=DEVICE, dtype=torch.float64)
    scaling = _scaling(case) or ("none",)
    slow = scaling[1] if scaling[0] == "base" else 1.0
    f = torch.exp(-i * (2.0 / n) * math.log(10000.0)
                  - (i * 2.0 / (n - 2) * math.log(slow) if n > 2 else 0.0))
    if scaling[0] == "linear":
        f = f / 4.0
    if scaling[0] == "parts":
        share = ((8192 * f / (2.0 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
        f = share * f + (1.0 - share) * f / 8.0
    turn = torch.polar(torch.ones((), device=DEVICE, dtype=torch.float64),
                       torch.outer(s["positions"].double(), f))[:, None]
    out = {}
    for name in ("q", "k", "dq", "dk") if case["op"] == "rotary_step" else ("q", "k"):
        x = s[name].double()
        pairs = x[:, :, :n].unflatten(2, (2, n // 2) if case["layout"] == "half" else (n // 2, 2))
        if case["layout"] == "half":
            pairs = pairs.transpose(2, 3)
        z = torch.view_as_complex(pairs.contiguous()) * (turn if len(name) == 1 else turn.conj())
        z = torch.view_as_real(z)
        if case["layout"] == "half":
            z = z.transpose(2, 3)
        out[name] = torch.cat([z.flatten(2), x[:, :, n:]], 2)
    return out


def _exact_held(v, chance, least):
    """The e4m3 values and power-of-two scales that v is held as."""
    top = v.abs().amax(1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / TOP)))
    scale = torch.where(top < NOTHING, 0.0, scale)
    y = torch.where(scale > 0, v / torch.where(scale > 0, scale, 1.0), 0.0)
    w = _exact_e4m3(y, chance)
    if least:
        w = torch.where(y > 0, w.clamp_min(2.0 ** -9), 0.0)
    return w, scale[:, 0]


def _exact_adamw(case, s):
    b1, b2 = BETAS
    g = s["grad"].double() / SCALE
    norm = float(g.square().sum().sqrt())
    if case["clip"] and norm > 1.0:
        g = g / norm
    m, v = s["exp_avg"].double(), s["exp_avg_sq"].double()
    if case["states"] == "e4m3":
        m = m * s["exp_avg_scale"].double()[:, None]
        v = (v * s["exp_avg_sq_scale"].double()[:, None]).square()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g.square()
    del g
    t = TAKEN + 1
    change = m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + ADAM_EPS)
    p = s["param"].double() * (1 - LR * DECAY) - LR * change
    del change
    out = {"norm": torch.tensor(norm, device=DEVICE, dtype=torch.float64), "param": p}
    if case["copy"]:
        out["copy"] = p
    if case["states"] == "f32":
        return out | {"exp_avg": m, "exp_avg_sq": v}
    # 64-bit temporaries of the held values of all elements: not for the largest cases
    if m.numel() > 150e6:
        return out | dict.fromkeys(("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"))
    chance = _rounding_numbers(s).double() / 65536.0
    for name, held, least in (("exp_avg", m, False), ("exp_avg_sq", v.sqrt(), True)):
        out[name], out[name + "_scale"] = _exact_held(held, chance, least)
    return out


def exact(case, seed):
    """In 64 bits.  (What an optimizer state is held as, and each norm's 8-bit
    value, is rounded as its definition says.)"""
    s = prepare(case, seed)
    if case["op"].startswith("residual"):
        return _exact_residual(case, s)
    if case["op"].startswith("rotary"):
        return _exact_rotary(case, s)
    return _exact_adamw(case, s)
