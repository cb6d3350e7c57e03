"""Cases of the language-model operators: token embedding and its gradient, the
RMS norm that keeps its input in 8 bits for the backward pass, and the output
layer's cross entropy with its gradients.

`run` computes an operator in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, through this
repository's entry points.  `exact` restates the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
GROUP = 128          # columns that share one scale of the 8-bit form
TINY = 2.0 ** -120   # a group below this is held as zeros
EPS = 1e-6           # of the norm
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGEST = 8192 * 131072 * 4096   # tokens * vocabulary * width of the largest loss


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding or debugging step's tokens: a lookup that is all latency
        {"name": "lookup_few", "op": "embed", "tokens": 8, "vocab": 32768, "dim": 1024,
         "table": "bf16", "act": "bf16", "ids": "i64"},
        # a long micro-batch read out of the fp32 master table as bf16 activations
        {"name": "lookup_batch", "op": "embed", "tokens": 32768, "vocab": 131072, "dim": 4096,
         "table": "f32", "act": "bf16", "ids": "i64"},
        # tied weights: added onto the output layer's gradient; odd token and row counts
        {"name": "lookup_grad_tied", "op": "embed_grad", "tokens": 8191, "vocab": 50021,
         "dim": 2048, "act": "bf16", "grad": "f32", "ids": "i32", "accumulate": True},
        # a long micro-batch's dense gradient, absent tokens' rows included
        {"name": "lookup_grad_batch", "op": "embed_grad", "tokens": 32768, "vocab": 131072,
         "dim": 4096, "act": "bf16", "grad": "f32", "ids": "i64", "accumulate": False},
        # inference: a few tokens of a small fp32 model, nothing kept
        {"name": "norm_few", "op": "norm", "tokens": 16, "dim": 1024, "act": "f32"},
        # a training micro-batch: forward, input kept in 8 bits, backward from the 8 bits
        {"name": "norm_step_batch", "op": "norm_step", "tokens": 16384, "dim": 4096,
         "act": "bf16"},
        # the same for a width that is no multiple of the group, fp32
        {"name": "norm_step_odd", "op": "norm_step", "tokens": 1023, "dim": 1000, "act": "f32"},
        # scoring one token: the weights are read once for one row
        {"name": "loss_one", "op": "loss", "tokens": 1, "vocab": 32768, "dim": 1024,
         "ids": "i64"},
        # evaluating held-out text with an odd vocabulary
        {"name": "loss_eval", "op": "loss", "tokens": 2000, "vocab": 50021, "dim": 2048,
         "ids": "i32"},
        # a short sequence's training step: the weights and their gradient are what moves
        {"name": "loss_train_short", "op": "loss_grad", "tokens": 100, "vocab": 50021,
         "dim": 1024, "grad": "bf16", "ids": "i64"},
        # a small model's training step: fp32 gradients for the gradient sync
        {"name": "loss_train_f32", "op": "loss_grad", "tokens": 2048, "vocab": 32000,
         "dim": 1024, "grad": "f32", "ids": "i64"},
        # a large model's training step with bf16 gradients
        {"name": "loss_train_large", "op": "loss_grad", "tokens": 8192, "vocab": 131072,
         "dim": 4096, "grad": "bf16", "ids": "i64"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    """A width in [lo, hi], a multiple of `step`."""
    d = max(lo, _log_uniform(rng, lo, hi) // step * step)
    return d + step if d == 3072 else d


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_step", "loss", "loss_grad"])
    act = rng.choice(["f32", "bf16"])
    ids = rng.choice(["i32", "i64"])
    if op in ("embed", "embed_grad"):
        case = {"op": op, "tokens": _log_uniform(rng, 1, 32768),
                "vocab": _log_uniform(rng, 500, 131072),
                "dim": _width(rng, 64, 4096, rng.choice([1, 8, 64])), "act": act, "ids": ids}
        if op == "embed":
            return dict(case, table=rng.choice(["f32", "bf16"]))
        return dict(case, grad=rng.choice(["f32", "bf16"]), accumulate=rng.random() < 0.5)
    if op in ("norm", "norm_step"):
        return {"op": op, "tokens": _log_uniform(rng, 1, 16384),
                "dim": _width(rng, 64, 8192, rng.choice([1, 8, 128])), "act": act}
    while True:
        case = {"op": op, "tokens": _log_uniform(rng, 1, 8192),
                "vocab": _log_uniform(rng, 500, 131072),
                "dim": _width(rng, 64, 4096, rng.choice([8, 64])), "ids": ids}
        if case["tokens"] * case["vocab"] * case["dim"] * 4 <= LARGEST:
            break
    return dict(case, grad=rng.choice(["f32", "bf16"])) if op == "loss_grad" else case


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _tokens(g, case, padding):
    """Token ids as text has them: the k-th most common with a frequency near
    1/k, in no order of the ids, and a share of padding (-1)."""
    t, v = case["tokens"], case["vocab"]
    u = torch.rand(t, generator=g, device=DEVICE, dtype=torch.float64)
    rank = ((v + 1.0) ** u).long().clamp_(1, v) - 1
    ids = torch.randperm(v, generator=g, device=DEVICE)[rank]
    if t > 1:
        ids[torch.rand(t, generator=g, device=DEVICE) < padding] = -1
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def prepare(case, seed):
    g = _generator(seed)
    op, dim, t = case["op"], case["dim"], case["tokens"]
    s = {"case": case}
    if op == "embed":
        s["scale"] = math.sqrt(dim)
        s["table"] = _randn(g, case["vocab"], dim).mul_(0.02).to(TYPES[case["table"]])
        s["ids"] = _tokens(g, case, 0.02)
    elif op == "embed_grad":
        s["scale"] = math.sqrt(dim)
        s["ids"] = _tokens(g, case, 0.02)
        s["dout"] = _randn(g, t, dim).mul_(1e-2).to(TYPES[case["act"]])
        s["dtable"] = _randn(g, case["vocab"], dim).mul_(1e-2).to(TYPES[case["grad"]])
    elif op in ("norm", "norm_step"):
        # a residual stream: a few columns far larger than the others
        x = _randn(g, t, dim)
        x *= torch.exp(0.5 * _randn(g, dim))
        x[:, torch.randint(dim, (max(1, dim // 512),), generator=g, device=DEVICE)] *= 30.0
        s["x"] = x.to(TYPES[case["act"]])
        s["weight"] = 1.0 + 0.1 * _randn(g, dim)
        s["dy"] = _randn(g, t, dim).mul_(1e-2).to(TYPES[case["act"]])
    else:
        w = _randn(g, case["vocab"], dim).mul_(2.0 / math.sqrt(dim))
        s["labels"] = _tokens(g, case, 0.05)
        # hidden states that know something of their label
        x = _randn(g, t, dim)
        x += 2.0 * w[s["labels"].long().clamp_min(0)] * (s["labels"] >= 0)[:, None]
        s["x"], s["w"] = x.bfloat16(), w.bfloat16()
        if op == "loss_grad":
            # the mean over the counted tokens, times a loss scale
            counted = (s["labels"] >= 0).float()
            s["dloss"] = counted * (1024.0 / counted.sum().clamp_min(1.0))
    return s


# ------------------------------------------------------------- plain forms

def _plain_kept(x):
    """What is left of x once it has been held in 8 bits: whole numbers in
    [-127, 127] and one scale for each group of columns."""
    t, dim = x.shape
    groups = -(-dim // GROUP)
    padded = torch.zeros(t, groups * GROUP, device=x.device)
    padded[:, :dim] = x
    grouped = padded.view(t, groups, GROUP)
    amax = grouped.abs().amax(2, keepdim=True)
    small = amax < TINY
    q = torch.round(grouped * torch.where(small, 0.0, 127.0 / amax))
    return (q * torch.where(small, 0.0, amax / 127.0)).view(t, -1)[:, :dim]


def _plain_embed(s):
    ids = s["ids"].long()
    inside = (ids >= 0) & (ids < s["table"].shape[0])
    rows = s["table"][torch.where(inside, ids, 0)].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(TYPES[s["case"]["act"]])


def _plain_embed_grad(s):
    ids, table = s["ids"].long(), s["dtable"]
    inside = (ids >= 0) & (ids < table.shape[0])
    order = torch.argsort(torch.where(inside, ids, table.shape[0]), stable=True)
    order = order[:int(inside.sum())]
    total = torch.zeros(table.shape, device=table.device)
    total.index_add_(0, ids[order], s["dout"][order].float())
    total *= s["scale"]
    if s["case"]["accumulate"]:
        total += table.float()
    table.copy_(total)
    return table


def _plain_norm(s):
    x = s["x"].float()
    r = torch.rsqrt(torch.mean(x * x, 1, keepdim=True) + EPS)
    y = (x * r * s["weight"]).to(s["x"].dtype)
    if s["case"]["op"] == "norm":
        return y
    x, dy = _plain_kept(s["x"]), s["dy"].float()
    r = torch.rsqrt(torch.mean(x * x, 1, keepdim=True) + EPS)
    n, d = x * r, dy * s["weight"]
    dx = r * (d - n * torch.mean(d * n, 1, keepdim=True))
    return {"y": y, "dx": dx.to(s["dy"].dtype), "dweight": torch.sum(dy * n, 0)}


def _plain_loss(s):
    labels = s["labels"].long()
    x, w = s["x"].float(), s["w"].float()
    inside = (labels >= 0) & (labels < w.shape[0])
    at = torch.where(inside, labels, 0)[:, None]
    z = x @ w.t()
    top = torch.amax(z, 1, keepdim=True)
    lse = top + torch.log(torch.sum(torch.exp(z - top), 1, keepdim=True))
    loss = torch.where(inside, (lse - torch.gather(z, 1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0]}
    if s["case"]["op"] == "loss_grad":
        z = torch.exp(z - lse)
        z.scatter_add_(1, at, torch.full_like(lse, -1.0))
        z *= torch.where(inside, s["dloss"], 0.0)[:, None]
        kind = TYPES[s["case"]["grad"]]
        out["dx"], out["dw"] = (z @ w).to(kind), (z.t() @ x).to(kind)
    return out


# --------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "norm": _plain_norm,
                "norm_step": _plain_norm, "loss": _plain_loss, "loss_grad": _plain_loss}[op](s)
    from gradient_sync_rcc_gb300 import rcc
    if op == "embed":
        return rcc.embedding_forward(s["table"], s["ids"], scale=s["scale"],
                                     out_dtype=TYPES[case["act"]])
    if op == "embed_grad":
        return rcc.embedding_backward(s["dout"], s["ids"], s["dtable"], scale=s["scale"],
                                      accumulate=case["accumulate"])
    if op == "norm":
        return rcc.rmsnorm_forward(s["x"], s["weight"], eps=EPS)
    if op == "norm_step":
        y, kept = rcc.rmsnorm_forward(s["x"], s["weight"], eps=EPS, keep=True)
        dx, dweight = rcc.rmsnorm_backward(s["dy"], kept, s["weight"], eps=EPS)
        return {"y": y, "dx": dx, "dweight": dweight}
    loss, lse = rcc.linear_ce_forward(s["x"], s["w"], s["labels"])
    if op == "loss":
        return {"loss": loss, "lse": lse}
    dx, dw = rcc.linear_ce_backward(s["x"], s["w"], s["labels"], lse, s["dloss"],
                                    grad_dtype=TYPES[case["grad"]])
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


# -------------------------------------------------------------------- work

def _size(kind):
    return {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}[kind]


def work(case):
    op, t, d = case["op"], case["tokens"], case["dim"]
    if op == "embed":
        rows = min(t, case["vocab"])
        return {"bytes": rows * d * _size(case["table"]) + t * d * _size(case["act"])
                + t * _size(case["ids"]), "flops": t * d}
    if op == "embed_grad":
        # written whole, or (accumulating) the rows of the distinct tokens read and written;
        # text with frequencies near 1/k has about V ln(1 + t / (V ln V)) distinct ones at most t
        v = case["vocab"]
        e = _size(case["grad"])
        distinct = min(t, v, v * math.log1p(t / math.log(v)) / math.log(v))
        table = 2 * distinct * d * e if case["accumulate"] else v * d * e
        return {"bytes": int(t * d * _size(case["act"]) + t * _size(case["ids"]) + table),
                "flops": t * d}
    if op == "norm":
        return {"bytes": 2 * t * d * _size(case["act"]) + d * 4, "flops": 4 * t * d}
    if op == "norm_step":
        # x, dy, y and dx once each; the 8-bit form and its scales written, then read
        return {"bytes": 4 * t * d * _size(case["act"])
                + 2 * t * (d + 4 * -(-d // GROUP)) + d * 12, "flops": 20 * t * d}
    v = case["vocab"]
    read = (t + v) * d * 2 + t * _size(case["ids"])
    if op == "loss":
        return {"bytes": read + 8 * t, "flops": 2 * t * v * d}
    return {"bytes": read + 12 * t + (t + v) * d * _size(case["grad"]), "flops": 6 * t * v * d}


# ------------------------------------------------------------------- exact

def _exact_kept(x):
    """Values of the 8-bit form of x from its definition, in 64 bits."""
    out = torch.zeros_like(x)
    for at in range(0, x.shape[1], GROUP):
        part = x[:, at:at + GROUP]
        top = part.abs().max(1, keepdim=True).values
        step = top / 127.0
        whole = torch.round(part / torch.where(top < TINY, 1.0, step))
        out[:, at:at + GROUP] = torch.where(top < TINY, 0.0, whole * step)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, t = case["op"], case["tokens"]
    if op == "embed":
        out = torch.zeros(t, case["dim"], device=DEVICE, dtype=torch.float64)
        hit = torch.nonzero(s["ids"] >= 0)[:, 0]
        out[hit] = s["table"][s["ids"][hit].long()].double() * s["scale"]
        return out
    if op == "embed_grad":
        out = s["dtable"].double() if case["accumulate"] else \
            torch.zeros(s["dtable"].shape, device=DEVICE, dtype=torch.float64)
        hit = torch.nonzero(s["ids"] >= 0)[:, 0]
        return out.index_add_(0, s["ids"][hit].long(), s["dout"][hit].double(),
                              alpha=s["scale"])
    if op in ("norm", "norm_step"):
        x, weight = s["x"].double(), s["weight"].double()
        rms = (x.square().sum(1, keepdim=True) / case["dim"] + EPS).sqrt()
        y = x / rms * weight
        if op == "norm":
            return y
        x, dy = _exact_kept(x), s["dy"].double()
        rms = (x.square().sum(1, keepdim=True) / case["dim"] + EPS).sqrt()
        back = dy * weight
        along = (back * x).sum(1, keepdim=True) / case["dim"] / rms.square()
        return {"y": y, "dx": (back - x * along) / rms, "dweight": (dy * x / rms).sum(0)}
    # the loss: pieces of the vocabulary, so that the 64-bit scores fit; FP64 runs near 1 TFLOP/s
    products = t * case["vocab"] * case["dim"]
    if products > 6e12:
        return None
    x, labels = s["x"].double(), s["labels"].long()
    piece = max(1, int(2e9) // (8 * t))
    parts = range(0, case["vocab"], piece)
    lse = torch.full((t,), -math.inf, device=DEVICE, dtype=torch.float64)
    for at in parts:
        lse = torch.logaddexp(lse, torch.logsumexp(x @ s["w"][at:at + piece].double().t(), 1))
    hit = labels >= 0
    score = (x * s["w"][labels.clamp_min(0)].double()).sum(1)
    out = {"loss": torch.where(hit, lse - score, 0.0), "lse": lse}
    if op == "loss_grad":
        out["dx"] = out["dw"] = None
        if products <= 2e12:
            factor = torch.where(hit, s["dloss"].double(), 0.0)[:, None]
            dx, dw = torch.zeros_like(x), []
            for at in parts:
                w = s["w"][at:at + piece].double()
                dz = torch.exp(x @ w.t() - lse[:, None])
                mine = torch.nonzero(hit & (labels >= at) & (labels < at + piece))[:, 0]
                dz[mine, labels[mine] - at] -= 1.0
                dz *= factor
                dx += dz @ w
                dw.append(dz.t() @ x)
            out["dx"], out["dw"] = dx, torch.cat(dw)
    return out
