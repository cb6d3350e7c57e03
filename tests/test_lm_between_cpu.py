"""Refusals of the residual RMS norm, rotary positions and AdamW plans by the C ABI
and the binding, and the frequencies of the positions (no GPU needed).

Every malformed call returns its status before any CUDA call, so the fake
addresses below are never dereferenced.
"""
import ctypes as C
import decimal
import math

import pytest
import torch

BASE = 0x7F0000000000   # fake device addresses, 256-byte aligned
E4M3 = torch.float8_e4m3fn


def at(i):
    return BASE + (i << 32)


@pytest.fixture
def L(rcc_lib):
    return rcc_lib


def refused(L, name, good, status, **by):
    st = L.raw(name, *dict(good, **by).values())
    assert st == status, (by, st, L.last_error())
    assert L.last_error()


# ------------------------------------------------------------- residual RMS norm

FORWARD = dict(x=at(0), ld_x=256, residual=at(1), ld_r=256, type=0, weight=at(2), eps=1e-6,
               tokens=4, dim=256, sum=at(3), y=at(4), y_scales=at(5), kept=at(6), scales=at(7),
               stream=None)


@pytest.mark.parametrize("by", [
    dict(x=None), dict(weight=None), dict(y=None), dict(kept=None), dict(scales=None),
    dict(residual=None), dict(sum=None), dict(residual=None, sum=None, y_scales=None),
    dict(type=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(dim=0),
    dict(dim=32769, ld_x=32769, ld_r=32769), dict(x=at(0) + 2), dict(residual=at(1) + 1),
    dict(sum=at(3) + 2), dict(y_scales=at(5) + 2), dict(kept=at(6) + 8), dict(y=at(0)),
    dict(y=at(3) + 64), dict(y_scales=at(4) + 1020), dict(scales=at(6) + 16),
    dict(sum=at(0), ld_x=257), dict(sum=at(1), ld_r=260), dict(sum=at(0) + 4),
    dict(tokens=1 << 31), dict(sum=at(2))])
def test_add_rmsnorm_forward_refusals(L, by):
    refused(L, "rcc_add_rmsnorm_forward", FORWARD, L.ERR_INVALID_ARGUMENT, **by)


def test_add_rmsnorm_forward_shapes_and_no_tokens(L):
    for by in (dict(ld_x=255), dict(ld_r=0)):
        refused(L, "rcc_add_rmsnorm_forward", FORWARD, L.ERR_SHAPE_MISMATCH, **by)
    assert L.raw("rcc_add_rmsnorm_forward", *dict(FORWARD, tokens=0, x=None).values()) == L.OK


def test_add_rmsnorm_backward_refusals(L):
    need = L.rmsnorm_backward_workspace(4, 256)
    good = dict(dy=at(0), ld_dy=256, dsum=at(1), ld_dsum=256, type=1, kept=at(2), scales=at(3),
                weight=at(4), eps=0.0, tokens=4, dim=256, dx=at(5), dweight=at(6), accumulate=0,
                ws=at(7), bytes=need, stream=None)
    for by in (dict(dy=None), dict(kept=None), dict(scales=None), dict(weight=None),
               dict(dx=None), dict(dweight=None), dict(ws=None), dict(type=5), dict(eps=-0.5),
               dict(dim=1 << 16, ld_dy=1 << 16, ld_dsum=1 << 16), dict(kept=at(2) + 4),
               dict(dx=at(0)), dict(dweight=at(4) + 4), dict(ws=at(7) + 16), dict(dsum=at(1) + 1),
               dict(dx=at(1), ld_dsum=264), dict(dx=at(1) + 2), dict(dsum=None, dx=at(0))):
        refused(L, "rcc_add_rmsnorm_backward", good, L.ERR_INVALID_ARGUMENT, **by)
    for by in (dict(bytes=0), dict(ld_dy=8), dict(ld_dsum=255)):
        refused(L, "rcc_add_rmsnorm_backward", good, L.ERR_SHAPE_MISMATCH, **by)
    assert L.raw("rcc_add_rmsnorm_backward", *dict(good, tokens=0, accumulate=1).values()) == L.OK


def test_the_binding_of_the_residual_norm_refuses(L):
    x, weight = torch.zeros(4, 256), torch.ones(256)
    r16 = x.bfloat16()
    for args, more in (((x, r16, weight), {}), ((x, x[:3], weight), {}), ((x, x, weight[:9]), {}),
                       ((x, None, weight), {}), ((x, x, weight), dict(out_dtype=torch.float16)),
                       ((x, x, weight), dict(out_dtype=torch.bfloat16)),
                       ((x, x.t(), weight), {}), ((x, x, weight), dict(h=x[:, :8])),
                       ((x, x, weight), dict(out=torch.zeros(4, 8))),
                       ((x, None, weight), dict(out_dtype=E4M3, h=x)),
                       ((x, x, weight), dict(out=x, out_dtype=E4M3)),
                       ((x, x, weight), dict(keep=L.Kept(3, 256, "cpu")))):
        with pytest.raises(ValueError):
            L.add_rmsnorm_forward(*args, **more)
    with pytest.raises(ValueError, match="CUDA device"):
        L.add_rmsnorm_forward(x, x, weight, keep=True)
    kept = L.Kept(4, 256, "cpu")
    for args, more in (((x, r16, kept, weight), {}), ((x, x[:3], kept, weight), {}),
                       ((x, x, L.Kept(4, 255, "cpu"), weight), {}),
                       ((x, x, kept, weight), dict(accumulate=True)),
                       ((x, x, kept, weight), dict(dx=r16))):
        with pytest.raises(ValueError):
            L.add_rmsnorm_backward(*args, **more)
    with pytest.raises(ValueError, match="CUDA device"):
        L.add_rmsnorm_backward(x, None, kept, weight)


# ------------------------------------------------------------------ rotary positions

def rows(L, i, heads=2, head_dim=64, **by):
    """Packed [tokens][heads][head_dim] at address i, out at i + 1."""
    f = dict(in_=at(i), out=at(i + 1), heads=heads, in_token=heads * head_dim, in_head=head_dim,
             out_token=heads * head_dim, out_head=head_dim)
    f.update(by)
    return L.RotaryRows(**f)


def rotary_args(L, q, k, **by):
    good = dict(q=q, k=k, type=0, tokens=10, head_dim=64, turns=at(20), pairs=32, layout=0,
                positions=at(21), index=1, offset=0, scale=1.0, stream=None)
    good.update(by)
    good["q"] = None if q is None else C.byref(q)
    good["k"] = None if k is None else C.byref(k)
    return list(good.values())


@pytest.mark.parametrize("by", [
    dict(type=2), dict(tokens=1 << 31), dict(head_dim=1), dict(head_dim=8193, pairs=4),
    dict(turns=None), dict(turns=at(20) + 4), dict(pairs=0), dict(pairs=33), dict(layout=2),
    dict(index=2), dict(positions=at(21) + 4), dict(offset=-1), dict(offset=1 << 31),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(turns=at(1)), dict(positions=at(3))])
@pytest.mark.parametrize("name", ["rcc_rotary_forward", "rcc_rotary_backward"])
def test_rotary_refusals(L, name, by):
    q, k = rows(L, 0), rows(L, 2)
    assert L.raw(name, *rotary_args(L, q, k, **by)) == L.ERR_INVALID_ARGUMENT, by
    assert L.last_error()


@pytest.mark.parametrize("status,by", [
    ("ERR_INVALID_ARGUMENT", dict(in_=None)), ("ERR_INVALID_ARGUMENT", dict(out=None)),
    ("ERR_INVALID_ARGUMENT", dict(in_=at(0) + 2)), ("ERR_INVALID_ARGUMENT", dict(heads=65537)),
    ("ERR_INVALID_ARGUMENT", dict(in_token=(1 << 30) + 1)),
    ("ERR_INVALID_ARGUMENT", dict(out_head=(1 << 40) + 1)),
    ("ERR_SHAPE_MISMATCH", dict(in_head=63)), ("ERR_SHAPE_MISMATCH", dict(out_token=127)),
    ("ERR_SHAPE_MISMATCH", dict(in_token=0)),
    ("ERR_INVALID_ARGUMENT", dict(out=at(0) + 4)),             # shifted over its input
    ("ERR_INVALID_ARGUMENT", dict(out=at(0), out_token=256)),  # in place with another stride
    ("ERR_INVALID_ARGUMENT", dict(out=at(2))),                 # over k's input
    ("ERR_INVALID_ARGUMENT", dict(out=at(3) + 256)),           # over k's output, token by token
])
def test_rotary_refuses_rows(L, status, by):
    st = L.raw("rcc_rotary_forward", *rotary_args(L, rows(L, 0, **by), rows(L, 2)))
    assert st == getattr(L, status), (st, L.last_error())


def test_rotary_nothing_to_do(L):
    q = rows(L, 0, in_=None, out=None)
    assert L.raw("rcc_rotary_forward", *rotary_args(L, q, None, tokens=0)) == L.OK
    q = rows(L, 0, heads=0)
    assert L.raw("rcc_rotary_forward", *rotary_args(L, q, None)) == L.OK
    assert L.raw("rcc_rotary_forward", *rotary_args(L, None, q)) == L.ERR_INVALID_ARGUMENT


def turns_of(L, pairs, base=10000.0, scaling=None):
    out = (C.c_uint64 * pairs)()
    st = L.raw("rcc_rotary_turns", pairs, base, None if scaling is None else C.byref(scaling), out)
    return st, list(out)


def test_rotary_turns_refusals(L):
    for args in ((0,), (4097,), (4, 0.5), (4, float("nan")), (4, float("inf"))):
        assert L.raw("rcc_rotary_turns", *(args + (10000.0,))[:2], None,
                     (C.c_uint64 * 8)()) == L.ERR_INVALID_ARGUMENT
    assert L.raw("rcc_rotary_turns", 4, 10000.0, None, None) == L.ERR_INVALID_ARGUMENT
    for s in ((4, 2.0, 0, 0, 0), (-1, 2.0, 0, 0, 0), (1, 0.5, 0, 0, 0), (2, float("inf"), 0, 0, 0),
              (3, 2.0, 0.0, 1, 4), (3, 2.0, 100.0, 4, 4), (3, 2.0, 100.0, -1, 4),
              (3, 2.0, float("nan"), 1, 4)):
        assert turns_of(L, 4, scaling=L.RotaryScaling(*s))[0] == L.ERR_INVALID_ARGUMENT, s
    for scaling in (("linear",), ("parts", 2.0), ("other", 2.0)):
        with pytest.raises(ValueError):
            L.rotary_turns(64, scaling=scaling, device="cpu")
    for turned in (0, 7):
        with pytest.raises(ValueError):
            L.rotary_turns(turned, device="cpu")
    with pytest.raises(L.RccError):
        L.rotary_turns(64, base=0.0, device="cpu")


@pytest.mark.parametrize("pairs", [1, 2, 10, 64])
@pytest.mark.parametrize("kind", ["none", "linear", "base", "parts"])
def test_rotary_turns_against_forty_digits(L, pairs, kind):
    """A few roundings of 2^-53 each: the power of a rounded exponent (at most
    ln 1e6 = 14 of them), a product and a quotient or two."""
    D = decimal.Decimal
    with decimal.localcontext() as ctx:
        ctx.prec = 40
        pi = D("3.141592653589793238462643383279502884197")
        base, factor = D(500000), D(8)
        if kind == "base" and pairs > 1:
            base *= factor ** (D(pairs) / D(pairs - 1))
        want = []
        for i in range(pairs):
            f = base ** (-D(i) / D(pairs)) / (2 * pi)
            if kind == "linear":
                f /= factor
            if kind == "parts":
                k = min(D(1), max(D(0), (D(8192) * f - 1) / 3))
                f *= k + (1 - k) / factor
            want.append(f * 2 ** 64)
        scaling = {"none": None, "linear": ("linear", 8.0), "base": ("base", 8.0),
                   "parts": ("parts", 8.0, 8192.0, 1.0, 4.0)}[kind]
        got = L.rotary_turns(2 * pairs, 500000.0, scaling, device="cpu")
        assert got.dtype == torch.int64 and got.shape == (pairs,)
        for g, w in zip(got.tolist(), want):
            assert abs(D(g) - w) <= w * D(40 * 2.0 ** -53) + 1


def test_the_binding_of_rotary_refuses(L):
    q, k = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    turns = L.rotary_turns(64, device="cpu")
    at64 = torch.zeros(5, dtype=torch.int64)
    for args, more in (((q.double(), k, turns), {}), ((q, k.bfloat16(), turns), {}),
                       ((q, k[:4], turns), {}), ((q, k[:, :, :32], turns), {}),
                       ((q[0], k, turns), {}), ((q.transpose(1, 2), None, turns), {}),
                       ((q, k, turns.int()), {}), ((q, k, L.rotary_turns(128, device="cpu")), {}),
                       ((q, k, turns, at64[:4]), {}), ((q, k, turns, at64.float()), {}),
                       ((q, k, turns), dict(layout="other")), ((q, None, turns), dict(k_out=k)),
                       ((q, k, turns), dict(q_out=k)), ((q, k, turns), dict(k_out=k.bfloat16()))):
        for call in (L.rotary_forward, L.rotary_backward):
            with pytest.raises(ValueError):
                call(*args, **more)
    with pytest.raises(ValueError, match="CUDA device"):
        L.rotary_forward(q, k, turns)


# --------------------------------------------------------------------------- AdamW

def adamw_tensor(L, i=0, numel=1000, eight=True, **by):
    f = dict(numel=numel, grad=at(8 * i), grad_type=1, param=at(8 * i + 1), exp_avg=at(8 * i + 2),
             exp_avg_sq=at(8 * i + 3), exp_avg_scale=at(8 * i + 4) if eight else None,
             exp_avg_sq_scale=at(8 * i + 5) if eight else None, copy=at(8 * i + 6))
    f.update(by)
    return L.AdamWTensor(*f.values())


def create(L, of, status, **by):
    arr = (L.AdamWTensor * len(of))(*of)
    need = L.raw("rcc_adamw_workspace", arr, len(of))
    out = C.c_void_p()
    good = dict(tensors=arr, n=len(of), seed=0, step=0, beta1=0.9, beta2=0.999, ws=at(100),
                bytes=need, stream=None, out=C.byref(out))
    good.update(by)
    st = L.raw("rcc_adamw_create", *good.values())
    assert st == status, (by, st, L.last_error())
    assert out.value is None


@pytest.mark.parametrize("by", [
    dict(tensors=None), dict(n=0), dict(n=-3), dict(step=-1), dict(beta1=1.0), dict(beta2=-0.1),
    dict(beta1=float("nan")), dict(ws=None), dict(ws=at(100) + 128), dict(out=None),
    dict(ws=at(1) + 256)])
def test_adamw_plan_refusals(L, by):
    create(L, [adamw_tensor(L), adamw_tensor(L, 1)], L.ERR_INVALID_ARGUMENT, **by)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("by", [
    dict(numel=0), dict(numel=(1 << 40) + 1), dict(grad=None), dict(param=None), dict(exp_avg=None),
    dict(exp_avg_sq=None), dict(grad_type=2), dict(grad=at(8) + 1), dict(param=at(9) + 2),
    dict(copy=at(14) + 1), dict(copy=at(9)), dict(exp_avg=at(1)), dict(param=at(0)),
    dict(exp_avg_sq=at(10) + 996), dict(exp_avg_scale="other"), dict(exp_avg_sq_scale="other")])
def test_adamw_plan_refuses_tensors(L, eight, by):
    other = None if eight else at(12)
    by = {k: other if v == "other" else v for k, v in by.items()}
    create(L, [adamw_tensor(L, 0, eight=eight), adamw_tensor(L, 1, eight=eight, **by)],
           L.ERR_INVALID_ARGUMENT, bytes=1 << 20)


def test_adamw_plan_mixed_states_and_short_workspace(L):
    create(L, [adamw_tensor(L, 0, eight=True), adamw_tensor(L, 1, eight=False)],
           L.ERR_INVALID_ARGUMENT)
    create(L, [adamw_tensor(L)], L.ERR_SHAPE_MISMATCH, bytes=300)
    arr = (L.AdamWTensor * 1)(adamw_tensor(L, numel=0))
    assert L.raw("rcc_adamw_workspace", arr, 1) == 0
    assert L.raw("rcc_adamw_workspace", None, 1) == 0
    many = (L.AdamWTensor * 3000)(*[adamw_tensor(L, numel=1 << 40) for _ in range(3000)])
    assert L.raw("rcc_adamw_workspace", many, 3000) == 0    # more items than a plan takes


def test_a_plan_that_does_not_exist(L):
    cfg = L.adamw_cfg()
    for plan in (None, 12345, (1 << 60) + 7):
        assert L.raw("rcc_adamw_step", plan, C.byref(cfg), 1.0, None) == \
            L.ERR_MISSING_REGISTRATION
        assert L.raw("rcc_adamw_destroy", plan) == L.ERR_MISSING_REGISTRATION
    # the calling convention that `refused` and `create` rely on
    assert C.sizeof(L.AdamWStatus) == 48 and math.isfinite(cfg.lr)


def test_the_plan_of_the_binding_refuses(L):
    p, g = torch.zeros(10), torch.zeros(10)
    for t in (dict(param=p), dict(param=p.double(), grad=g), dict(param=p, grad=g[:9]),
              dict(param=p, grad=g.half()), dict(param=p, grad=g, copy=g),
              dict(param=p, grad=g, exp_avg=p.clone(), exp_avg_sq=p.to(E4M3)),
              dict(param=p, grad=g, other=p), dict(param=torch.zeros(20)[::2], grad=g),
              dict(param=p, grad=g, exp_avg_scale=torch.zeros(1)), dict(grad=g),
              dict(param=p, grad=g, exp_avg=p.to(E4M3)),
              dict(param=p, grad=g, exp_avg=p.to(E4M3), exp_avg_sq=p.to(E4M3),
                   exp_avg_scale=torch.zeros(1), exp_avg_sq_scale=torch.zeros(2))):
        with pytest.raises(ValueError):
            L.AdamWPlan([t])
    with pytest.raises(ValueError):
        L.AdamWPlan([dict(param=p, grad=g)], states=torch.bfloat16)
    with pytest.raises(ValueError):
        L.AdamWPlan([])
    with pytest.raises(ValueError, match="CUDA device"):
        L.AdamWPlan([dict(param=p, grad=g)], states=E4M3)
    with pytest.raises(ValueError, match="adamw_cfg"):
        L.adamw_step(None, dict(lr=1.0))
