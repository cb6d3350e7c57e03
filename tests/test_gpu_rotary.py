"""Rotary positions on the GPU against exact fractions of a turn.

The error of a result is that of its sine and cosine times the pair's sizes: the
argument, half turns as a float, is 2^-25 off (pi 2^-25 in angle) and loses 2^-31;
sincospi is up to 2 ulp (2^-23); the scale, two products and a sum are rounded
(2^-24 each, on a and b alike).
"""
import math

import numpy as np
import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV, GUARD_BYTE

pytestmark = pytest.mark.gpu

U, F32, BF16 = defs.U, defs.F32, defs.BF16
WORST = math.pi * 2.0 ** -25 + math.pi * 2.0 ** -31 + 2.0 ** -23 + 4 * U


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def turned_64(x, turns, positions, layout, scale, inverse):
    """The definition: each angle from the exact remainder of its turns."""
    p = np.array(positions, dtype=np.int64)
    left = np.where(p < 0, 0, p).astype(np.uint64)[:, None] * turns.cpu().numpy().view(np.uint64)
    angle = torch.from_numpy(left.astype(np.float64) * (2 * math.pi * 2.0 ** -64)).to(DEV)
    c, s = scale * torch.cos(angle)[:, None], scale * torch.sin(angle)[:, None]
    s = -s if inverse else s
    n, v = turns.numel(), x.double()
    want, size = v.clone(), torch.zeros_like(v)
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else \
        (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = v[:, :, first], v[:, :, second]
    want[:, :, first], want[:, :, second] = a * c - b * s, a * s + b * c
    size[:, :, first] = size[:, :, second] = (a.abs() + b.abs()) * abs(scale)
    return want, size


def check(got, x, turns, positions, layout="half", scale=1.0, inverse=False):
    want, size = turned_64(x, turns, positions, layout, scale, inverse)
    defs.within(got, want, WORST * size + torch.where(size > 0, defs.half_ulp(want, got.dtype),
                                                      0.0) + 2.0 ** -148)


SHAPES = [(1, 1, 1, 2, 2), (3, 2, 1, 64, 64), (7, 5, 3, 80, 20), (5, 4, 4, 96, 48), (2, 3, 0, 7, 4),
          (33, 8, 2, 128, 128), (130, 6, 2, 128, 32), (4, 64, 8, 256, 256), (9, 7, 1, 40, 16),
          (2, 33, 11, 100, 98)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,key_heads,head_dim,turned", SHAPES)
def test_rotary(dtype, layout, tokens, heads, key_heads, head_dim, turned):
    g = defs.gen(71)
    q = defs.randn(g, tokens, heads, head_dim, dtype=dtype)
    k = defs.randn(g, tokens, key_heads, head_dim, dtype=dtype) if key_heads else None
    turns = rcc.rotary_turns(turned, 10000.0, ("parts", 8.0, 512, 1.0, 4.0), device=DEV)
    far = torch.randint(1 << 31, (tokens,), generator=g, device=DEV)
    far[0] = 0
    for positions, offset in ((far, 0), ((far >> 12).int(), 5), (None, 1000), (None, 0)):
        at = [(offset + p) for p in (range(tokens) if positions is None else positions.tolist())]
        for scale in (1.0, 1.25):
            args = dict(positions=positions, offset=offset, layout=layout, scale=scale)
            q2, k2 = rcc.rotary_forward(q, k, turns, **args)
            check(q2, q, turns, at, layout, scale)
            back, _ = rcc.rotary_backward(q, None, turns, **args)
            check(back, q, turns, at, layout, scale, inverse=True)
            if key_heads:
                check(k2, k, turns, at, layout, scale)
                assert torch.equal(k2, rcc.rotary_forward(k, None, turns, **args)[0])
            else:
                assert k2 is None
            assert torch.equal(q2, rcc.rotary_forward(q, None, turns, **args)[0])
            # past the pairs nothing changes, whatever the scale
            assert torch.equal(q2[:, :, turned:], q[:, :, turned:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("turned,extra", [(64, 0), (32, 8), (64, 3), (20, 0)])
def test_strides_and_places(dtype, layout, turned, extra):
    """Packed rows turned in place, heads before tokens, boundaries off: the same
    bits as contiguous ones, and nothing else written."""
    g = defs.gen(72)
    tokens, heads, key_heads, hd = 11, 6, 2, 64
    turns = rcc.rotary_turns(turned, device=DEV)
    wide = (heads + 2 * key_heads) * hd + extra
    flat = torch.full((tokens * wide + 64,), GUARD_BYTE, dtype=torch.uint8,
                      device=DEV).to(dtype)
    packed = flat[extra:extra + tokens * wide].view(tokens, wide)
    packed[:, :wide - extra] = defs.randn(g, tokens, wide - extra, dtype=dtype)
    before = flat.clone()
    q = packed[:, :heads * hd].unflatten(1, (heads, hd))
    k = packed[:, heads * hd:(heads + key_heads) * hd].unflatten(1, (key_heads, hd))
    want = rcc.rotary_forward(q.clone(), k.clone(), turns, offset=3, layout=layout)
    out = rcc.rotary_forward(q, k, turns, offset=3, layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(flat, before)
    # q alone, then k alone in the same rows
    rcc.rotary_forward(q, None, turns, offset=3, layout=layout, q_out=q)
    assert torch.equal(q, want[0])
    rcc.rotary_forward(k, None, turns, offset=3, layout=layout, q_out=k)
    assert torch.equal(k, want[1])
    q[:], k[:] = 0, 0
    rest = flat.clone()
    flat.copy_(before)
    got = rcc.rotary_forward(q, k, turns, offset=3, layout=layout, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    q[:], k[:] = 0, 0
    assert torch.equal(flat, rest)
    # heads before tokens, on both sides
    turned_q = want[0].transpose(0, 1).contiguous()
    src = before[extra:extra + tokens * wide].view(tokens, wide)[:, :heads * hd]
    src = src.unflatten(1, (heads, hd)).transpose(0, 1).contiguous()
    dst = torch.empty_like(src)
    rcc.rotary_forward(src.transpose(0, 1), None, turns, offset=3, layout=layout,
                       q_out=dst.transpose(0, 1))
    assert torch.equal(dst, turned_q)


def test_a_turn_back_and_the_gradient():
    """The backward pass turns back, and <d, R q> = <R^T d, q>."""
    g = defs.gen(73)
    q, d = defs.randn(g, 50, 3, 64), defs.randn(g, 50, 3, 64)
    turns = rcc.rotary_turns(48, device=DEV)
    positions = torch.randint(1 << 20, (50,), generator=g, device=DEV)
    out, _ = rcc.rotary_forward(q, None, turns, positions)
    back, _ = rcc.rotary_backward(out, None, turns, positions)
    size = (q.abs() + q.abs().amax(2, keepdim=True)).double()
    defs.within(back, q.double(), 4 * WORST * size)
    grad, _ = rcc.rotary_backward(d, None, turns, positions)
    left, right = (d.double() * out.double()).sum(), (grad.double() * q.double()).sum()
    both = (d.double().abs() * size).sum() + (grad.double().abs() * q.double().abs()).sum()
    assert abs(float(left - right)) <= 2 * WORST * float(both)
    # differences: the pass is linear
    along = defs.randn(g, 50, 3, 64)
    f = [(d.double() * rcc.rotary_forward(q + s * along, None, turns, positions)[0].double()).sum()
         for s in (1, -1)]
    assert abs(float((f[0] - f[1]) / 2 - (grad.double() * along.double()).sum())) <= \
        4 * WORST * float((d.abs() * (q.abs() + along.abs()).amax(2, keepdim=True) * 2).double().sum())


def test_padding_and_scale():
    q = defs.randn(defs.gen(74), 4, 2, 32, dtype=BF16)
    turns = rcc.rotary_turns(32, device=DEV)
    for kind in (torch.int32, torch.int64):
        positions = torch.tensor([-1, 7, torch.iinfo(kind).min, 0], dtype=kind, device=DEV)
        out, _ = rcc.rotary_forward(q, None, turns, positions, offset=100)
        assert torch.equal(out[[0, 2]], q[[0, 2]])      # a position below 0 does not turn
        check(out, q, turns, [-1, 107, -1, 100])
    out, _ = rcc.rotary_forward(q, None, turns, positions, scale=0.5)
    assert torch.equal(out[0], q[0] * 0.5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_pair(bad):
    q = defs.randn(defs.gen(75), 3, 2, 64)
    q[1, 1, 5] = bad
    out, _ = rcc.rotary_forward(q, None, rcc.rotary_turns(32, device=DEV), offset=9)
    wrong = torch.zeros(3, 2, 64, dtype=torch.bool, device=DEV)
    wrong[1, 1, 5] = wrong[1, 1, 21] = True
    assert torch.equal(~torch.isfinite(out), wrong)


def test_nothing_to_turn():
    turns = rcc.rotary_turns(64, device=DEV)
    q, k = torch.empty(0, 4, 64, device=DEV), torch.empty(0, 2, 64, device=DEV)
    a, b = rcc.rotary_forward(q, k, turns, torch.empty(0, dtype=torch.int32, device=DEV))
    assert a.shape == q.shape and b.shape == k.shape
    none, k = torch.empty(5, 0, 64, device=DEV), torch.ones(5, 1, 64, device=DEV)
    a, b = rcc.rotary_forward(none, k, turns)
    assert a.shape == none.shape
    check(b, k, turns, range(5))


def test_refusals_on_the_gpu():
    turns = rcc.rotary_turns(64, device=DEV)
    q = torch.ones(5, 2, 64, device=DEV)
    wide = torch.ones(6, 2, 64, device=DEV)
    for args, more in (((wide[1:], None), dict(q_out=wide[:5])),       # overlapping, not in place
                       ((q.expand(5, 2, 64)[:, :1].expand(5, 2, 64), None), {}),
                       ((q, q[:, :1]), dict(q_out=q)),                 # k is a part of q
                       ((q, q), dict(q_out=wide[:5], k_out=wide[:5])),
                       ((q, None), dict(offset=-1)), ((q, None), dict(scale=float("nan")))):
        with pytest.raises((ValueError, rcc.RccError)):
            rcc.rotary_forward(*args, turns, **more)
    # one buffer read as both is fine
    a, b = rcc.rotary_forward(q, q, turns)
    assert torch.equal(a, b)


def test_captured_and_on_a_given_stream():
    g = defs.gen(76)
    q, k = defs.randn(g, 700, 9, 128, dtype=BF16), defs.randn(g, 700, 3, 128, dtype=BF16)
    turns = rcc.rotary_turns(128, device=DEV)
    want = rcc.rotary_forward(q, k, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rcc.rotary_forward(q, k, turns, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = rcc.rotary_forward(q, k, turns)
    got[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
