"""The RMS norm with the residual's addition and its output in 8 bits, on the GPU.

Tolerances are worst-case rounding bounds, as in test_gpu_lm.py; where another
call's bits are what is documented, they are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import test_gpu_lm as defs
from gradient_sync_rcc_gb300 import rcc
from gpu_util import DEV, GUARD_BYTE, GUARD_BYTES, Guarded

pytestmark = pytest.mark.gpu

U, F32, BF16, E4M3 = defs.U, defs.F32, defs.BF16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gradient_sync_rcc_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class GuardedBytes:
    """n bytes between two bands of a fixed pattern, `offset` off their boundary."""

    def __init__(self, n, offset=0):
        self.raw = torch.full((2 * GUARD_BYTES + n + offset,), GUARD_BYTE, dtype=torch.uint8,
                              device=DEV)
        self.lo, self.n = GUARD_BYTES + offset, n
        self.t = self.raw[self.lo:self.lo + n]

    def guards_intact(self):
        return bool((self.raw[:self.lo] == GUARD_BYTE).all()) and \
            bool((self.raw[self.lo + self.n:] == GUARD_BYTE).all())


def inputs(g, dtype, tokens, dim, extra):
    x = defs.randn(g, tokens, dim, dtype=dtype)
    r = defs.randn(g, tokens, dim, dtype=dtype, scale=3.0)
    r[:, dim // 2] *= 40
    if tokens > 2:
        x[1] = r[1] = 0                  # a row of nothing
        x[2] *= 2.0 ** -124              # below what 8-bit forms hold
        r[2] *= 2.0 ** -124
    if extra:
        x, r = defs.strided(x, extra), defs.strided(r, 2 * extra)
    return x, r


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,dim,extra", defs.NORM_SHAPES)
def test_forward_is_the_sum_and_its_norm(dtype, tokens, dim, extra):
    g = defs.gen(61)
    x, r = inputs(g, dtype, tokens, dim, extra)
    weight = 1.0 + defs.randn(g, dim, scale=0.2)
    out, total = Guarded(tokens * dim, dtype), Guarded(tokens * dim, dtype)
    y, h, kept = rcc.add_rmsnorm_forward(x, r, weight, eps=1e-5, keep=True,
                                         out=out.t.view(tokens, dim), h=total.t.view(tokens, dim))
    want = (x.float() + r.float()).to(dtype)
    assert torch.equal(h, want) and h.data_ptr() == total.t.data_ptr()
    y2, kept2 = rcc.rmsnorm_forward(want, weight, eps=1e-5, keep=True)
    assert torch.equal(y, y2) and torch.equal(kept.data, kept2.data)
    assert out.guards_intact() and total.guards_intact()
    # nothing kept; in place of the residual, and of x
    for name in ("r", "x"):
        xs, rs = x.contiguous().clone(), r.contiguous().clone()
        place = xs if name == "x" else rs
        y3, h3 = rcc.add_rmsnorm_forward(xs, rs, weight, eps=1e-5, h=place)
        assert h3.data_ptr() == place.data_ptr()
        assert torch.equal(h3, want) and torch.equal(y3, y)
    # a vector type that is not on its boundary
    if dim % 8 == 0:
        odd = Guarded(tokens * dim, dtype, offset_elems=1, fill=x.reshape(-1))
        assert torch.equal(rcc.add_rmsnorm_forward(odd.t.view(tokens, dim), r, weight,
                                                   eps=1e-5)[1], want)


def eight_reference(y):
    """The 8-bit form of fp32 values, operation for operation."""
    t, d = y.shape
    n = -(-d // 128)
    v = torch.zeros(t, n * 128, device=DEV)
    v[:, :d] = y
    v = v.view(t, n, 128)
    top = v.abs().amax(2, keepdim=True)
    small = top < 2.0 ** -120
    inv = torch.where(small, 0.0, 448.0 * (1.0 / top))
    q = (v * inv).clamp(-448, 448).to(E4M3).view(t, -1)[:, :d].contiguous()
    return q, torch.where(small, 0.0, top * (1.0 / 448.0))[:, :, 0]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("tokens,dim,extra", defs.NORM_SHAPES)
def test_eight_bit_output_of_fp32(residual, tokens, dim, extra):
    g = defs.gen(62)
    x, r = inputs(g, F32, tokens, dim, extra)
    r = r if residual else None
    weight = 1.0 + defs.randn(g, dim, scale=0.2)
    n = -(-dim // 128)
    values, scales = GuardedBytes(tokens * dim), Guarded(tokens * n, F32)
    out = rcc.Scaled(values.t.view(E4M3).view(tokens, dim), scales.t.view(tokens, n))
    y, h, kept = rcc.add_rmsnorm_forward(x, r, weight, out=out, keep=True)
    assert y is out and (h is None) == (r is None)
    h = x if r is None else h
    y32, kept2 = rcc.rmsnorm_forward(h, weight, keep=True)
    q, s = eight_reference(y32)
    assert torch.equal(y.values.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(y.scales, s) and torch.equal(kept.data, kept2.data)
    assert values.guards_intact() and scales.guards_intact()
    y, h = rcc.add_rmsnorm_forward(x, r, weight, out_dtype=E4M3)
    assert torch.equal(y.values.view(torch.uint8), q.view(torch.uint8))
    # half a step: 2^-4 of a value, or half of 2^-9 of a scale; the scale and the
    # product are each rounded
    back = y.dequantize()
    bound = y32.abs() * (2.0 ** -4 + 8 * U) + \
        y.scales.repeat_interleave(128, 1)[:, :dim] * 2.0 ** -10 + 2.0 ** -120
    assert bool(((back.double() - y32.double()).abs() <= bound).all())


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("tokens,dim,extra", defs.NORM_SHAPES)
def test_eight_bit_output_of_bf16(residual, tokens, dim, extra):
    g = defs.gen(63)
    x, r = inputs(g, BF16, tokens, dim, extra)
    weight = 1.0 + defs.randn(g, dim, scale=0.2)
    y, h = rcc.add_rmsnorm_forward(x, r if residual else None, weight, eps=1e-5, out_dtype=E4M3)
    x64 = (h if residual else x).double()
    want = x64 / (x64.square().mean(1, keepdim=True) + np.float32(1e-5)).sqrt() * weight.double()
    n = -(-dim // 128)
    v = torch.zeros(tokens, n * 128, device=DEV, dtype=torch.float64)
    v[:, :dim] = want
    top = v.view(tokens, n, 128).abs().amax(2)
    held = top >= 2.0 ** -119
    # 48 U of the norm itself (test_rmsnorm), two roundings of the scale
    assert bool(((y.scales.double() - top / 448).abs()[held] <= (52 * U * top / 448)[held]).all())
    bound = want.abs() * (2.0 ** -4 + 64 * U) + \
        (top / 448).repeat_interleave(128, 1)[:, :dim] * (2.0 ** -10 + 64 * U) + 2.0 ** -119
    defs.within(y.dequantize(), want, bound)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,dim,extra", defs.NORM_SHAPES)
def test_backward(dtype, tokens, dim, extra):
    g = defs.gen(64)
    x, r = inputs(g, dtype, tokens, dim, extra)
    weight = 1.0 + defs.randn(g, dim, scale=0.2)
    eps = 1e-5
    _, _, kept = rcc.add_rmsnorm_forward(x, r, weight, eps=eps, keep=True)
    dy, dh = defs.randn(g, tokens, dim, dtype=dtype), defs.randn(g, tokens, dim, dtype=dtype)
    if extra:
        dy, dh = defs.strided(dy, extra), defs.strided(dh, 3 * extra)
    grad, dweight = Guarded(tokens * dim, dtype), Guarded(dim, F32)
    rcc.add_rmsnorm_backward(dy, dh, kept, weight, eps=eps, dx=grad.t.view(tokens, dim),
                             dweight=dweight.t)
    x64, w64 = kept.dequantize().double(), weight.double()
    s64 = kept.scales.double()[:, :, None] * kept.values.double().view(tokens, -1, 128)
    x64 = s64.view(tokens, -1)[:, :dim]
    rr = 1 / (x64.square().mean(1, keepdim=True) + np.float32(eps)).sqrt()
    n, d = x64 * rr, dy.double() * w64
    inner = rr * (d - n * (d * n).mean(1, keepdim=True))
    size = rr * (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True))
    want = dh.double() + inner
    # the norm's own bound (test_rmsnorm), one more addition, one rounding
    defs.within(grad.t.view(tokens, dim), want,
                256 * U * size + U * want.abs() + 2.0 ** -149 + defs.half_ulp(want, dtype))
    terms = dy.double() * n
    defs.within(dweight.t, terms.sum(0), (tokens + 64) * U * terms.abs().sum(0) + 2.0 ** -140)
    assert grad.guards_intact() and dweight.guards_intact()
    alone, _ = rcc.rmsnorm_backward(dy, kept, weight, eps=eps)
    # without another use of h; in place of dh; added to a gradient
    dx, dw = rcc.add_rmsnorm_backward(dy, None, kept, weight, eps=eps)
    assert torch.equal(dx, alone)
    place = dh.contiguous().clone()
    base = defs.randn(g, dim)
    need = rcc.rmsnorm_backward_workspace(tokens, dim)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    dx, added = rcc.add_rmsnorm_backward(dy, place, kept, weight, eps=eps, dx=place,
                                         dweight=base.clone(), accumulate=True, workspace=ws)
    assert dx.data_ptr() == place.data_ptr() and torch.equal(place, grad.t.view(tokens, dim))
    assert torch.equal(added, base + dweight.t)


def test_gradient_against_differences():
    """Central differences of <dy, norm(x + r)> + <dh, x + r> in 64 bits, at the
    kept sum; each of the two inputs has the whole gradient."""
    g = defs.gen(65)
    tokens, dim = 4, 300
    weight = 1.0 + defs.randn(g, dim, scale=0.2)
    _, _, kept = rcc.add_rmsnorm_forward(defs.randn(g, tokens, dim), defs.randn(g, tokens, dim),
                                         weight, keep=True)
    dy, dh = defs.randn(g, tokens, dim), defs.randn(g, tokens, dim)
    dx, dweight = rcc.add_rmsnorm_backward(dy, dh, kept, weight)
    at, w = kept.dequantize().double(), weight.double()

    def f(h, w):
        y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * w
        return float((dy.double() * y + dh.double() * h).sum())

    step = 1e-5
    for _ in range(3):
        along, aw = defs.randn(g, tokens, dim).double(), defs.randn(g, dim).double()
        diff = (f(at + step * along, w + step * aw) - f(at - step * along, w - step * aw)) / (2 * step)
        got = float((dx.double() * along).sum() + (dweight.double() * aw).sum())
        size = float((dx.double().abs() * along.abs()).sum() +
                     (dweight.double().abs() * aw.abs()).sum())
        assert abs(diff - got) <= 1e-5 * size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite(dtype, bad):
    """It reaches its row: h, y or the scales of its 8-bit form, and the gradient."""
    g = defs.gen(66)
    x, r = defs.randn(g, 3, 300, dtype=dtype), defs.randn(g, 3, 300, dtype=dtype)
    x[1, 140] = bad
    weight = torch.ones(300, device=DEV)
    y, h, kept = rcc.add_rmsnorm_forward(x, r, weight, keep=True)
    assert not torch.isfinite(h[1, 140]) and not torch.isfinite(y[1]).all()
    assert torch.isfinite(y[[0, 2]]).all()
    y8, _ = rcc.add_rmsnorm_forward(x, r, weight, out_dtype=E4M3)
    assert torch.isnan(y8.scales).any(1).tolist() == [False, True, False]
    assert not torch.isfinite(y8.dequantize()[1]).all()
    assert torch.isfinite(y8.dequantize()[[0, 2]]).all()
    dx, dweight = rcc.add_rmsnorm_backward(torch.ones_like(x), h, kept, weight)
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[[0, 2]]).all()
    assert torch.isnan(dweight).all()


def test_sums_that_overflow_their_type():
    x = torch.full((1, 64), 3e38, device=DEV)
    y, h = rcc.add_rmsnorm_forward(x, x, torch.ones(64, device=DEV))
    assert torch.isinf(h).all() and not torch.isfinite(y).any()
    y8, _ = rcc.add_rmsnorm_forward(x, -x, torch.ones(64, device=DEV), out_dtype=E4M3)
    assert not y8.dequantize().any() and not y8.scales.any()


def test_no_tokens():
    weight = torch.ones(40, device=DEV)
    x = torch.empty(0, 40, device=DEV)
    y, h, kept = rcc.add_rmsnorm_forward(x, x, weight, keep=True)
    assert y.shape == h.shape == (0, 40)
    with pytest.raises(rcc.RccError):
        rcc.add_rmsnorm_forward(x, x, weight, eps=-1.0)
    y8, _ = rcc.add_rmsnorm_forward(x, None, weight, out_dtype=E4M3)
    assert y8.values.shape == (0, 40) and y8.scales.shape == (0, 1)
    base = torch.ones(40, device=DEV)
    dx, dw = rcc.add_rmsnorm_backward(x, x, kept, weight, dweight=base.clone(), accumulate=True)
    assert dx.shape == (0, 40) and torch.equal(dw, base)
    assert not rcc.add_rmsnorm_backward(x, x, kept, weight, dweight=base.clone())[1].any()


def test_refusals_on_the_gpu():
    x, weight = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    for more in (dict(h=x[:, :32]), dict(out=x), dict(eps=-1.0)):
        with pytest.raises((ValueError, rcc.RccError)):
            rcc.add_rmsnorm_forward(x, x.clone(), weight, **more)
    wide = torch.zeros(4, 128, device=DEV)
    with pytest.raises((ValueError, rcc.RccError)):   # a strided residual is not written over
        rcc.add_rmsnorm_forward(x, wide[:, :64], weight, h=wide[:, :64])
    with pytest.raises(ValueError):
        rcc.add_rmsnorm_forward(x, x.cpu(), weight)


def test_many_rows_and_a_captured_call():
    """Blocks take several rows each; the captured calls give the same bits."""
    g = defs.gen(67)
    for dtype, dim in ((BF16, 4096), (F32, 520), (BF16, 1000)):
        x, r = defs.randn(g, 5000, dim, dtype=dtype), defs.randn(g, 5000, dim, dtype=dtype)
        weight = 1.0 + defs.randn(g, dim, scale=0.2)

        def step():
            y, h, kept = rcc.add_rmsnorm_forward(x, r, weight, keep=True)
            y8, _ = rcc.add_rmsnorm_forward(x, r, weight, out_dtype=E4M3)
            dx, dw = rcc.add_rmsnorm_backward(y, h, kept, weight)
            return y, h, kept.data, y8.values.view(torch.uint8), y8.scales, dx, dw
        want = step()
        y2, kept2 = rcc.rmsnorm_forward(want[1], weight, keep=True)
        assert torch.equal(want[1], (x.float() + r.float()).to(dtype))
        assert torch.equal(want[0], y2) and torch.equal(want[2], kept2.data)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [9, 257, 1001, 2047, 4095, 4096, 20001])
def test_rows_anywhere(dtype, dim):
    """Rows that are on no boundary, their neighbours NaN: the bits of rows that
    stand alone, in blocks that take many of them."""
    g = defs.gen(68)
    tokens = 7 if dim > 5000 else 3000 if dim > 300 else 9000
    clean = [defs.randn(g, tokens, dim, dtype=dtype) for _ in range(2)]
    weight = 1.0 + defs.randn(g, dim, scale=0.2)

    def place(t, offset, extra):
        wide = torch.full((offset + tokens * (dim + extra),), float("nan"), dtype=dtype, device=DEV)
        rows = wide[offset:].view(tokens, dim + extra)[:, :dim]
        rows.copy_(t)
        return rows

    def run(offset, extra):
        x, r = place(clean[0], offset, extra), place(clean[1], 1, 2 * extra + 1)
        y, h, kept = rcc.add_rmsnorm_forward(x, r, weight, keep=True)
        y8, _ = rcc.add_rmsnorm_forward(x, r, weight, out_dtype=E4M3)
        dx, dw = rcc.add_rmsnorm_backward(x, r, kept, weight)
        alone, kept2 = rcc.rmsnorm_forward(place(h, offset, extra), weight, keep=True)
        assert torch.equal(alone, y) and torch.equal(kept2.data, kept.data)
        return y, h, kept.data, y8.values.view(torch.uint8), y8.scales, dx, dw
    want = run(1, 1)
    assert torch.equal(want[1], (clean[0].float() + clean[1].float()).to(dtype))
    assert torch.isfinite(want[5]).all() and torch.isfinite(want[6]).all()
    for offset, extra in ((3, 0), (0, 3), (7, 6), (5, 8)):
        assert all(torch.equal(a, b) for a, b in zip(run(offset, extra), want))
    # in place, each row written once it has been read
    x, r = place(clean[0], 1, 1), clean[1].clone()
    y, h = rcc.add_rmsnorm_forward(x, r, weight, h=r)
    assert h.data_ptr() == r.data_ptr() and torch.equal(h, want[1]) and torch.equal(y, want[0])
    dh = want[1].clone()
    dx, _ = rcc.add_rmsnorm_backward(place(clean[0], 1, 0), dh, rcc.Kept(tokens, dim, data=want[2]),
                                     weight, dx=dh)
    again, _ = rcc.add_rmsnorm_backward(place(clean[0], 3, 1), want[1],
                                        rcc.Kept(tokens, dim, data=want[2]), weight)
    assert dx.data_ptr() == dh.data_ptr() and torch.equal(dx, again)
