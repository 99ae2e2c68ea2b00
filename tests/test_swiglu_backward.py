"""The gated activation's gradient against fp64, in both layouts, as values and as FP8 codes.

u = 2^-24.  The logistic function's exponent is off by 2^-23 |g| (a product and a rounded constant), its exponential and
reciprocal by 2^-22.5 and 2^-23 (PTX's bounds), its addition by u: together below d(g) = (5 + 1.173 |g|) 2^-23 of
itself, and a result below 2^-126 is 0: d sig + 2^-126 in all.  d_up = dh g sig: d + 3u.  d_gate = dh u sig (1 + g (1 -
sig)): the bracket is off by |g| (sig d + 2u) + 2u and the rest by d + 4u of itself.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_rms_norm import BF16, F16, F32, F64, HALF, SMALL, U, gen

pytestmark = pytest.mark.gpu
LAYOUTS = [moe.MOE_GATE_UP_INTERLEAVED, moe.MOE_GATE_UP_STACKED]


def matrix(g, R, C, dtype, stride=None, shift=0, scale=1.0):
    stride = C if stride is None else stride
    flat = torch.zeros(shift + R * stride + 16, dtype=dtype, device="cuda")
    m = flat[shift:shift + R * stride].view(R, stride)[:, :C]
    m.copy_(scale * torch.randn(R, C, generator=g, device="cuda"))
    return m


def halves(v, layout):
    I = v.shape[1] // 2
    return (v[:, :I], v[:, I:]) if layout == moe.MOE_GATE_UP_STACKED else (v[:, 0::2], v[:, 1::2])


def gradient64(gate_up, dh, layout):
    """(gradient, bound of the fp32 error) in fp64."""
    g, u = (t.to(F64) for t in halves(gate_up, layout))
    d = dh.to(F64)
    sig = torch.sigmoid(g)
    delta = (5 + 1.173 * g.abs()) * 2.0 ** -23
    grad, bound = torch.empty(gate_up.shape, dtype=F64, device="cuda"), torch.empty(gate_up.shape, dtype=F64, device="cuda")
    for out, gate, up in ((grad, d * u * sig * (1 + g * (1 - sig)), d * g * sig),
                          (bound, (d * u * sig).abs() * ((delta + 4 * U) * (1 + g * (1 - sig)).abs() +
                                                         g.abs() * (sig * delta + 2 * U) + 2 * U),
                           (d * g * sig).abs() * (delta + 3 * U))):
        a, b = halves(out, layout)
        a.copy_(gate)
        b.copy_(up)
    # 2^-126 on the logistic function, times what it multiplies; products below fp32's normal numbers, 2^-149 each
    for out, lost in zip(halves(bound, layout), ((d * u).abs() * (1 + g.abs()) + 1, (d * g).abs() + 1)):
        out.add_(lost * 2.0 ** -126)
    return grad, bound


def check_codes(codes, scales, v, off):
    """Codes and scales of values known to within `off`."""
    R, C = v.shape
    blocks = lambda t: torch.nn.functional.pad(t, (0, -C % 128)).view(R, -1, 128)  # noqa: E731
    m, e = blocks(v).abs().amax(2), blocks(off).amax(2)
    assert bool(((scales.to(F64) - m / 448).abs() <= e / 448 + 2 * U * m / 448).all())
    k = 448.0 / m.clamp_min(1e-300)[..., None]
    flat = lambda t: t.reshape(R, -1)[:, :C]  # noqa: E731
    q = flat(blocks(v) * k)
    slack = flat(blocks(off) * k) + q.abs() * (flat((e / m.clamp_min(1e-300))[..., None].expand_as(blocks(v))) + 2.0 ** -20 + 4 * U)
    code = codes.view(torch.float8_e4m3fn).to(F64)
    half = torch.maximum((q.abs() + slack) * 2.0 ** -4, torch.full_like(q, 2.0 ** -10))
    assert bool(((code - q).abs() <= half + slack).all())


def run(R, I, dtype, layout, codes=True, values=True, pad=0, shift=0, scale=1.5):
    g = gen(R + I)
    gate_up = matrix(g, R, 2 * I, dtype, 2 * I + pad, shift, scale)
    dh = matrix(g, R, I, dtype, I + pad, shift)
    hold = torch.full((R, 2 * I + pad), -77.0, dtype=dtype, device="cuda")
    d = hold[:, :2 * I] if values else None
    c = torch.full((R, 2 * I), 0x55, dtype=torch.uint8, device="cuda") if codes else None
    s = torch.full((R, -(-2 * I // 128)), -7.0, device="cuda") if codes else None
    moe.moe_swiglu_backward(gate_up, dh, d_gate_up=d, codes=c, scales=s, layout=layout)
    want, bound = gradient64(gate_up, dh, layout)
    if values:
        err = (d.to(F64) - want).abs()
        assert bool((err <= HALF[dtype] * want.abs() + bound * 1.01 + SMALL[dtype]).all())
        assert bool((hold[:, 2 * I:] == -77.0).all())
    if codes:
        check_codes(c, s, want, bound)
    return gate_up, dh, d, c, s


@pytest.mark.parametrize("I", [1, 3, 8, 32, 63, 64, 100, 128, 192, 256, 264, 640, 1152, 2049, 4104])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_gradient(I, dtype, layout):
    if layout == moe.MOE_GATE_UP_STACKED and I % 128:
        I = 128 * (I // 128 + 1)
    for R in (1, 9, 333):
        run(R, I, dtype, layout)
    run(5, I, dtype, layout, codes=False)
    run(5, I, dtype, layout, values=False)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (3, 5)])
def test_strides_and_alignment(layout, pad, shift):
    for dtype in (BF16, F32):
        run(37, 384, dtype, layout, pad=pad, shift=shift)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_in_place(layout):
    gate_up, dh, d, c, s = run(77, 640, BF16, layout)
    moe.moe_swiglu_backward(gate_up, dh, d_gate_up=gate_up, layout=layout)
    assert torch.equal(gate_up, d)


def test_far_gates():
    """Gates to +-120, where exp passes fp32's range: no NaN, and the bounds hold."""
    run(50, 256, F32, moe.MOE_GATE_UP_STACKED, scale=40.0)
    run(50, 256, F32, moe.MOE_GATE_UP_INTERLEAVED, scale=40.0)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_nan_stays_in_its_block(layout):
    gate_up, dh, d, c, s = run(6, 256, BF16, layout)
    bad = dh.clone()
    bad[2, 7] = float("nan")
    d2, c2, s2 = torch.empty_like(d), torch.empty_like(c), torch.empty_like(s)
    moe.moe_swiglu_backward(gate_up, bad, d_gate_up=d2, codes=c2, scales=s2, layout=layout)
    cols = [7, 256 + 7] if layout == moe.MOE_GATE_UP_STACKED else [14, 15]
    hit = torch.zeros(d.shape, dtype=torch.bool, device="cuda")
    hit[2, cols] = True
    assert bool(torch.isnan(d2[hit]).all()) and torch.equal(d2[~hit], d[~hit])
    assert bool(((c2[hit] & 127) == 127).all())
    blocks = sorted({k // 128 for k in cols})
    other = [b for b in range(4) if b not in blocks]
    assert torch.equal(s2[:, other], s[:, other]) and torch.equal(c2[[0, 1, 3, 4, 5]], c[[0, 1, 3, 4, 5]])


def test_gradient_by_differences():
    layout, h = moe.MOE_GATE_UP_INTERLEAVED, 1e-5
    gate_up, dh, d, _, _ = run(11, 40, F32, layout)
    e = torch.randn(11, 80, generator=gen(2), device="cuda", dtype=F64)

    def f(v):
        g, u = halves(v, layout)
        return float((g * torch.sigmoid(g) * u * dh.to(F64)).sum())
    along = (f(gate_up.to(F64) + h * e) - f(gate_up.to(F64) - h * e)) / (2 * h)
    assert abs(float((d.to(F64) * e).sum()) - along) <= 1e-5 * float((d.to(F64) * e).abs().sum())


def test_no_rows_and_graph():
    z = torch.empty(0, 256, dtype=BF16, device="cuda")
    moe.moe_swiglu_backward(torch.empty(0, 512, dtype=BF16, device="cuda"), z,
                            d_gate_up=torch.empty(0, 512, dtype=BF16, device="cuda"))
    gate_up, dh, d, c, s = run(40, 640, BF16, moe.MOE_GATE_UP_INTERLEAVED)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_swiglu_backward(gate_up, dh, d_gate_up=d, codes=c, scales=s)
    dh.copy_(torch.randn(40, 640, generator=gen(8), device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    want = [t.clone() for t in (d, c, s)]
    moe.moe_swiglu_backward(gate_up, dh, d_gate_up=d, codes=c, scales=s)
    assert all(torch.equal(a, b) for a, b in zip(want, (d, c, s)))
