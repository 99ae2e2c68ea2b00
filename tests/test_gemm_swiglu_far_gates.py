"""The gated product with gates far below zero, where silu decays to nothing, in each of its forms.

Every row of x holds a single 1 and all scales are 1, so the products are exact: gate and up are the weights' own values.
The logistic function is off by (5 + 1.173 |g|) 2^-23 of itself, and 0 below 2^-126 (test_swiglu_backward.py), the two
multiplications by 2^-24 each: h = silu(g) u is held to that alone, however small it is.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_fp8_block import offsets_of
from test_fp8_block_forms import PAIR, SINGLE, SPLIT, VECTOR
from test_gemm_swiglu import STACK, TURN, product
from test_rms_norm import BF16, F32, F64, HALF, U
from test_swiglu_backward import check_codes

pytestmark = pytest.mark.gpu
I = 384
NEAR = [v * s for v in (0.5, 1.0, 3.25, 7.0, 13.0, 24.0, 40.0) for s in (1, -1)]
FAR = [-44.0, -48.0, -52.0, -56.0, -60.0]              # 2^-126 < sig < 2^-60, and far above 2^-100 / |g u|
GONE = [-128.0, -160.0, -224.0, -320.0, -448.0]        # sig < 2^-126
UP = [v * s for v in (1.0, 1.5, 2.75, 6.0) for s in (1, -1)]
FORMS = {
    "vector": (VECTOR, 528, lambda s: [1, 0, 2]),
    "split": (SPLIT, 4096, lambda s: [3, 0, 1, 4, 0, 0, 8, 0]),
    "single": (SINGLE, 400, lambda s: [37, 0, 15, 1, 64, 130, 0, 33, 5] * 9),
    "pair": (PAIR, 2064, lambda s: [523 * s, 0, 15, 1200 * s + 7, 33]),
}


def pick(g, values, *shape):
    return torch.tensor(values, device="cuda")[torch.randint(len(values), shape, generator=g, device="cuda")]


def problem(counts, K, layout, seed):
    """x, its scales, w, its scales, and gate and up of every row.  Columns [0, 128) of h have near gates with a few far
    ones among them, [128, 256) far ones alone, [256, 384) those whose logistic function is 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, M = len(counts), sum(counts)
    gate = torch.cat([pick(g, NEAR * 3 + FAR + GONE, E, 128, K), pick(g, FAR, E, 128, K), pick(g, GONE, E, 128, K)], 1)
    up = pick(g, UP, E, I, K)
    w = torch.cat([gate, up], 1) if layout == STACK else torch.stack([gate, up], 2).view(E, 2 * I, K)
    at = torch.randint(K, (M,), generator=g, device="cuda")
    x = torch.zeros(M, K, device="cuda")
    x[torch.arange(M, device="cuda"), at] = 1
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    codes = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    blocks = -(-K // 128)
    args = (codes(x), torch.ones(M, blocks, device="cuda"), codes(w), torch.ones(E, 2 * I // 128, blocks, device="cuda"))
    return args, gate[e, :, at].to(F64), up[e, :, at].to(F64), at


def run(form, layout, dtype, spoil=None, by=float("inf"), **what):
    want, K, sizes = FORMS[form]
    for s in (1, 2, 4, 8, 16, 32):
        counts = sizes(s)
        args, gate, up, at = problem(counts, K, layout, s)
        if spoil is not None:
            args[1][spoil, at[spoil] // 128] = by
        got, ran = product(args, offsets_of(counts).cuda(), layout, dtype, **what)
        if ran == want:
            return got, gate, up
    pytest.fail(f"no size ran as {form}")


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("layout", [TURN, STACK])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_gates(form, layout, dtype):
    got, gate, up = run(form, layout, dtype)
    h = gate * torch.sigmoid(gate) * up
    off = h.abs() * ((5 + 1.173 * gate.abs()) * 2.0 ** -23 + 3 * U) + (gate * up).abs() * 2.0 ** -126
    err = (got["out"].to(F64) - h).abs()
    assert bool((err <= off + HALF[dtype] * (h.abs() + off) + 2.0 ** -133).all()), f"worst {float((err / off).max()):.3g}"
    codes, scales = got["codes"], got["scales"]
    check_codes(codes[:, :256].contiguous(), scales[:, :2].contiguous(), h[:, :256].contiguous(), off[:, :256].contiguous())
    assert bool((scales[:, 2] == 0).all()) and bool(((codes[:, 256:] & 127) == 0).all())


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_infinite_gates(form, layout):
    """An infinite scale leaves its row without a finite h, and every other row its bits.  The tiles scale whole blocks of
    the reduction, none of which is 0 here: silu(-inf) is -inf times 0, silu(inf) is inf.  (The vector form scales a
    lane's 16 products, of which all but one are 0, and 0 times infinity is NaN.)"""
    clean, gate, up = run(form, layout, F32)
    got, _, _ = run(form, layout, F32, spoil=1)
    out, below = got["out"][1], gate[1] < 0
    assert not bool(torch.isfinite(out).any()) and bool(torch.isnan(out[below]).all())
    if form != "vector":
        assert bool((out[~below] == torch.sign(up[1][~below]) * float("inf")).all())
    rest = torch.arange(gate.shape[0], device="cuda") != 1
    assert torch.equal(got["out"][rest], clean["out"][rest]) and torch.equal(got["codes"][rest], clean["codes"][rest])


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_overflowing_gates(form, layout):
    """Products of 2^127 and more, finite or past fp32's range, in every form alike: fp32's own silu and products."""
    got, gate, up = run(form, layout, F32, spoil=1, by=2.0 ** 127)
    g, u = (t[1].float() * 2.0 ** 127 for t in (gate, up))
    want, out = g * torch.where(g < 0, 0.0, 1.0) * u, got["out"][1]
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and bool(torch.isnan(want).any())
    rest = ~torch.isnan(want)
    near = (out.to(F64) - want.to(F64)).abs() <= 8 * U * want.to(F64).abs()  # a sigmoid of 1, two products
    assert bool(((out == want) | near)[rest].all())
