"""The gated FP8 product in each of its forms (vector, single CTAs, CTA pairs, split reduction), both layouts, and
everything that it can leave: h, its codes, the products.

Against fp64 on the GPU.  A product is off by e = (blocks + 16) 2^-22 sum |terms| (the bound of test_fp8_block.py), so
h = silu(g) u is off by 1.1 |u| e_g + |silu(g)| e_u + 1.1 e_g e_u (|silu'| < 1.1) and by the logistic function's
(5 + 1.173 |g|) 2^-23 and three roundings of itself (test_swiglu_backward.py); a stored value adds half a step.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_fp8_block import NAN_CODES, ceil_div, make_rows, make_weights, offsets_of, workspace
from test_fp8_block_forms import PAIR, SINGLE, SPLIT, VECTOR, values
from test_rms_norm import BF16, F16, F32, F64, HALF, SMALL, U
from test_swiglu_backward import check_codes, halves

pytestmark = pytest.mark.gpu
TURN, STACK = moe.MOE_GATE_UP_INTERLEAVED, moe.MOE_GATE_UP_STACKED
FILL = -77.0


def problem(M, I, K, E, seed, tame=False):
    """Codes and scales of wide ranges, whose gates are far out on either side; or ``tame``: gates of a few units."""
    w, ws = make_weights(E, 2 * I, K, seed)
    x, xs = make_rows(M, K, seed + 10)
    args = [t.cuda() for t in (x, xs, w, ws)]
    if tame and M:
        size = (values(args[0], args[1], 1) @ values(args[2][0], args[3][0], 128).t()).std().clamp_min(1e-30)
        args[3] *= torch.exp2(torch.round(torch.log2(3.0 / size))).float()
    return args


def product(args, offsets, layout, dtype, out=True, codes=True, keep=True):
    x, xs, w, ws = args
    (E, N, K), M = w.shape, x.shape[0]
    I = N // 2
    got = {"out": torch.full((M, I), FILL, dtype=dtype, device="cuda") if out else None,
           "codes": torch.full((M, I), 0x55, dtype=torch.uint8, device="cuda") if codes else None,
           "scales": torch.full((M, ceil_div(I, 128)), FILL, device="cuda") if codes else None,
           "gate_up": torch.full((M, N), FILL, dtype=dtype, device="cuda") if keep else None}
    space = workspace(M, N, K, E)
    moe.moe_gemm_fp8_block_swiglu(x, xs, w, ws, space, layout=layout, offsets=offsets, **got)
    if M == 0:  # a call without rows leaves the workspace as it is
        return got, None
    assert moe.moe_read_device_status(space) == 0
    return got, int(space.view(torch.int32)[7])


def reference(args, counts, layout):
    """(products, their bound, h, its bound) in fp64 for the rows that groups hold."""
    x, xs, w, ws = args
    off = offsets_of(counts).tolist()
    X = values(x, xs, 1)
    v, e = (torch.zeros(off[-1], w.shape[1], dtype=F64, device="cuda") for _ in range(2))
    for i in range(len(counts)):
        a, b = off[i], off[i + 1]
        if a < b:
            W = values(w[i], ws[i], 128)
            v[a:b], e[a:b] = X[a:b] @ W.t(), X[a:b].abs() @ W.t().abs()
    e *= (ceil_div(x.shape[1], 128) + 16) * 2.0 ** -22
    (g, u), (eg, eu) = halves(v, layout), halves(e, layout)
    sig = torch.sigmoid(g)
    h = g * sig * u
    eh = 1.1 * u.abs() * eg + (g * sig).abs() * eu + 1.1 * eg * eu + h.abs() * ((5 + 1.173 * g.abs()) * 2.0 ** -23 + 3 * U)
    return v, e, h, eh + (1 + (g * u).abs()) * 2.0 ** -60  # a logistic function below 2^-60 is 2^-60 or 0


def check(args, got, counts, layout, dtype):
    v, e, h, eh = reference(args, counts, layout)
    R = v.shape[0]
    top = 65504.0 * 0.99 if dtype == F16 else float("inf")
    for name, want, off in (("out", h, eh), ("gate_up", v, e)):
        t = got[name]
        if t is None:
            continue
        err, bound = (t[:R].to(F64) - want).abs(), HALF[dtype] * want.abs() + off + SMALL[dtype]
        past = want.abs() + bound > top  # a value that far off may round to f16's infinity
        assert bool(((err <= bound) | past).all()), f"{name}: worst {float((err / bound)[~past].max()):.3g}"
        assert bool((t[R:] == FILL).all())
    if got["codes"] is not None and R:
        check_codes(got["codes"][:R], got["scales"][:R], h, eh)
    if got["codes"] is not None:
        assert bool((got["codes"][R:] == 0x55).all()) and bool((got["scales"][R:] == FILL).all())


def run(counts, I, K, layout, dtype, form=None, E=None, extra=0, seed=0, grouped=True, **what):
    for tame in (False, True):
        args = problem(sum(counts) + extra, I, K, len(counts), seed, tame)
        got, ran = product(args, offsets_of(counts).cuda() if grouped else None, layout, dtype, **what)
        if form is not None:
            assert ran == form
        check(args, got, counts, layout, dtype)
    return args, got, ran


CODES = lambda I: I % 16 == 0  # noqa: E731


@pytest.mark.parametrize("I", [1, 63, 64, 100, 128, 144, 512, 1152])
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_vector(I, layout):
    if layout == STACK and I % 128:
        I = 128 * ceil_div(I, 128)
    for M, dtype in ((1, BF16), (2, F32), (3, F16), (4, BF16)):
        run([M], I, 1040, layout, dtype, VECTOR, grouped=False, codes=CODES(I))
    run([0, 2, 0, 1, 1], I, 272, layout, BF16, VECTOR, codes=CODES(I))
    run([0, 1, 0], I, 272, layout, BF16, VECTOR, codes=CODES(I), extra=2)


@pytest.mark.parametrize("counts", [[3, 0, 1, 4, 0, 0, 8, 0], [0, 0, 0, 5], [0, 40, 0, 0, 1], [17, 16, 31], [0, 130, 0, 2]])
@pytest.mark.parametrize("I", [256, 144, 136, 125])
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_split(counts, I, layout):
    if layout == STACK:
        I = 128 * ceil_div(I, 128)
    run(counts, I, 4096, layout, BF16, SPLIT, codes=CODES(I), extra=3)
    run(counts, I, 4096, layout, F32, SPLIT, codes=CODES(I), keep=False)
    if CODES(I):
        run(counts, I, 4096, layout, F16, SPLIT, out=False, keep=False)


@pytest.mark.parametrize("S,I,M", [(2, 2048, 100), (4, 1024, 100), (8, 512, 100), (2, 4096, 5), (4, 2304, 128)])
def test_split_widths(S, I, M):
    """Few and many columns of h a CTA of the cluster."""
    run([M], I, 5120, TURN, BF16, SPLIT, grouped=False)


@pytest.mark.parametrize("I", [384, 400, 392, 396, 395, 65, 1])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_single(I, dtype, layout):
    if layout == STACK:
        I = 128 * ceil_div(I, 128)
    counts = [37, 0, 15, 1, 64, 130, 0, 33, 5] * 9
    run(counts, I, 400, layout, dtype, SINGLE, codes=CODES(I), extra=5)
    run(counts, I, 144, layout, dtype, SINGLE, codes=CODES(I), keep=False)
    if CODES(I):
        run(counts, I, 144, layout, dtype, SINGLE, out=False, keep=False)


def on_pairs(I, K, layout, dtype, seed, tame=False, **what):
    for s in (1, 2, 4, 8, 16, 32):
        counts = [523 * s, 0, 15, 1200 * s + 7, 33]
        args = problem(sum(counts) + 2, I, K, len(counts), seed, tame)
        got, form = product(args, offsets_of(counts).cuda(), layout, dtype, **what)
        if form == PAIR:
            return args, got, counts
    pytest.fail("no size ran on pairs")


@pytest.mark.parametrize("I", [512, 528, 520, 516, 514, 513, 560])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_pairs(I, dtype, layout):
    if layout == STACK:
        I = 128 * ceil_div(I, 128)
    for what in (dict(), dict(tame=True), dict(keep=False), dict(out=False, keep=False), dict(out=False, tame=True)):
        if not CODES(I) and what.get("out") is False:
            continue
        args, got, counts = on_pairs(I, 2064, layout, dtype, I, codes=CODES(I), **what)
        check(args, got, counts, layout, dtype)


@pytest.mark.parametrize("form", ["single", "pair", "split", "vector"])
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_nan_and_inf_stay_in_their_row_and_block(form, layout):
    """A NaN code, an infinite scale and a NaN weight change their row, and their column in the rows of their expert;
    an infinite or NaN h leaves its block's scale to the other columns."""
    I, K = 256, 4096 if form == "split" else 1040
    counts = {"single": [37, 15, 64, 130, 33] * 9, "pair": None, "split": [9, 14, 3], "vector": [1, 1, 1]}[form]
    if form == "pair":
        args, got, counts = on_pairs(I, K, layout, F32, 5)
    else:
        args, got, ran = run(counts, I, K, layout, F32)
        assert ran == {"single": SINGLE, "split": SPLIT, "vector": VECTOR}[form]
    x, xs, w, ws = args
    off = offsets_of(counts).tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(len(counts)) if counts[e] > 0]
    last, first, (e, a, b) = spans[0][2] - 1, spans[1][1], spans[2]
    x2, xs2, w2 = x.clone(), xs.clone(), w.clone()
    x2[last, 3] = NAN_CODES[0]
    xs2[first, 0] = float("inf")
    w2[e, 14, 9] = NAN_CODES[1]  # gate row 7, or 14
    col = 14 if layout == STACK else 7
    new, _ = product((x2, xs2, w2, ws), offsets_of(counts).cuda(), layout, F32)
    rows, cols = torch.arange(x.shape[0], device="cuda"), torch.arange(I, device="cuda")
    inside = (rows >= a) & (rows < b)
    touched = (rows == last)[:, None] | (rows == first)[:, None] | (inside[:, None] & (cols == col))
    assert bool(torch.isnan(new["out"][last]).all()) and not bool(torch.isfinite(new["gate_up"][first]).any())
    assert bool(torch.isnan(new["out"][inside][:, col]).all())
    # Columns 2j and 2j + 1 share a reciprocal: the neighbour of the NaN's column keeps its value, within what two
    # logistic functions may differ by, and every other element keeps its bits.
    beside = inside[:, None] & (cols == (col ^ 1)) & ~touched
    assert torch.equal(new["out"][~touched & ~beside], got["out"][~touched & ~beside])
    gate = halves(got["gate_up"], layout)[0].to(F64)
    apart = (new["out"].to(F64) - got["out"].to(F64)).abs()
    bound = got["out"].to(F64).abs() * ((10 + 2.4 * gate.abs()) * 2.0 ** -23 + 6 * U) + 2.0 ** -126
    assert bool((apart <= bound)[beside].all())
    assert bool(((new["codes"][inside][:, col] & 127) == 127).all()) and bool(((new["codes"][last] & 127) == 127).all())
    assert bool((new["scales"][last] == 0).all())
    other = ~touched & (~inside[:, None] | (cols >= 128))
    assert torch.equal(new["codes"][other], got["codes"][other])


def test_out_of_range_offsets_and_no_rows():
    args = problem(70, 128, 272, 3, 1)
    z = problem(0, 128, 272, 3, 1)
    product(z, torch.zeros(4, dtype=torch.int64, device="cuda"), TURN, BF16)
    got, _ = product(args, torch.tensor([-5, 30, 30, 900], device="cuda"), TURN, BF16)
    check(args, got, [30, 0, 40], TURN, BF16)
    got, _ = product(args, torch.tensor([0, 0, 0, 0], device="cuda"), TURN, BF16)
    assert bool((got["out"] == FILL).all()) and bool((got["codes"] == 0x55).all())


def test_same_as_the_steps_one_by_one():
    """h and its codes against moe_gemm_fp8_block, the activation in fp64 and moe_quantize_fp8_block: the same products
    bit for bit (kept in fp32), so h within its own roundings."""
    counts, I, K = [300, 0, 77, 5], 384, 1040
    args = problem(sum(counts), I, K, len(counts), 3)
    x, xs, w, ws = args
    got, _ = product(args, offsets_of(counts).cuda(), TURN, F32)
    v = torch.empty(sum(counts), 2 * I, device="cuda")
    moe.moe_gemm_fp8_block(x, xs, w, ws, v, workspace(sum(counts), 2 * I, K, len(counts)), offsets=offsets_of(counts).cuda())
    near = (got["gate_up"].to(F64) - v.to(F64)).abs() <= 2.0 ** -20 * v.to(F64).abs() + 1e-3 * 2.0 ** -10
    assert bool(near.all())
    check_codes(got["codes"], got["scales"], got["out"].to(F64), 2 * U * got["out"].to(F64).abs())


@pytest.mark.parametrize("M", [1, 40, 3000])
def test_graph_and_stream(M):
    args = problem(M, 256, 1040, 1, M)
    x, xs, w, ws = args
    out, codes = torch.empty(M, 256, dtype=BF16, device="cuda"), torch.empty(M, 256, dtype=torch.uint8, device="cuda")
    scales, space = torch.empty(M, 2, device="cuda"), workspace(M, 512, 1040, 1)
    call = lambda **a: moe.moe_gemm_fp8_block_swiglu(x, xs, w, ws, space, out=out, codes=codes, scales=scales, **a)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    new, ns = make_rows(M, 1040, M + 99)
    x.copy_(new)
    xs.copy_(ns)
    graph.replay()
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(space) == 0
    got = [t.clone() for t in (out, codes, scales)]
    call()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, codes, scales)))
    check(args, {"out": out, "codes": codes, "scales": scales, "gate_up": None}, [M], TURN, BF16)
