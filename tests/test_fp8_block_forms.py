"""The forms of the FP8 product (vector, single CTAs, CTA pairs, split reduction), each on the groups, widths and
contents where it can go wrong.  The library chooses a form by an estimated time and leaves it in word 7 of
the workspace; a test that means one form grows its problem until that form runs, or fails.

Against fp64 on the GPU with the bound of test_fp8_block.py: u |ref| + (blocks + 16) 2^-22 sum |terms|.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_fp8_block import DTYPES, NAN_CODES, SMALLEST, U, ceil_div, make_rows, make_weights, offsets_of, workspace

pytestmark = pytest.mark.gpu
VECTOR, SINGLE, PAIR, SPLIT = 1, 2, 3, 4


def values(codes, scales, block_rows):
    rows, K = codes.shape
    s = scales.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).double() * s


def product(x, xs, w, ws, offsets, out_dtype, dgrad=False):
    """The product of GPU tensors and the form that ran."""
    E, N, K = w.shape
    M = x.shape[0]
    out = torch.full((M, K if dgrad else N), -77.0, dtype=out_dtype, device="cuda")
    space = workspace(M, N, K, E)
    call = moe.moe_gemm_fp8_block_dgrad if dgrad else moe.moe_gemm_fp8_block
    call(x, xs, w, ws, out, space, offsets=offsets)
    assert moe.moe_read_device_status(space) == 0
    return out, int(space.view(torch.int32)[7])


def problem(M, N, K, E, dgrad, seed):
    w, ws = make_weights(E, N, K, seed)
    x, xs = make_rows(M, N if dgrad else K, seed + 10)
    return [t.cuda() for t in (x, xs, w, ws)]


def check(args, out, counts, out_dtype, dgrad):
    x, xs, w, ws = args
    off = offsets_of(counts).tolist()
    X, red = values(x, xs, 1), x.shape[1]
    for e in range(len(counts)):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        W = values(w[e], ws[e], 128)
        B = W if dgrad else W.t()
        ref, size = X[a:b] @ B, X[a:b].abs() @ B.abs()
        bound = U[out_dtype] * ref.abs() + (ceil_div(red, 128) + 16) * 2.0 ** -22 * size + SMALLEST[out_dtype]
        fits = ref.abs() < (65504.0 if out_dtype == torch.float16 else float("inf")) * 0.99
        err = (out[a:b].double() - ref).abs()
        assert bool((err <= bound)[fits].all()), f"expert {e}: worst {float((err / bound)[fits].max()):.3g}"
    assert bool((out[off[-1]:] == -77.0).all())


SPLIT_GROUPS = [[3, 0, 1, 4, 0, 0, 8, 0], [0, 0, 0, 5], [0, 40, 0, 0, 1], [17, 16, 31], [0, 130, 0, 2]]


@pytest.mark.parametrize("counts", SPLIT_GROUPS)
@pytest.mark.parametrize("cols", [512, 272, 250])
@pytest.mark.parametrize("dgrad", [False, True])
def test_split_reduction_over_groups(counts, cols, dgrad):
    """Tiles found by the search over groups, clusters beyond the last tile (empty groups), rows that no group holds."""
    if dgrad:
        cols = ceil_div(cols, 16) * 16
    N, K = (4096, cols) if dgrad else (cols, 4096)
    for extra, out_dtype in ((0, torch.bfloat16), (3, torch.float32)):
        args = problem(sum(counts) + extra, N, K, len(counts), dgrad, len(counts))
        out, form = product(*args, offsets_of(counts).cuda(), out_dtype, dgrad)
        assert form == SPLIT
        check(args, out, counts, out_dtype, dgrad)


def on_pairs(N, K, dgrad, out_dtype, seed):
    """Ragged groups, the smallest of a growing sequence that runs on pairs: (arguments, output, counts)."""
    for s in (1, 2, 4, 8, 16, 32):
        counts = [523 * s, 0, 15, 1200 * s + 7, 33]
        args = problem(sum(counts) + 2, N, K, len(counts), dgrad, seed)
        out, form = product(*args, offsets_of(counts).cuda(), out_dtype, dgrad)
        if form == PAIR:
            return args, out, counts
    pytest.fail("no size ran on pairs")


# Output rows on 32, 16, 8 and 4 bytes and off them, tiles' whole columns and the rest; long reductions, from which
# 16-bit rows off the 4-byte boundaries leave through the staging, and shorter ones
@pytest.mark.parametrize("cols", [1040, 1032, 1036, 1034, 1033])
@pytest.mark.parametrize("red", [1040, 2064])
@pytest.mark.parametrize("out_dtype", DTYPES)
def test_pair_rows_on_and_off_the_boundaries(cols, red, out_dtype):
    args, out, counts = on_pairs(cols, red, False, out_dtype, cols)
    check(args, out, counts, out_dtype, False)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_pair_gradient(out_dtype):
    args, out, counts = on_pairs(2064, 1040, True, out_dtype, 3)
    check(args, out, counts, out_dtype, True)


@pytest.mark.parametrize("counts,N,K", [([1] * 16, 200, 400), ([17], 1000, 272), ([8] * 8, 1000, 1040)])
def test_few_rows_off_the_wide_boundaries_run_on_single_ctas(counts, N, K):
    """Rows on 16 but not 32 bytes, fewer than a TMA store's 32 a group: a pair's stores would not run under the
    next tile's sums, and pairs are the slower form."""
    args = problem(sum(counts), N, K, len(counts), False, N)
    out, form = product(*args, offsets_of(counts).cuda(), torch.bfloat16)
    assert form == SINGLE
    check(args, out, counts, torch.bfloat16, False)


def test_vector_form():
    for counts, E in (([1], 1), ([0, 2, 0, 1, 1], 5)):
        args = problem(sum(counts), 129, 1040, E, False, E)
        out, form = product(*args, offsets_of(counts).cuda(), torch.float32)
        assert form == VECTOR
        check(args, out, counts, torch.float32, False)


def check_contained(run, args, out, counts, out_dtype, dgrad):
    """A NaN code, an infinite scale and a NaN weight change their own row, row and column, and no other bit, rows of
    the neighbouring groups in the same 32 among them."""
    x, xs, w, ws = args
    off = offsets_of(counts).tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(len(counts)) if counts[e] > 0]
    last, first = spans[0][2] - 1, spans[1][1]  # neighbours of two groups
    e = spans[2][0]
    x2, xs2, w2 = x.clone(), xs.clone(), w.clone()
    x2[last, 3] = NAN_CODES[0]
    xs2[first, 0] = float("inf")
    w2[e, 7, 9] = NAN_CODES[1]
    col = 9 if dgrad else 7
    got = run(x2, xs2, w2, ws)
    rows = torch.arange(out.shape[0], device="cuda")
    cols = torch.arange(out.shape[1], device="cuda")
    inside = (rows >= spans[2][1]) & (rows < spans[2][2])
    touched = (rows == last)[:, None] | (rows == first)[:, None] | (inside[:, None] & (cols == col))
    assert bool(torch.isnan(got[last]).all()) and not bool(torch.isfinite(got[first]).any())
    assert bool(torch.isnan(got[inside][:, col]).all())
    assert torch.equal(got[~touched], out[~touched])


@pytest.mark.parametrize("cols", [1040, 1033])
@pytest.mark.parametrize("dgrad", [False, True])
def test_nan_and_inf_stay_in_their_row_and_column_on_pairs(cols, dgrad):
    if dgrad:
        cols = ceil_div(cols, 16) * 16
    N, K = (2064, cols) if dgrad else (cols, 2064)
    args, out, counts = on_pairs(N, K, dgrad, torch.float32, 5)

    def run(*changed):
        got, form = product(*changed, offsets_of(counts).cuda(), torch.float32, dgrad)
        assert form == PAIR
        return got

    check_contained(run, args, out, counts, torch.float32, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
def test_nan_and_inf_stay_in_their_row_and_column_under_a_split(dgrad):
    counts = [9, 0, 14, 3, 0, 0]
    N, K = (4096, 272) if dgrad else (272, 4096)
    args = problem(sum(counts), N, K, len(counts), dgrad, 6)

    def run(*changed):
        got, form = product(*changed, offsets_of(counts).cuda(), torch.float32, dgrad)
        assert form == SPLIT
        return got

    check_contained(run, args, run(*args), counts, torch.float32, dgrad)
