"""FP8 with a scale for each block of 128: the quantiser and the products, against fp64.

Products: an output is u |ref| (rounding to its type) plus the error of its fp32 sums: a block's sum
is at most 5 accumulations of 32 exact products (a truncating one costs 2^-23 of the partial sum) and
the blocks add up in fp32, each with two roundings of its scaled value: at most
(blocks + 16) 2^-22 of the sum of |terms|.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe

gpu = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
NAN_CODES = (0x7F, 0xFF)


def ceil_div(a, b):
    return -(-a // b)


def decode(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


TABLE = decode(torch.arange(127, dtype=torch.uint8))


def nearest(v):
    """Index of the E4M3 code nearest to |v| <= 448, ties to the even code."""
    mid = (TABLE[1:] + TABLE[:-1]) / 2
    i = torch.searchsorted(mid, v.abs().contiguous())
    return i + ((v.abs() == mid[i.clamp(max=125)]) & (i % 2 == 1)).long()


def blocks_of(x, block_rows):
    """fp64 [rows, K] -> [row blocks, block_rows, column blocks, 128], padded with zeros."""
    rows, K = x.shape
    p = torch.zeros(ceil_div(rows, block_rows) * block_rows, ceil_div(K, 128) * 128, dtype=torch.float64)
    p[:rows, :K] = x
    return p.view(-1, block_rows, p.shape[1] // 128, 128)


def quantized(x, block_rows):
    """(codes uint8, scales fp64) from the definition in fp64, finite x."""
    rows, K = x.shape
    v = blocks_of(x.double(), block_rows)
    m = v.abs().amax((1, 3), keepdim=True)
    tiny = m < 2.0 ** -100
    q = torch.where(tiny, 0.0, v * 448 / torch.where(tiny, 1.0, m))
    codes = nearest(q).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 7)
    return codes.reshape(-1, v.shape[2] * 128)[:rows, :K], torch.where(tiny, 0.0, m / 448)[:, 0, :, 0]


def values(codes, scales, block_rows):
    rows, K = codes.shape
    s = scales.cpu().double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :K]
    return decode(codes) * s


def data(rows, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, K, generator=g) * torch.exp(0.7 * torch.randn(K, generator=g))).to(dtype)


def run_quant(x, block_rows=1):
    rows, K = x.shape
    codes = torch.full((rows, K), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((ceil_div(rows, block_rows), ceil_div(K, 128)), -1.0, device="cuda")
    moe.moe_quantize_fp8_block(x, codes, scales, block_rows)
    return codes.cpu(), scales.cpu()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 128), (2, 130), (7, 5120), (128, 128), (129, 1000), (300, 77), (64, 7168), (3, 65536)])
def test_quantize(rows, K, block_rows, dtype):
    x = data(rows, K, dtype, rows + K)
    codes, scales = run_quant(x.cuda(), block_rows)
    want, ws = quantized(x, block_rows)
    assert bool(((scales.double() - ws).abs() <= 2.0 ** -24 * ws).all())  # one rounded division
    if dtype != torch.float32:
        assert torch.equal(codes, want)
    else:  # a quotient within 2^-20 of a tie may take either neighbour
        off = codes != want
        v = blocks_of(x.double(), block_rows)
        q = (v * 448 / v.abs().amax((1, 3), keepdim=True)).reshape(-1, v.shape[2] * 128)[:rows, :K][off].abs()
        mid = (TABLE[1:] + TABLE[:-1]) / 2
        near = (q[:, None] / mid - 1).abs().amin(1)
        assert bool((near <= 2.0 ** -20).all()) and int(off.sum()) <= 1 + rows * K // 10000


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_every_tie(dtype):
    """Blocks whose maximum is every 8-bit (bf16) mantissa against elements on a fine grid: ties in plenty."""
    m = torch.arange(128, 256, dtype=torch.float64) / 128
    grid = torch.arange(1, 128, dtype=torch.float64) / 128
    x = torch.cat([m[:, None], m[:, None] * 0 + grid], 1).to(dtype)
    codes, _ = run_quant(x.cuda())
    want, _ = quantized(x, 1)
    assert torch.equal(codes, want)


@gpu
def test_quantize_edges():
    """Zero, tiny, subnormal and huge blocks, signed zeros, and non-finite elements that leave their block alone."""
    x = torch.zeros(10, 256)
    x[1, ::2] = -0.0
    x[2] = 2.0 ** -101
    x[3] = -2.0 ** -100
    x[4] = 3.0e38
    x[4, 1:] = -1.0
    x[5, 3] = 1e-40
    x[6] = data(1, 256, torch.float32, 1)[0]
    x[7] = x[6]
    x[6, 5], x[6, 130] = float("inf"), float("nan")
    x[8] = float("-inf")
    x[9] = float("nan")
    codes, scales = run_quant(x.cuda())
    ref, rs = run_quant(x[7:8].clone().index_fill(1, torch.tensor([5, 130]), 0.0).cuda())
    assert bool((scales[[0, 1, 2, 5, 8, 9]] == 0).all())
    assert bool(((codes[[0, 1, 2, 5]] & 0x7F) == 0).all()) and int(codes[1, 0]) == 0x80
    assert bool((codes[3] == 0xFE).all()) and bool((scales[3] == 2.0 ** -100 / 448).all())
    assert int(codes[4, 0]) == 0x7E and torch.isfinite(scales[4]).all()
    finite = [i for i in range(256) if i not in (5, 130)]
    assert torch.equal(codes[6, finite], ref[0, finite]) and torch.equal(scales[6], rs[0])
    assert (int(codes[6, 5]) & 0x7F) == 0x7F and (int(codes[6, 130]) & 0x7F) == 0x7F
    assert bool(((codes[8:] & 0x7F) == 0x7F).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,k,E,drop", [(1, 128, 1, 1, 0.0), (5, 1000, 3, 7, 0.3), (64, 5120, 6, 384, 0.0), (33, 77, 8, 8, 0.5), (100, 7168, 2, 4, 0.0)])
def test_permute_quantize(T, K, k, E, drop, dtype):
    """The same codes and scales as quantising and permuting in turn; unnamed rows keep what they held."""
    g = torch.Generator().manual_seed(T)
    R = T * k + 3
    inv = torch.randperm(R, generator=g)[:T * k].to(torch.int32)
    inv[torch.rand(T * k, generator=g) < drop] = -1
    inv = inv.view(T, k)
    x = data(T, K, dtype, 5).cuda()
    qc, qs = run_quant(x)
    codes = torch.full((R, K), 0x11, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, ceil_div(K, 128)), -2.0, device="cuda")
    want_c, want_s = codes.cpu(), scales.cpu()
    moe.moe_permute_quantize_fp8_block(x, inv.cuda(), codes, scales)
    for j in range(k):
        on = inv[:, j] >= 0
        want_c[inv[on, j].long()], want_s[inv[on, j].long()] = qc[on], qs[on]
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)


@gpu
def test_quantize_strided_rows():
    x = data(9, 300, torch.bfloat16, 3).cuda()
    ref = run_quant(x[:, 8:264].contiguous())
    for lo in (8, 1):
        v = torch.empty(9, 300, dtype=torch.bfloat16, device="cuda")[:, lo:lo + 256]
        v.copy_(x[:, 8:264])
        got = run_quant(v)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# ---------------------------------------------------------------- products

def make_weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (E, N, K), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.rand(E, ceil_div(N, 128), ceil_div(K, 128), generator=g) + 0.5
    return codes, scales


def make_rows(M, K, seed):
    w, s = make_weights(1, M, K, seed)
    g = torch.Generator().manual_seed(seed + 1)
    return w[0], torch.exp(torch.randn(M, ceil_div(K, 128), generator=g))


def weight_values(w, ws):
    return torch.stack([values(w[e], ws[e], 128) for e in range(w.shape[0])])


def offsets_of(counts):
    return torch.tensor([0] + torch.cumsum(torch.tensor(counts), 0).tolist(), dtype=torch.int64)


def workspace(M, N, K, E):
    return torch.empty(moe.moe_gemm_fp8_block_workspace_bytes(M, N, K, E), dtype=torch.uint8, device="cuda")


def product(x, xs, w, ws, offsets, out_dtype, dgrad=False, stream=None):
    E, N, K = w.shape
    M = x.shape[0]
    out = torch.full((M, K if dgrad else N), -77.0, dtype=out_dtype, device="cuda")
    space = workspace(M, N, K, E)
    call = moe.moe_gemm_fp8_block_dgrad if dgrad else moe.moe_gemm_fp8_block
    call(x, xs, w, ws, out, space, offsets=offsets, stream=stream)
    torch.cuda.synchronize()
    assert M == 0 or moe.moe_read_device_status(space) == 0
    return out


def check_product(M, N, K, counts, out_dtype, dgrad=False, seed=0):
    E = len(counts) if counts is not None else 1
    w, ws = make_weights(E, N, K, seed)
    red = N if dgrad else K
    x, xs = make_rows(M, red, seed + 10)
    off = None if counts is None else offsets_of(counts)
    out = product(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), None if off is None else off.cuda(), out_dtype, dgrad)
    X, W = values(x, xs, 1), weight_values(w, ws)
    spans = [(0, 0, M)] if counts is None else [(e, int(off[e]), int(off[e + 1])) for e in range(E)]
    covered = torch.zeros(M, dtype=torch.bool)
    got = out.double().cpu()
    for e, a, b in spans:
        covered[a:b] = True
        B = W[e] if dgrad else W[e].t()
        ref, size = X[a:b] @ B, X[a:b].abs() @ B.abs()
        bound = U[out_dtype] * ref.abs() + (ceil_div(red, 128) + 16) * 2.0 ** -22 * size + SMALLEST[out_dtype]
        lim = 65504.0 if out_dtype == torch.float16 else float("inf")
        fits = ref.abs() < lim * 0.99
        err = (got[a:b] - ref).abs()
        assert bool((err <= bound)[fits].all()), f"expert {e}: worst {float((err / bound)[fits].max()):.3g}"
    assert bool((got[~covered] == -77.0).all())


DENSE = [(1, 1, 16), (1, 2304, 5120), (2, 128, 128), (3, 130, 144), (5, 257, 1040), (8, 384, 2048), (9, 100, 4096),
         (16, 640, 128), (17, 1000, 272), (33, 256, 384), (64, 512, 512), (127, 127, 528), (128, 256, 256), (129, 259, 400),
         (200, 1152, 640), (256, 512, 1024), (300, 72, 2064), (515, 768, 896), (1025, 320, 256)]


@gpu
@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("out_dtype", DTYPES)
def test_dense_product(M, N, K, out_dtype):
    check_product(M, N, K, None, out_dtype, seed=M)


@gpu
@pytest.mark.parametrize("M,N,K", [(m, ceil_div(n, 16) * 16, k) for m, n, k in DENSE])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_dense_dgrad(M, N, K, out_dtype):
    check_product(M, N, K, None, out_dtype, dgrad=True, seed=M)


GROUPS = [[0, 0, 0, 5], [1] * 16, [3, 0, 1, 8, 9, 0, 17], [0, 128, 0, 129, 127, 1], [300, 0, 0, 0], [0, 0, 257, 31, 512, 2],
          [7] * 60 + [0] * 4, [64, 65, 63, 200, 33, 0, 96]]


@gpu
@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("N,K", [(384, 256), (200, 400)])
def test_grouped_product(counts, N, K):
    check_product(sum(counts), N, K, counts, torch.bfloat16, seed=len(counts))
    check_product(sum(counts) + 3, N, K, counts, torch.float32, seed=len(counts))  # rows past the last group


@gpu
@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("N,K", [(384, 256), (208, 400)])
def test_grouped_dgrad(counts, N, K):
    check_product(sum(counts), N, K, counts, torch.bfloat16, dgrad=True, seed=len(counts))
    check_product(sum(counts) + 3, N, K, counts, torch.float32, dgrad=True, seed=len(counts))


@gpu
@pytest.mark.parametrize("N,K,dgrad", [(328, 256, False), (329, 256, False), (264, 400, False), (272, 336, True)])
@pytest.mark.parametrize("out_dtype", DTYPES)
def test_many_rows(N, K, dgrad, out_dtype):
    """Full and ragged tiles of 256 rows side by side, columns past the last whole tile, rows on and off 16 bytes."""
    counts = [9000, 0, 15, 12345, 33]
    check_product(sum(counts) + 2, N, K, counts, out_dtype, dgrad=dgrad, seed=N)


@gpu
def test_no_rows():
    w, ws = make_weights(3, 64, 128, 0)
    for off in (torch.zeros(4, dtype=torch.int64), torch.tensor([0, 0, 4, 4])):
        M = int(off[-1])
        x, xs = make_rows(max(M, 1), 128, 1)
        product(x[:M].contiguous().cuda(), xs[:M].contiguous().cuda(), w.cuda(), ws.cuda(), off.cuda(), torch.float32)
    # every row outside the groups: nothing is written
    x, xs = make_rows(6, 128, 1)
    out = product(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), torch.zeros(4, dtype=torch.int64).cuda(), torch.float32)
    assert bool((out == -77.0).all())


@gpu
@pytest.mark.parametrize("M", [4, 200])
def test_offsets_out_of_range_are_clamped(M):
    """Offsets past M or negative read and write nothing outside the M rows."""
    w, ws = make_weights(3, 64, 128, 0)
    x, xs = make_rows(M, 128, 1)
    off = torch.tensor([-5, 2, M + 100, 2 ** 40], dtype=torch.int64).cuda()
    out = product(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), off, torch.float32).cpu()
    X, W = values(x, xs, 1), weight_values(w, ws)
    for e, a, b in ((0, 0, 2), (1, 2, M)):
        ref = X[a:b] @ W[e].t()
        size = X[a:b].abs() @ W[e].t().abs()
        assert bool(((out[a:b].double() - ref).abs() <= 17 * 2.0 ** -22 * size).all())


@gpu
@pytest.mark.parametrize("M", [3, 150])
@pytest.mark.parametrize("dgrad", [False, True])
def test_nan_and_inf_stay_in_their_row_and_column(M, dgrad):
    N, K = 160, 256
    w, ws = make_weights(1, N, K, 4)
    red, cols = (N, K) if dgrad else (K, N)
    x, xs = make_rows(M, red, 5)
    clean = product(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), None, torch.float32, dgrad).cpu()
    x2, xs2, w2 = x.clone(), xs.clone(), w.clone()
    x2[1, 3] = NAN_CODES[0]
    xs2[2, 0] = float("inf")
    w2[0, 7, 9] = NAN_CODES[1]
    out = product(x2.cuda(), xs2.cuda(), w2.cuda(), ws.cuda(), None, torch.float32, dgrad).cpu()
    bad_col = 9 if dgrad else 7
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[:, bad_col]).all())
    assert not bool(torch.isfinite(out[2]).any())
    keep_r = [r for r in range(M) if r not in (1, 2)]
    keep_c = [c for c in range(cols) if c != bad_col]
    assert torch.equal(out[keep_r][:, keep_c], clean[keep_r][:, keep_c])


@gpu
@pytest.mark.parametrize("M", [2, 40, 260])
def test_zero_scales_and_extreme_codes(M):
    """All-448 codes with scales of both extremes: sums stay exact integers times scales; zero-scale blocks give 0."""
    N, K = 130, 384
    x, w = torch.full((M, K), 0x7E, dtype=torch.uint8), torch.full((1, N, K), 0xFE, dtype=torch.uint8)
    xs, ws = torch.full((M, 3), 2.0 ** -60), torch.full((1, 2, 3), 2.0 ** 40)
    xs[:, 1] = 0.0
    out = product(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), None, torch.float32).cpu()
    assert bool((out == -(448.0 ** 2) * 256 * 2.0 ** -20).all())


@gpu
@pytest.mark.parametrize("M", [5, 300])
def test_dgrad_is_the_adjoint_and_matches_differences(M):
    """<dy, product(x)> = <dgrad(dy), x>, and a changed x moves the product by what dgrad says."""
    N, K = 272, 528
    w, ws = make_weights(1, N, K, 6)
    x, xs = make_rows(M, K, 7)
    dy, dys = make_rows(M, N, 8)
    x2, _ = make_rows(M, K, 9)
    g = [t.cuda() for t in (x, xs, x2, dy, dys, w, ws)]
    y = product(g[0], g[1], g[5], g[6], None, torch.float32).double().cpu()
    y2 = product(g[2], g[1], g[5], g[6], None, torch.float32).double().cpu()
    dx = product(g[3], g[4], g[5], g[6], None, torch.float32, dgrad=True).double().cpu()
    X, X2, D, W = values(x, xs, 1), values(x2, xs, 1), values(dy, dys, 1), weight_values(w, ws)[0]
    size = ((D.abs() @ W.abs()) * (X.abs() + X2.abs())).sum(1)
    bound = 40 * 2.0 ** -22 * size
    assert bool((((D * y).sum(1) - (dx * X).sum(1)).abs() <= bound).all())
    assert bool((((D * (y2 - y)).sum(1) - (dx * (X2 - X)).sum(1)).abs() <= bound).all())


@gpu
def test_streams_and_repeat_bits():
    for M, counts in ((24, [5, 0, 12, 7]), (700, [300, 100, 0, 300])):
        w, ws = make_weights(4, 384, 512, 1)
        x, xs = make_rows(M, 512, 2)
        g = [t.cuda() for t in (x, xs, w, ws, offsets_of(counts))]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        outs = [product(*g, torch.float32, stream=st) for st in (None, s, s)]
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@gpu
def test_product_in_a_graph():
    w, ws = make_weights(1, 256, 256, 1)
    x, xs = make_rows(40, 256, 2)
    g = [t.cuda() for t in (x, xs, w, ws)]
    out, space = torch.zeros(40, 256, device="cuda"), workspace(40, 256, 256, 1)
    want = product(*g, None, torch.float32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_gemm_fp8_block(*g, out, space)
    out.fill_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@gpu
def test_weights_past_4_gib():
    """Expert offsets past 2^32 bytes: the last expert of a 4.5 GiB weight tensor, few rows and many."""
    E, N, K = 144, 4096, 8192
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, N // 128, K // 128, device="cuda")
    last, _ = make_weights(1, N, K, 3)
    w[-1] = last[0].cuda()
    W = values(last[0][:256], torch.ones(2, K // 128), 128)
    for M in (3, 200):
        x, xs = make_rows(M, K, 4)
        off = torch.zeros(E + 1, dtype=torch.int64)
        off[-1] = M
        out = product(x.cuda(), xs.cuda(), w, ws, off.cuda(), torch.float32)[:, :256].double().cpu()
        X = values(x, xs, 1)
        ref, size = X @ W.t(), X.abs() @ W.t().abs()
        assert bool(((out - ref).abs() <= (64 + 16) * 2.0 ** -22 * size).all())


@gpu
@pytest.mark.parametrize("N", [32768, 32765])
def test_output_past_4_gib(N):
    """Output offsets past 2^32 bytes, aligned rows and not: the last rows of 70000."""
    M, K = 70000, 128
    w, ws = make_weights(1, N, K, 3)
    x, xs = make_rows(64, K, 4)
    full = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    scale = torch.ones(M, 1, device="cuda")
    full[-64:], scale[-64:] = x.cuda(), xs.cuda()
    out = product(full, scale, w.cuda(), ws.cuda(), None, torch.bfloat16)
    got = out[-64:].double().cpu()
    ref, size = values(x, xs, 1) @ weight_values(w, ws)[0].t(), values(x, xs, 1).abs() @ weight_values(w, ws)[0].t().abs()
    assert bool(((got - ref).abs() <= U[torch.bfloat16] * ref.abs() + 17 * 2.0 ** -22 * size).all())
    assert bool((out[:-64] == 0).all())


def test_refusals():
    u8, f32 = lambda *s: torch.zeros(*s, dtype=torch.uint8), torch.zeros  # noqa: E731
    ws = u8(256)
    ok = dict(x=u8(4, 128), xs=f32(4, 1), w=u8(2, 64, 128), s=f32(2, 1, 1), out=f32(4, 64), off=torch.zeros(3, dtype=torch.int64))

    def call(**kw):
        a = {**ok, **kw}
        moe.moe_gemm_fp8_block(a["x"], a["xs"], a["w"], a["s"], a["out"], ws, offsets=a["off"])

    bad = [
        lambda: call(x=u8(4, 144)), lambda: call(xs=f32(4, 2)), lambda: call(w=u8(64, 128)), lambda: call(s=f32(2, 2, 1)),
        lambda: call(out=f32(4, 65)), lambda: call(out=f32(4, 64).double()), lambda: call(off=torch.zeros(2, dtype=torch.int64)),
        lambda: call(off=torch.zeros(3, dtype=torch.int32)), lambda: call(),  # host tensors
        lambda: moe.moe_quantize_fp8_block(f32(4, 128), u8(4, 128), f32(4, 2)),
        lambda: moe.moe_quantize_fp8_block(f32(4, 128), u8(4, 128), f32(4, 1), block_rows=64),
        lambda: moe.moe_quantize_fp8_block(f32(4, 128).double(), u8(4, 128), f32(4, 1)),
        lambda: moe.moe_permute_quantize_fp8_block(f32(4, 128), torch.zeros(3, 2, dtype=torch.int32), u8(8, 128), f32(8, 1)),
    ]
    for f in bad:
        with pytest.raises(moe.MoeError) as ei:
            f()
        assert ei.value.status == 1


def test_c_refusals():
    L = moe.lib()
    p, n = 4096, 1 << 30

    def gemm(x=p, xs=p, w=p, s=p, off=p, M=4, N=64, K=128, E=2, out=p, dt=0, space=p, size=n, name="moe_gemm_fp8_block"):
        return getattr(L, name)(x, xs, w, s, off, M, N, K, E, out, dt, space, size, None)

    assert gemm(M=-1) == 1 and gemm(N=0) == 1 and gemm(E=0) == 1 and gemm(dt=3) == 1
    assert gemm(off=None) == 1                       # several experts need offsets
    assert gemm(K=120) == 2 and gemm(E=1025) == 2 and gemm(N=70000) == 2
    assert gemm(N=72, name="moe_gemm_fp8_block_dgrad") == 2
    assert gemm(x=None) == 1 and gemm(w=None) == 1 and gemm(space=None) == 1 and gemm(out=None) == 1
    assert gemm(x=p + 8) == 7 and gemm(w=p + 4) == 7 and gemm(out=p + 1) == 7 and gemm(space=p + 16) == 7
    assert gemm(size=8) == 4
    assert gemm(M=0, x=None, xs=None, out=None) == 0  # nothing to do
    assert moe.moe_gemm_fp8_block_workspace_bytes(4, 64, 128, 2) >= 32
    assert moe.moe_gemm_fp8_block_workspace_bytes(4, 0, 128, 2) == 0
    assert L.moe_quantize_fp8_block(p, 128, 0, 4, 128, 64, p, p, None) == 1
    assert L.moe_quantize_fp8_block(p, 127, 0, 4, 128, 1, p, p, None) == 1
    assert L.moe_quantize_fp8_block(p + 1, 128, 0, 4, 128, 1, p, p, None) == 7
    assert L.moe_quantize_fp8_block(None, 128, 0, 0, 128, 1, None, None, None) == 0
    assert L.moe_permute_quantize_fp8_block(p, 128, 0, p, 4, 128, 9, p, p, 8, None) == 2
    assert L.moe_permute_quantize_fp8_block(p, 128, 0, None, 4, 128, 2, p, p, 8, None) == 1
