"""The RMS norm (with residual, as values, FP8 block codes and MX codes) and its gradients against fp64.

u = 2^-24.  A thread sums at most 64 squares one after the other and the threads' sums meet in at most 10 + 1
additions; a square of the rounded sum is off by 3u.  The mean of positive terms is off by (64 + 11 + 3 + 2)u, its
root by half of that and one rounding more, y by the sum's rounding and two multiplications on top: below 48u; 64u
is used.  A stored value adds half a step of its type.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe

pytestmark = pytest.mark.gpu
BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}     # half a step, relative
SMALL = {BF16: 0.0, F16: 2.0 ** -25, F32: 0.0}                 # half of the smallest step
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, T, H, dtype, stride=None, shift=0):
    """T rows N(0, 1) in a matrix with that stride, starting `shift` elements into its memory."""
    stride = H if stride is None else stride
    flat = torch.zeros(shift + T * stride + 16, dtype=dtype, device="cuda")
    m = flat[shift:shift + T * stride].view(T, stride)[:, :H]
    m.copy_(torch.randn(T, H, generator=g, device="cuda") * torch.exp(torch.randn(H, generator=g, device="cuda")))
    return m


def like(m, fill=-77.0):
    stride = m.stride(0) if m.shape[0] > 1 else m.shape[1]
    return torch.full((m.shape[0], max(stride, m.shape[1])), fill, dtype=m.dtype, device="cuda")[:, :m.shape[1]]


def norm64(x, r, w, eps=EPS):
    s = x.to(F64) + (0 if r is None else r.to(F64))
    rstd = 1.0 / (s.square().mean(1) + eps).sqrt()
    return s, rstd, s * rstd[:, None] * w.to(F64)


def near(got, want, rel, more=0.0):
    err = (got.to(F64) - want).abs()
    bound = rel * want.abs() + more
    assert bool((err <= bound).all()), f"worst {float((err / bound.clamp_min(1e-300)).max()):.3g} of the bound"


def check_fp8(codes, scales, y):
    """Codes and 1x128 scales of fp64 rows y, with y off by 64u: the scale by 65u, the quotient by 130u more than
    the 2^-20 that a rounding to 20 bits costs, and the code by half a step."""
    T, H = y.shape
    pad = torch.nn.functional.pad(y, (0, -H % 128)).view(T, -1, 128)
    m = pad.abs().amax(2)
    near(scales, m / 448.0, 66 * U)
    q = (pad * 448.0 / m.clamp_min(1e-300)[..., None]).view(T, -1)[:, :H]
    code = codes.view(torch.float8_e4m3fn).to(F64)
    bound = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) + q.abs() * (2.0 ** -20 + 132 * U)
    assert bool(((code - q).abs() <= bound).all())


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def check_mx(fmt, codes, scales, y):
    """MX codes: the scale byte from the exponent of the block's maximum (either where the maximum is within 64u of a
    power of two), each code the nearest representable value, saturating."""
    T, H = y.shape
    b = y.view(T, -1, 32)
    amax = b.abs().amax(2)
    emax = 8 if fmt == moe.MOE_ACT_MXFP8 else 2
    lo = torch.frexp(amax * (1 - 64 * U)).exponent - 1 - emax + 127
    hi = torch.frexp(amax * (1 + 64 * U)).exponent - 1 - emax + 127
    byte = scales.to(torch.int64)
    assert bool(((byte == lo.clamp(0, 254)) | (byte == hi.clamp(0, 254))).all())
    v = b / torch.ldexp(torch.ones_like(amax), byte - 127)[..., None]
    if fmt == moe.MOE_ACT_MXFP8:
        top, code = 448.0, codes.view(torch.float8_e4m3fn).to(F64).view(v.shape)
        half = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))
    else:
        top = 6.0
        table = torch.tensor(E2M1 + [-e for e in E2M1], dtype=F64, device="cuda")
        nib = torch.stack([codes & 15, codes >> 4], 2).view(T, H).long()
        code = table[nib].view(v.shape)
        half = torch.where(v.abs() < 2, 0.25, torch.where(v.abs() < 4, 0.5, 1.0))
    v = v.clamp(-top, top)
    assert bool(((code - v).abs() <= half + v.abs() * 64 * U).all())


WIDTHS = [1, 7, 8, 32, 100, 128, 136, 256, 264, 1000, 2056, 5120, 7167, 8192, 8200, 16392, 20001, 32768]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(H, dtype, residual):
    for T, wtype in ((1, dtype), (5, F32), (337, dtype)):
        g = gen(H + T)
        x, r = rows(g, T, H, dtype), rows(g, T, H, dtype) if residual else None
        w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wtype)
        out, total = like(x), like(x) if residual else None
        rstd = torch.full((T,), -7.0, device="cuda")
        moe.moe_rms_norm(x, w, EPS, out, residual=r, residual_out=total, rstd=rstd)
        s, rs, y = norm64(x, r, w)
        near(out, y, 64 * U + HALF[dtype], SMALL[dtype])
        near(rstd, rs, 64 * U)
        if residual:
            near(total, s, 2 * U + HALF[dtype], SMALL[dtype])


@pytest.mark.parametrize("H", [32, 64, 96, 128, 160, 1024, 5120, 7168, 8224, 20000])
@pytest.mark.parametrize("kind", ["fp8", "mx8", "mx4"])
def test_quantised(H, kind):
    for T, dtype, keep, shift in ((1, BF16, True, 0), (67, F16, False, 0), (350, F32, True, 0), (19, BF16, True, 1)):
        g = gen(H + T)
        x, r = rows(g, T, H, dtype, H + 8, shift), rows(g, T, H, dtype)
        w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dtype)
        out, total = (like(x), like(r)) if keep else (None, None)
        _, _, y = norm64(x, r, w)
        if kind == "fp8":
            codes = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda")
            scales = torch.full((T, -(-H // 128)), -7.0, device="cuda")
            moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales, out=out, residual=r, residual_out=total)
            check_fp8(codes, scales, y)
        else:
            fmt = moe.MOE_ACT_MXFP8 if kind == "mx8" else moe.MOE_ACT_MXFP4
            codes = torch.full((T, H if kind == "mx8" else H // 2), 0x55, dtype=torch.uint8, device="cuda")
            scales = torch.full((T, H // 32), 0x55, dtype=torch.uint8, device="cuda")
            moe.moe_rms_norm_quantize_mx(x, w, EPS, fmt, codes, scales, out=out, residual=r, residual_out=total)
            check_mx(fmt, codes, scales, y)
        if keep:
            near(out, y, 64 * U + HALF[dtype], SMALL[dtype])


@pytest.mark.parametrize("H", [1, 7, 100, 129, 1000, 7167])
def test_fp8_codes_of_any_width(H):
    for T, dtype in ((1, F32), (66, BF16)):
        g = gen(H)
        x, w = rows(g, T, H, dtype), torch.ones(H, device="cuda")
        codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
        moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales)
        check_fp8(codes, scales, norm64(x, None, w)[2])


@pytest.mark.parametrize("H,stride,shift", [(128, 128, 1), (128, 136, 0), (128, 131, 0), (1024, 1031, 3), (5120, 5128, 8)])
def test_strides_and_alignment(H, stride, shift):
    T = 41
    for dtype in (BF16, F32):
        g = gen(stride)
        x, r = rows(g, T, H, dtype, stride, shift), rows(g, T, H, dtype, stride + 1)
        w = torch.randn(H + 1, generator=g, device="cuda")[1:].contiguous()
        hold = torch.full((T, stride + 5), -77.0, dtype=dtype, device="cuda")
        out = hold[:, 3:3 + H]
        moe.moe_rms_norm(x, w, EPS, out, residual=r)
        near(out, norm64(x, r, w)[2], 64 * U + HALF[dtype], SMALL[dtype])
        assert bool((hold[:, :3] == -77.0).all()) and bool((hold[:, 3 + H:] == -77.0).all())


def test_outputs_over_their_inputs():
    """residual_out over residual, out over x; the same bits as apart."""
    for T, H in ((1, 7168), (301, 5120), (23, 100)):
        g = gen(T)
        x, r, w = rows(g, T, H, BF16), rows(g, T, H, BF16), torch.rand(H, generator=g, device="cuda").to(BF16)
        out, total = like(x), like(x)
        moe.moe_rms_norm(x, w, EPS, out, residual=r, residual_out=total)
        moe.moe_rms_norm(x, w, EPS, x, residual=r, residual_out=r)
        assert torch.equal(x, out) and torch.equal(r, total)


@pytest.mark.parametrize("H", [96, 100, 5120])
def test_rows_that_have_no_norm_stay_apart(H):
    """A row of zeros gives zeros, NaN and infinities stay in their row; every other row keeps its bits."""
    T = 70
    g = gen(3)
    x, w = rows(g, T, H, BF16), torch.rand(H, generator=g, device="cuda")
    want, codes0, scales0 = like(x), torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
    moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes0, scales0, out=want)
    y = x.clone()
    y[7] = 0
    y[8, 5] = float("nan")
    y[20, H - 1] = float("inf")
    got, codes, scales = like(x), torch.empty_like(codes0), torch.empty_like(scales0)
    moe.moe_rms_norm_quantize_fp8_block(y, w, EPS, codes, scales, out=got)
    rest = [t for t in range(T) if t not in (7, 8, 20)]
    assert torch.equal(got[rest], want[rest]) and torch.equal(codes[rest], codes0[rest]) and torch.equal(scales[rest], scales0[rest])
    assert bool((got[7] == 0).all()) and bool((scales[7] == 0).all()) and bool((codes[7] == 0).all())
    assert bool(torch.isnan(got[8]).all()) and bool(((codes[8] & 127) == 127).all())
    assert bool(torch.isnan(got[20, H - 1])) and bool((got[20, :H - 1] == 0).all())


def test_layer_takes_the_codes():
    """norm -> MX codes -> the prequantised layer gives what the layer gives for codes of moe_quantize_mx's rule."""
    import synth
    T, H, I, E, k = 33, 256, 128, 8, 2
    g = gen(5)
    x, r, w = rows(g, T, H, BF16), rows(g, T, H, BF16), torch.rand(H, generator=g, device="cuda").to(BF16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    w1, s1, w2, s2 = synth.weights_codes(E, H, I, 0, device="cuda")
    codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    rounded = like(x)
    moe.moe_rms_norm_quantize_mx(x, w, EPS, moe.MOE_ACT_MXFP8, codes, scales, out=rounded, residual=r)
    space = torch.empty(moe.moe_workspace_bytes(T, H, I, E, k), dtype=torch.uint8, device="cuda")
    out, plain = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, H, dtype=BF16, device="cuda")
    moe.moe_a8w4_forward_prequant(codes, scales, logits, w1, s1, w2, s2, out, E, k, space)
    moe.moe_a8w4_forward(rounded, logits, w1, s1, w2, s2, plain, E, k, space)
    # the second one rounds the rows to bf16 before it quantises them: 2^-8 against a code's 2^-4
    rel = float((out.double() - plain.double()).norm() / plain.double().norm())
    assert 0 < rel < 2.0 ** -4


def backward64(dy, x, w, rstd, dres):
    xh, g = x.to(F64) * rstd.to(F64)[:, None], dy.to(F64) * w.to(F64)
    R = rstd.to(F64)[:, None]
    dx = R * (g - xh * (g * xh).mean(1, keepdim=True))
    size = R * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dx, size = dx + dres.to(F64), size + dres.to(F64).abs()
    return dx, size, (dy.to(F64) * xh).sum(0), (dy.to(F64) * xh).abs().sum(0)


def run_backward(T, H, dtype, wtype, residual, stride=None, shift=0, need_dw=True):
    g = gen(H + T)
    dy, x = rows(g, T, H, dtype, stride, shift), rows(g, T, H, dtype, stride)
    dres = rows(g, T, H, dtype) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wtype)
    rstd = norm64(x, None, w)[1].float()
    dx = like(x)
    dw = torch.full((H,), -7.0, device="cuda") if need_dw else None
    space = torch.full((moe.moe_rms_norm_backward_workspace_bytes(T, H),), 0x7f, dtype=torch.uint8, device="cuda")
    args = (dy, x, w, rstd, dx, dw, space if need_dw else None)
    moe.moe_rms_norm_backward(*args, d_residual=dres)
    want, size, want_dw, size_dw = backward64(dy, x, w, rstd, dres)
    # a term of the row's sum: three roundings; 64 + 11 additions; four operations after it
    near(dx, want, HALF[dtype], 96 * U * size + SMALL[dtype])
    if need_dw:
        # a term: two roundings; each row is one addition at most, in whatever order, and so is each block's sum
        near(dw, want_dw, 0.0, (2 + T + 456 + 64) * U * size_dw + 1e-40)
    return args, dres


@pytest.mark.parametrize("H", [1, 7, 8, 16, 100, 128, 256, 264, 1000, 2056, 5120, 7167, 7168, 8200, 16384, 20001, 32768])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_gradients(H, dtype, residual):
    for T, wtype in ((1, dtype), (3, F32), (700, dtype)):
        run_backward(T, H, dtype, wtype, residual)


@pytest.mark.parametrize("T", [2, 7, 8, 9, 303, 304, 305, 609, 1300])
def test_gradients_over_rounds(T):
    for H in (64, 2048, 7168, 57, 1002, 2052, 7163):
        run_backward(T, H, BF16, BF16, True)


@pytest.mark.parametrize("H,stride,shift", [(128, 128, 1), (128, 136, 0), (1024, 1031, 3), (5120, 5128, 8), (20000, 20001, 0)])
def test_gradients_of_strided_rows(H, stride, shift):
    for dtype in (BF16, F32):
        run_backward(77, H, dtype, dtype, True, stride, shift)
        run_backward(77, H, dtype, dtype, False, stride, shift, need_dw=False)


def test_gradients_over_their_inputs_and_again():
    """dx over dy, x or d_residual gives the same bits as apart, and a second call the same dw."""
    for H in (7168, 100, 20000):
        (dy, x, w, rstd, dx, dw, space), dres = run_backward(333, H, BF16, BF16, True)
        for name in ("dy", "x", "dres"):
            t = {"dy": dy.clone(), "x": x.clone(), "dres": dres.clone()}
            dw2 = torch.empty_like(dw)
            moe.moe_rms_norm_backward(t["dy"], t["x"], w, rstd, t[name], dw2, space, d_residual=t["dres"])
            assert torch.equal(t[name], dx) and torch.equal(dw2, dw)


def test_gradient_by_differences():
    """fp32 rows, small enough to difference the fp64 norm: <dx, d> is the change of <dy, norm> along d."""
    T, H, h = 9, 48, 1e-5
    g = gen(1)
    (dy, x, w, rstd, dx, dw, _), _ = run_backward(T, H, F32, F32, False)
    d = torch.randn(T, H, generator=g, device="cuda", dtype=F64)
    e = torch.randn(H, generator=g, device="cuda", dtype=F64)
    f = lambda X, W: float((norm64(X, None, W)[2] * dy.to(F64)).sum())  # noqa: E731
    X, W = x.to(F64), w.to(F64)
    along_x = (f(X + h * d, W) - f(X - h * d, W)) / (2 * h)
    along_w = (f(X, W + h * e) - f(X, W - h * e)) / (2 * h)
    # central differences: h^2 of third derivatives (below 1e3 of the values here); products in fp32
    size = float((dx.to(F64) * d).abs().sum() + (dw.to(F64) * e).abs().sum())
    assert abs(float((dx.to(F64) * d).sum()) - along_x) <= 1e-5 * size
    assert abs(float((dw.to(F64) * e).sum()) - along_w) <= 1e-5 * size


def test_no_rows():
    w, x = torch.ones(64, device="cuda"), torch.empty(0, 64, device="cuda")
    moe.moe_rms_norm(x, w, EPS, torch.empty_like(x))
    dw = torch.full((64,), 3.0, device="cuda")
    space = torch.empty(moe.moe_rms_norm_backward_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    moe.moe_rms_norm_backward(x, x, w, torch.empty(0, device="cuda"), torch.empty_like(x), dw, space)
    assert bool((dw == 0).all())


def test_graph_and_stream():
    """Captured once and replayed on new values; on a stream of its own."""
    T, H = 130, 5120
    g = gen(9)
    x, r, w = rows(g, T, H, BF16), rows(g, T, H, BF16), torch.rand(H, generator=g, device="cuda").to(BF16)
    out, total, rstd, dx = like(x), like(x), torch.empty(T, device="cuda"), like(x)
    codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda")
    dw = torch.empty(H, device="cuda")
    space = torch.empty(moe.moe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales, out=out, residual=r, residual_out=total,
                                            rstd=rstd, stream=stream)
        moe.moe_rms_norm_backward(out, total, w, rstd, dx, dw, space, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(rows(g, T, H, BF16))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, total, rstd, codes, scales, dx, dw)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, total, rstd, codes, scales, dx, dw)))


def test_many_rows_of_short_heads():
    """Offsets past 2^31 elements: the last rows of 17 M heads of 128."""
    T, H = (1 << 31) // 128 + 1000, 128
    x = torch.empty(T, H, dtype=BF16, device="cuda")
    x[:1000].normal_(generator=gen(1))
    x[1000:-1000] = 1
    x[-1000:].normal_(generator=gen(2))
    out, w = torch.empty_like(x), torch.ones(H, device="cuda", dtype=BF16)
    moe.moe_rms_norm(x, w, EPS, out)
    near(out[-1000:], norm64(x[-1000:], None, w)[2], 64 * U + HALF[BF16])
    near(out[:1000], norm64(x[:1000], None, w)[2], 64 * U + HALF[BF16])
