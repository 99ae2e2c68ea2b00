"""Token rows to expert rows and back, their gradients and the router's gradient, against fp64.

Tolerances: u is the unit roundoff of the output type (2^-8 bf16, 2^-11 f16, 2^-24 f32).  A sum of n
fp32 terms rounded once is within u |ref| + n 2^-24 sum |terms| of the exact one; the dot products of
the unpermute gradient add at most 64 terms in a row (32 in a thread, then 5 + 8 over threads).
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe

gpu = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (T, H, k, E): one token, odd widths, rows shorter and longer than a block's threads cover
SIZES = [(1, 1, 1, 1), (1, 7168, 6, 384), (3, 64, 2, 8), (17, 121, 3, 16), (64, 1887, 8, 64), (33, 5120, 3, 128),
         (130, 514, 4, 5), (257, 2056, 1, 3), (5, 65536, 2, 4)]


def mapping(T, k, E, seed, drop=0.0, extra=0):
    """inv [T, k] of a stable sort of random distinct ids by expert, dropped pairs -1; R rows of which `extra` unnamed."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    key = torch.where(torch.rand(T * k, generator=g) < drop, E, ids.reshape(-1))
    order = torch.argsort(key, stable=True)
    inv = torch.empty(T * k, dtype=torch.int32)
    inv[order] = torch.arange(T * k, dtype=torch.int32)
    inv[key == E] = -1
    return ids, inv.view(T, k), int((key < E).sum()) + extra


def rows_like(*shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def close(got, want, bound):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound).all()), f"max error over bound {float((err / bound).max()):.3g}"


@gpu
@pytest.mark.parametrize("dtype", DTYPES + [torch.uint8])
@pytest.mark.parametrize("T,H,k,E", SIZES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_permute_copies_kept_pairs_and_nothing_else(T, H, k, E, dtype, drop):
    _, inv, R = mapping(T, k, E, 1, drop, extra=2)
    x = (torch.randint(0, 256, (T, H), dtype=torch.uint8) if dtype == torch.uint8 else rows_like(T, H, dtype=dtype, seed=2))
    rows = torch.full((R, H), 7, dtype=dtype)
    want = rows.clone()
    on = inv >= 0
    want[inv[on].long()] = x[:, None].expand(T, k, H)[on]
    d = rows.cuda()
    moe.moe_permute(x.cuda(), inv.cuda(), d)
    assert torch.equal(d.cpu(), want)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,k,E", SIZES)
@pytest.mark.parametrize("drop", [0.0, 0.6])
def test_unpermute_and_gradients(T, H, k, E, dtype, drop):
    _, inv, R = mapping(T, k, E, 3, drop, extra=1)
    rows, dout = rows_like(R, H, dtype=dtype, seed=4), rows_like(T, H, dtype=dtype, seed=5)
    w = torch.softmax(rows_like(T, k, dtype=torch.float32, seed=6), 1)
    on = (inv >= 0)[..., None]
    full = torch.where(on, rows.double()[inv.clamp(min=0).long()], 0.0)  # [T, k, H]
    rows_g, inv_g, w_g, dout_g = rows.cuda(), inv.cuda(), w.cuda(), dout.cuda()
    out = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
    moe.moe_unpermute(rows_g, inv_g, w_g, out)
    terms = full * w.double()[..., None]
    close(out, terms.sum(1), U[dtype] * terms.sum(1).abs() + k * 2.0 ** -24 * terms.abs().sum(1) + SMALLEST[dtype])
    moe.moe_permute_backward(rows_g, inv_g, out)
    close(out, full.sum(1), U[dtype] * full.sum(1).abs() + k * 2.0 ** -24 * full.abs().sum(1) + SMALLEST[dtype])
    # gradients: unnamed rows keep what they held
    drows = torch.full((R, H), 3.0, dtype=dtype, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_unpermute_backward(dout_g, rows_g, inv_g, w_g, drows, dw)
    want = torch.full((R, H), 3.0, dtype=torch.float64)
    want[inv[inv >= 0].long()] = (w.double()[..., None] * dout.double()[:, None])[inv >= 0]
    close(drows, want, 2 * U[dtype] * want.abs() + SMALLEST[dtype])
    prod = full * dout.double()[:, None]
    close(dw, prod.sum(2), 64 * 2.0 ** -24 * prod.abs().sum(2))
    assert bool((dw.cpu()[inv < 0] == 0).all())
    # each result alone, the same bits
    drows2, dw2 = torch.full_like(drows, 3.0), torch.empty_like(dw)
    moe.moe_unpermute_backward(dout_g, None, inv_g, w_g, drows2, None)
    moe.moe_unpermute_backward(dout_g, rows_g, inv_g, w_g, None, dw2)
    assert torch.equal(drows, drows2) and torch.equal(dw, dw2)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_alignment(dtype):
    """Row strides larger than the row and bases off the 16-byte grid give the same bits."""
    T, H, k, E = 19, 256, 3, 8
    _, inv, R = mapping(T, k, E, 7)
    x, rows = rows_like(T, H, dtype=dtype, seed=8).cuda(), rows_like(R, H, dtype=dtype, seed=9).cuda()
    w, inv = torch.softmax(rows_like(T, k, dtype=torch.float32, seed=10), 1).cuda(), inv.cuda()

    def shifted(t, by, pad):
        big = torch.zeros(t.shape[0], t.shape[1] + by + pad, dtype=t.dtype, device="cuda")
        v = big[:, by:by + t.shape[1]]
        v.copy_(t)
        return v

    ref = [torch.empty_like(rows), torch.empty_like(x), torch.empty_like(rows)]
    dw = torch.empty(T, k, device="cuda")
    moe.moe_permute(x, inv, ref[0])
    moe.moe_unpermute(rows, inv, w, ref[1])
    moe.moe_unpermute_backward(x, rows, inv, w, ref[2], dw)
    for by, pad in [(0, 8), (8, 0), (4, 4), (2, 2), (1, 2)]:
        got = [shifted(torch.zeros_like(t), by, pad) for t in ref]
        xs, rs, dw2 = shifted(x, by, pad), shifted(rows, by, pad), torch.empty_like(dw)
        moe.moe_permute(xs, inv, got[0])
        moe.moe_unpermute(rs, inv, w, got[1])
        moe.moe_unpermute_backward(xs, rs, inv, w, got[2], dw2)
        for a, b in zip(got, ref):
            assert torch.equal(a, b), (by, pad)
        assert torch.allclose(dw2, dw, rtol=0, atol=64 * 2.0 ** -24 * float((x.abs().max() * rows.abs().max()) * H))


@gpu
def test_dropped_rows_are_never_read():
    """NaN and infinities in rows that no pair names, and tokens without a kept pair."""
    T, H, k = 6, 128, 2
    inv = torch.tensor([[0, 1], [-1, 2], [-1, -1], [9, -5], [4, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    rows = torch.ones(9, H)
    rows[5:] = float("nan")
    w = torch.full((T, k), 0.5)
    w[2:4] = float("inf")
    out = torch.empty(T, H, device="cuda")
    moe.moe_unpermute(rows.cuda(), inv.cuda(), w.cuda(), out)
    assert torch.equal(out[:, 0].cpu(), torch.tensor([1.0, 0.5, 0.0, 0.0, 1.0, 0.0]))
    moe.moe_permute_backward(rows.cuda(), inv.cuda(), out)
    assert torch.equal(out[:, 0].cpu(), torch.tensor([2.0, 1.0, 0.0, 0.0, 2.0, 0.0]))
    none = torch.empty(0, H, device="cuda")
    moe.moe_unpermute(none, inv.cuda(), w.cuda(), out)
    assert bool((out == 0).all())
    moe.moe_permute(out, inv.cuda(), none)


@gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 384, 6), (7, 5, 5), (64, 128, 3), (33, 1024, 8), (9, 131, 2), (1000, 384, 6)])
def test_route_backward(T, E, k):
    g = torch.Generator().manual_seed(T + E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    dw = torch.randn(T, k, generator=g)
    out = torch.full((T, E), float("nan"), device="cuda")
    moe.moe_topk_route_backward(ids.cuda(), w.cuda(), dw.cuda(), out)
    W, D = w.double(), dw.double()
    grad = W * (D - (W * D).sum(1, keepdim=True))
    want = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids.long(), grad)
    size = W * (D.abs() + (W * D).abs().sum(1, keepdim=True))
    bound = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids.long(), (k + 3) * 2.0 ** -24 * size)
    err = (out.double().cpu() - want).abs()
    assert bool((err <= bound).all())


@gpu
def test_route_backward_against_differences():
    """d loss / d logits of loss = sum dw * w by central differences of moe_topk_route's own weights.
    h = 2^-7: truncation under h^2 |dw|, rounding k 2^-23 |dw| / 2h = 2^-14, both below 2e-4 of |dw| <= 1."""
    T, E, k, h = 16, 24, 4, 2.0 ** -7
    g = torch.Generator().manual_seed(0)
    # well separated logits: no step changes the selection
    lg = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.25
    dw = torch.rand(T, k, generator=g) * 2 - 1

    def route(x):
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        moe.moe_topk_route(x.cuda(), k, ids, w)
        return ids, w

    ids, w = route(lg)
    got = torch.empty(T, E, device="cuda")
    moe.moe_topk_route_backward(ids, w, dw.cuda(), got)
    loss = lambda x: (route(x)[1].double().cpu() * dw.double()).sum(1)  # noqa: E731
    for j in range(k):
        step = torch.zeros(T, E).scatter_(1, ids.cpu().long()[:, j:j + 1], h)
        diff = (loss(lg + step) - loss(lg - step)) / (2 * h)
        have = got.double().cpu().gather(1, ids.cpu().long()[:, j:j + 1])[:, 0]
        assert float((have - diff).abs().max()) <= 2e-4


@gpu
def test_row_gradients_against_differences():
    """<dout, unpermute(rows)> is linear in rows and in w: differences of the forward with steps that are
    powers of two equal the gradients up to fp32 rounding of the forward (H k 2^-23 of its terms)."""
    T, H, k, E = 9, 96, 3, 8
    _, inv, R = mapping(T, k, E, 11, 0.2)
    rows, dout = rows_like(R, H, dtype=torch.float32, seed=12), rows_like(T, H, dtype=torch.float32, seed=13)
    w = torch.softmax(rows_like(T, k, dtype=torch.float32, seed=14), 1)
    step_r, step_w = rows_like(R, H, dtype=torch.float32, seed=15), rows_like(T, k, dtype=torch.float32, seed=16)
    inv_g = inv.cuda()

    def loss(r, wt):
        out = torch.empty(T, H, device="cuda")
        moe.moe_unpermute(r.cuda(), inv_g, wt.cuda(), out)
        return float((out.double().cpu() * dout.double()).sum())

    drows, dw = torch.zeros(R, H, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_unpermute_backward(dout.cuda(), rows.cuda(), inv_g, w.cuda(), drows, dw)
    tol = T * H * k * 2.0 ** -23 * float(rows.abs().max() * dout.abs().max()) * 4
    diff_r = (loss(rows + step_r, w) - loss(rows - step_r, w)) / 2
    assert abs(diff_r - float((drows.double().cpu() * step_r.double()).sum())) <= tol
    diff_w = (loss(rows, w + step_w) - loss(rows, w - step_w)) / 2
    assert abs(diff_w - float((dw.double().cpu() * step_w.double()).sum())) <= tol
    # permute: <drows, permute(x)> differences against permute_backward
    x, dx = rows_like(T, H, dtype=torch.float32, seed=17), torch.empty(T, H, device="cuda")
    moe.moe_permute_backward(rows.cuda(), inv_g, dx)
    moved = torch.zeros(R, H, device="cuda")
    moe.moe_permute(x.cuda(), inv_g, moved)
    assert abs(float((moved.double().cpu() * rows.double()).sum()) - float((dx.double().cpu() * x.double()).sum())) <= tol


@gpu
@pytest.mark.parametrize("H", [32768, 32767])
def test_rows_past_4_gib(H):
    """Row offsets past 2^32 bytes: the last rows of an 8.6 GiB matrix."""
    R = 70000
    rows = torch.empty(R, H, dtype=torch.float32, device="cuda")
    inv = torch.tensor([[R - 1, 0], [R - 2, 1]], dtype=torch.int32, device="cuda")
    x = rows_like(2, H, dtype=torch.float32, seed=22).cuda()
    w = torch.tensor([[0.5, 0.25], [1.0, -1.0]], device="cuda")
    moe.moe_permute(x, inv, rows)
    assert torch.equal(rows[-1], x[0]) and torch.equal(rows[-2], x[1]) and torch.equal(rows[0], x[0])
    out = torch.empty_like(x)
    moe.moe_unpermute(rows, inv, w, out)
    assert torch.equal(out[0], 0.75 * x[0]) and bool((out[1] == 0).all())
    dw = torch.empty(2, 2, device="cuda")
    moe.moe_unpermute_backward(out, rows, inv, w, rows, dw)
    assert torch.equal(rows[-1], 0.5 * out[0]) and bool((rows[-2] == 0).all())


@gpu
def test_odd_strides():
    """Rows that overlap (an expanded matrix) are refused; one column, or one row, may have any stride there."""
    inv = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    w, rows, x = torch.ones(4, 2, device="cuda"), torch.zeros(8, 64, device="cuda"), torch.ones(4, 64, device="cuda")
    same, wide = torch.ones(1, 64, device="cuda").expand(4, 64), torch.ones(1, 64, device="cuda").expand(8, 64)
    codes, scales = torch.zeros(8, 64, dtype=torch.uint8, device="cuda"), torch.zeros(8, 1, device="cuda")
    for call in (lambda: moe.moe_permute(same, inv, rows), lambda: moe.moe_unpermute(wide, inv, w, x),
                 lambda: moe.moe_permute_backward(wide, inv, x), lambda: moe.moe_unpermute_backward(same, rows, inv, w, rows, w),
                 lambda: moe.moe_unpermute_backward(x, wide, inv, w, None, w), lambda: moe.moe_quantize_fp8_block(wide, codes, scales),
                 lambda: moe.moe_permute_quantize_fp8_block(same, inv, codes, scales)):
        with pytest.raises(moe.MoeError) as ei:
            call()
        assert ei.value.status == 1
    col = torch.arange(16.0, device="cuda").view(4, 4)[:, 1:2]
    got = torch.zeros(8, 1, device="cuda")
    moe.moe_permute(col, inv, got)
    assert got[:, 0].tolist() == [1, 1, 5, 5, 9, 9, 13, 13]
    one = torch.arange(64.0, device="cuda").view(1, 64).as_strided((1, 64), (1, 1))
    moe.moe_permute(one, inv[:1], rows)
    assert torch.equal(rows[1], one[0]) and bool((rows[2:] == 0).all())


@gpu
def test_other_stream_and_repeat_bits():
    T, H, k, E = 200, 1024, 6, 64
    _, inv, R = mapping(T, k, E, 18)
    rows, dout = rows_like(R, H, dtype=torch.bfloat16, seed=19).cuda(), rows_like(T, H, dtype=torch.bfloat16, seed=20).cuda()
    w, inv = torch.softmax(rows_like(T, k, dtype=torch.float32, seed=21), 1).cuda(), inv.cuda()
    res = []
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s, s):
        d, dw, out = torch.empty_like(rows), torch.empty(T, k, device="cuda"), torch.empty_like(dout)
        torch.cuda.synchronize()
        moe.moe_unpermute_backward(dout, rows, inv, w, d, dw, stream=stream)
        moe.moe_unpermute(rows, inv, w, out, stream=stream)
        torch.cuda.synchronize()
        res.append((d, dw, out))
    for other in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], other))


def test_refusals():
    """Bad arguments raise before anything runs (no GPU needed)."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x, rows, w = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4, 2)
    bad = [
        lambda: moe.moe_permute(x, i32(4, 2).long(), rows),
        lambda: moe.moe_permute(x, i32(3, 2), rows),
        lambda: moe.moe_permute(x, i32(4, 2), rows.half()),
        lambda: moe.moe_permute(x.t(), i32(64, 2), rows),
        lambda: moe.moe_permute(x.double(), i32(4, 2), rows.double()),
        lambda: moe.moe_permute(x, i32(4, 2), torch.zeros(8, 65)),
        lambda: moe.moe_permute(x, i32(4, 2), rows),  # host tensors
        lambda: moe.moe_unpermute(rows, i32(4, 2), w.double(), x),
        lambda: moe.moe_unpermute(rows, i32(4, 2), None, x),
        lambda: moe.moe_unpermute_backward(x, None, i32(4, 2), w, rows, w),
        lambda: moe.moe_unpermute_backward(x, rows, i32(4, 2), w, torch.zeros(9, 64), w),
        lambda: moe.moe_topk_route_backward(i32(4, 2), w, torch.zeros(4, 3), torch.zeros(4, 8)),
    ]
    for call in bad:
        with pytest.raises(moe.MoeError) as ei:
            call()
        assert ei.value.status == 1


def test_c_refusals():
    L = moe.lib()
    p = 4096  # never dereferenced: every call is refused, or has nothing to do
    assert L.moe_permute(p, 64, 0, p, -1, 64, 2, p, 64, 8, None) == 1
    assert L.moe_permute(p, 63, 0, p, 4, 64, 2, p, 64, 8, None) == 1       # stride < H
    assert L.moe_permute(p, 64, 4, p, 4, 64, 2, p, 64, 8, None) == 1       # unknown type
    assert L.moe_permute(p, 64, 0, p, 4, 64, 9, p, 64, 8, None) == 2       # k > 8
    assert L.moe_permute(p, 70000, 0, p, 4, 70000, 2, p, 70000, 8, None) == 2
    assert L.moe_permute(p + 1, 64, 0, p, 4, 64, 2, p, 64, 8, None) == 7
    assert L.moe_permute(None, 64, 0, p, 4, 64, 2, p, 64, 8, None) == 1
    assert L.moe_permute(None, 64, 0, None, 0, 64, 2, None, 64, 0, None) == 0
    assert L.moe_unpermute(p, 64, 8, 3, p, p, 4, 64, 2, p, 64, None) == 1  # bytes have no sum
    assert L.moe_unpermute(p, 64, 8, 0, p, None, 4, 64, 2, p, 64, None) == 1
    assert L.moe_permute_backward(p, 64, 8, 0, p, 4, 64, 2, p + 1, 64, None) == 7
    assert L.moe_unpermute_backward(p, 64, None, 64, 8, 0, p, p, 4, 64, 2, p, 64, p, None) == 1
    assert L.moe_unpermute_backward(p, 64, None, 64, 8, 0, p, p, 4, 64, 2, None, 64, None, None) == 0
    assert L.moe_topk_route_backward(p, p, p, 4, 2, 3, p, None) == 1       # k > E
    assert L.moe_topk_route_backward(p, p, p, 4, 2048, 3, p, None) == 2
    assert L.moe_topk_route_backward(p, p, None, 4, 8, 3, p, None) == 1
    assert L.moe_topk_route_backward(p, p, p + 2, 4, 8, 3, p, None) == 7
