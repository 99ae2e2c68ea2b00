"""16-bit rows of widths that leave them between two 16-byte boundaries: every shift, rows that end with the matrix,
neighbours that are NaN.  Bounds as in test_rms_norm.py."""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_rms_norm import BF16, EPS, F16, F32, HALF, SMALL, U, backward64, check_fp8, gen, like, near, norm64, rows

pytestmark = pytest.mark.gpu
WIDTHS = [2, 3, 5, 9, 57, 127, 130, 132, 843, 1002, 2052, 5181, 8197, 12290, 16370, 16377]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("wtype", [None, F32])
def test_norm_and_codes(H, dtype, wtype):
    for T in (2, 9, 400):
        g = gen(H + T)
        x, r = rows(g, T, H, dtype), rows(g, T, H, dtype)
        w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wtype or dtype)
        s, rs, y = norm64(x, r, w)
        out, total, rstd = like(x), like(x), torch.empty(T, device="cuda")
        moe.moe_rms_norm(x, w, EPS, out, residual=r, residual_out=total, rstd=rstd)
        near(out, y, 64 * U + HALF[dtype], SMALL[dtype])
        near(total, s, 2 * U + HALF[dtype], SMALL[dtype])
        near(rstd, rs, 64 * U)
        codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
        again = like(x)
        moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales, out=again, residual=r)
        check_fp8(codes, scales, y)
        near(again, y, 64 * U + HALF[dtype], SMALL[dtype])


@pytest.mark.parametrize("H", [57, 130, 843, 5181])
def test_neighbours_keep_their_bits(H):
    """Rows of NaN before and behind a row, in the same 16 bytes, change no bit of it, forward or backward."""
    T = 40
    g = gen(H)
    x, r, dy, w = rows(g, T, H, BF16), rows(g, T, H, BF16), rows(g, T, H, BF16), torch.rand(H, generator=g, device="cuda")
    rstd = torch.rand(T, generator=g, device="cuda")

    def run(x, dy):
        out, total, dx = like(x), like(x), like(x)
        codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
        moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales, out=out, residual=r, residual_out=total)
        moe.moe_rms_norm_backward(dy, x, w, rstd, dx, d_residual=r)
        return out, total, codes, scales, dx

    want = run(x, dy)
    bad = torch.arange(T, device="cuda") % 3 == 1
    x2, dy2 = x.clone(), dy.clone()
    x2[bad] = float("nan")
    dy2[bad] = float("inf")
    for a, b in zip(run(x2, dy2), want):
        assert torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("H,stride", [(100, 107), (843, 843), (1000, 1003), (57, 1000)])
def test_padding_stays(H, stride):
    """Columns behind a row's last are not written, whatever the shift."""
    T = 33
    g = gen(stride)
    x, r, dy = (rows(g, T, H, BF16, stride) for _ in range(3))
    w = torch.rand(H, generator=g, device="cuda").to(BF16)
    held = [torch.full((T, stride), -77.0, dtype=BF16, device="cuda") for _ in range(3)]
    out, total, dx = (t[:, :H] for t in held)
    moe.moe_rms_norm(x, w, EPS, out, residual=r, residual_out=total)
    rstd = norm64(x, None, w)[1].float()
    moe.moe_rms_norm_backward(dy, x, w, rstd, dx)
    near(out, norm64(x, r, w)[2], 64 * U + HALF[BF16])
    want, size, _, _ = backward64(dy, x, w, rstd, None)
    near(dx, want, HALF[BF16], 96 * U * size)
    for t in held:
        assert bool((t[:, H:] == -77.0).all())


@pytest.mark.parametrize("H", [2, 57, 132, 843, 3001, 7163, 8190])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients(H, dtype):
    for T, wtype in ((2, F32), (17, dtype), (1000, dtype)):
        g = gen(H + T)
        dy, x, dres = rows(g, T, H, dtype), rows(g, T, H, dtype), rows(g, T, H, dtype)
        whole = torch.rand(H + 1, generator=g, device="cuda").to(wtype)
        for w in (whole[:H].clone(), whole[1:]):  # on and off the 16-byte boundaries
            rstd = norm64(x, None, w)[1].float()
            dx, dw = like(x), torch.empty(H, device="cuda")
            space = torch.empty(moe.moe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
            moe.moe_rms_norm_backward(dy, x, w, rstd, dx, dw, space, d_residual=dres)
            want, size, dw64, size_dw = backward64(dy, x, w, rstd, dres)
            near(dx, want, HALF[dtype], 96 * U * size)
            near(dw, dw64, 0.0, (2 + T + 456 + 64) * U * size_dw + 1e-40)
