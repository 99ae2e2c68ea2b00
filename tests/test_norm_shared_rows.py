"""16-bit rows between two 16-byte boundaries whose norm leaves as FP8 codes: y passes through shared memory, up to the
width that a block's default limit of it holds beside the row's sums, and wider rows go element by element.  Both sides
of that width, and every shift.  Bounds as in test_rms_norm.py."""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_rms_norm import BF16, EPS, F16, F32, HALF, SMALL, U, check_fp8, gen, like, near, norm64, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,stride", [(12250, 12250), (12255, 12255), (12256, 12257), (12257, 12257), (12258, 12260),
                                      (12287, 12287), (12288, 12289), (12289, 12289)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("wtype", [None, F32])
def test_codes(H, stride, dtype, wtype):
    for T in (2, 9, 330):
        g = gen(H + T)
        x, r = rows(g, T, H, dtype, stride), rows(g, T, H, dtype, stride)
        w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wtype or dtype)
        s, _, y = norm64(x, r, w)
        out, total = like(x), like(x)
        codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
        moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales, out=out, residual=r, residual_out=total)
        check_fp8(codes, scales, y)
        near(out, y, 64 * U + HALF[dtype], SMALL[dtype])
        near(total, s, 2 * U + HALF[dtype], SMALL[dtype])
