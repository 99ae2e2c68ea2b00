"""Rows whose squares leave fp32's range: what the header says of them, and that they stay by themselves."""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_rms_norm import BF16, EPS, F32, gen, like, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [100, 128, 5120])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_squares_past_the_range(H, dtype):
    T = 40
    g = gen(H)
    x, w = rows(g, T, H, dtype), 1 + 0.1 * torch.randn(H, generator=g, device="cuda")

    def run(x, eps):
        out, rstd = like(x), torch.empty(T, device="cuda")
        codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
        moe.moe_rms_norm_quantize_fp8_block(x, w, eps, codes, scales, out=out, rstd=rstd)
        return out, rstd, codes, scales

    for eps in (EPS, 0.0):
        want = run(x, eps)
        y = x.clone()
        y[3] = 1e25   # squares of 1e50
        y[9] = 1e-30  # of 1e-60
        y[10] = 0
        out, rstd, codes, scales = run(y, eps)
        rest = [t for t in range(T) if t not in (3, 9, 10)]
        assert all(torch.equal(a[rest], b[rest]) for a, b in zip((out, rstd, codes, scales), want))
        assert float(rstd[3]) == 0 and bool((out[3] == 0).all()) and bool((scales[3] == 0).all())
        if eps == 0.0:
            assert bool((rstd[[9, 10]] == float("inf")).all()) and bool(torch.isnan(out[10]).all())
        else:
            assert bool(torch.isfinite(rstd).all()) and bool((out[10] == 0).all()) and bool((codes[10] == 0).all())
            assert bool((out[9].float() - 1e-30 * rstd[9] * w).abs().max() <= 2.0 ** -6 * 1e-27)
