"""The ring of the norm's gradients where threads own pieces of 16 bytes that lie wholly behind the row's end, at every
shift of a row from the 16-byte boundaries: nothing is read there (the elements behind a row are NaN), and nothing
written.  Bounds as in test_rms_norm.py."""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_rms_norm import BF16, F16, F32, HALF, U, backward64, gen, near, norm64

pytestmark = pytest.mark.gpu


def held(g, T, H, stride, dtype):
    """Rows in a matrix whose elements between the rows, and behind the last, are NaN."""
    flat = torch.full((T * stride + 64,), float("nan"), dtype=dtype, device="cuda")
    m = flat[:T * stride].view(T, stride)
    m[:, :H].copy_(torch.randn(T, H, generator=g, device="cuda"))
    return m[:, :H]


# threads of a row: 4, 8, 16 and whole warps, of which the last pieces are past it
@pytest.mark.parametrize("H", [33, 41, 97, 130, 201, 258, 515, 1030, 5185])
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_pieces_behind_the_row(H, pad, dtype):
    stride = H + pad
    for T in (1, 5, 64, 700):
        g = gen(stride + T)
        dy, x, dres = (held(g, T, H, stride, dtype) for _ in range(3))
        w = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
        rstd = norm64(x, None, w)[1].float()
        whole = torch.full((T, stride), -77.0, dtype=dtype, device="cuda")
        dx, dw = whole[:, :H], torch.empty(H, device="cuda")
        space = torch.empty(moe.moe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        for residual in (dres, None):
            moe.moe_rms_norm_backward(dy, x, w, rstd, dx, dw, space, d_residual=residual)
            want, size, dw64, size_dw = backward64(dy, x, w, rstd, residual)
            near(dx, want, HALF[dtype], 96 * U * size + (2.0 ** -25 if dtype == F16 else 0.0))
            near(dw, dw64, 0.0, (2 + T + 456 + 64) * U * size_dw + 1e-40)
            assert bool((whole[:, H:] == -77.0).all())
