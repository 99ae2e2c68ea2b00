"""The gradients of unpermute over what decides which kernel instance runs: the slots (up to four, or more), the
access width that addresses, strides and row length allow, short and long rows, few and many tokens.

A dot product of H terms is shared by 32 threads or more: a thread adds at most ceil(H / 32) + 16 terms (its share
rounded up to a round of loads), five shuffles and at most 32 warps' sums follow, so that it is within
(ceil(H / 32) + 53) 2^-24 sum |terms| of the exact one.  A row of the other gradient is one product, rounded to
fp32 and to its type: within 2 u of itself.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_expert_rows import DTYPES, SMALLEST, U, mapping, rows_like

pytestmark = pytest.mark.gpu


def reference(dout, rows, inv, w):
    """(d_rows where named, d_topk_w, sum of |terms|) in fp64 on the GPU."""
    on = inv >= 0
    full = torch.where(on[..., None], rows.double()[inv.clamp(min=0).long()], 0.0)
    prod = full * dout.double()[:, None]
    drows = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
    drows[inv[on].long()] = (w.double()[..., None] * dout.double()[:, None])[on]
    return drows, prod.sum(2), prod.abs().sum(2)


def check(dout, rows, inv, w, drows, dw, named_only):
    H, dtype = rows.shape[1], rows.dtype
    want_rows, want_dw, size = reference(dout, rows, inv, w)
    named = torch.zeros(rows.shape[0], dtype=torch.bool, device="cuda")
    named[inv[inv >= 0].long()] = True
    err = (drows.double() - want_rows).abs()[named]
    assert bool((err <= 2 * U[dtype] * want_rows[named].abs() + SMALLEST[dtype]).all())
    assert bool((drows[~named] == named_only).all())
    err = (dw.double() - want_dw).abs()
    bound = (-(-H // 32) + 53) * 2.0 ** -24 * size
    assert bool((err <= bound).all()), f"worst {float((err / bound).nan_to_num().max()):.3g}"
    assert bool((dw[inv < 0] == 0).all())


def inputs(T, H, k, E, dtype, drop, seed):
    _, inv, R = mapping(T, k, E, seed, drop, extra=2)
    return (rows_like(T, H, dtype=dtype, seed=seed + 1).cuda(), rows_like(R, H, dtype=dtype, seed=seed + 2).cuda(),
            inv.cuda(), torch.softmax(rows_like(T, k, dtype=torch.float32, seed=seed + 3), 1).cuda())


# (T, H, k, E); T <= 152 spreads a row wider
CASES = [(200, 4104, 6, 16), (200, 2054, 8, 16), (200, 1887, 6, 16), (40, 124, 8, 16), (160, 64, 5, 8), (200, 130, 7, 9),
         (180, 65, 8, 16), (300, 7168, 8, 32), (200, 5120, 5, 16), (200, 2048, 7, 16), (200, 2044, 6, 16), (200, 1028, 4, 8),
         (200, 2054, 3, 16), (200, 1887, 4, 16), (200, 7168, 2, 8), (170, 260, 3, 8), (153, 516, 5, 6), (152, 4104, 6, 16),
         (16, 2054, 7, 16), (3, 1887, 8, 8), (1, 5120, 6, 8)]


@pytest.mark.parametrize("T,H,k,E", CASES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.5])
def test_against_fp64(T, H, k, E, dtype, drop):
    dout, rows, inv, w = inputs(T, H, k, E, dtype, drop, T + H)
    drows = torch.full_like(rows, 3.0)
    dw = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_unpermute_backward(dout, rows, inv, w, drows, dw)
    check(dout, rows, inv, w, drows, dw, 3.0)
    alone, dw_alone = torch.full_like(rows, 3.0), torch.empty_like(dw)
    moe.moe_unpermute_backward(dout, None, inv, w, alone, None)
    moe.moe_unpermute_backward(dout, rows, inv, w, None, dw_alone)
    assert torch.equal(alone, drows) and torch.equal(dw_alone, dw)


@pytest.mark.parametrize("k", [3, 6])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("by", [8, 4, 2, 1])
def test_narrow_accesses(k, dtype, by):
    """Strides and bases that leave 16, 8, 4 and 2-byte accesses to rows of one length."""
    T, H = 170, 1056
    dout, rows, inv, w = inputs(T, H, k, 16, dtype, 0.2, by)

    def shifted(t):
        v = torch.zeros(t.shape[0], H + 2 * by, dtype=dtype, device="cuda")[:, by:by + H]
        v.copy_(t)
        return v

    drows, dw = shifted(torch.full_like(rows, 3.0)), torch.empty(T, k, device="cuda")
    moe.moe_unpermute_backward(shifted(dout), shifted(rows), inv, w, drows, dw)
    check(dout, rows, inv, w, drows, dw, 3.0)


@pytest.mark.parametrize("T,H,k,E", [(200, 4104, 6, 16), (200, 2054, 8, 16), (200, 1887, 4, 16), (40, 124, 8, 16),
                                     (16, 7168, 6, 16), (200, 2048, 7, 16), (200, 1028, 4, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_in_place_of_the_rows(T, H, k, E, dtype):
    """d_rows may be rows: every element is read before it is written, by the thread that writes it."""
    dout, rows, inv, w = inputs(T, H, k, E, dtype, 0.3, 7)
    drows, dw = rows.clone(), torch.empty(T, k, device="cuda")
    moe.moe_unpermute_backward(dout, rows, inv, w, drows, dw)
    same, dw2 = rows.clone(), torch.empty_like(dw)
    moe.moe_unpermute_backward(dout, same, inv, w, same, dw2)
    assert torch.equal(same, drows) and torch.equal(dw2, dw)
