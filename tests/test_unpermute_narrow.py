"""unpermute and the gradient of permute on rows that allow 8-byte accesses: both forms of the sums (four 8-byte or
four 4-byte accesses a thread), by slots, row length and unused accesses, against fp64.

A sum of k terms in fp32, rounded once: within u |ref| + k 2^-24 sum |terms| of the exact one.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_expert_rows import DTYPES, SMALLEST, U, mapping, rows_like

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1, 2, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("row_bytes", [8, 248, 504, 1032, 2056, 3784, 10248, 14328])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_on_eight_bytes(k, row_bytes, dtype):
    T, H = 21, row_bytes // dtype.itemsize
    _, inv, R = mapping(T, k, max(k, 9), row_bytes + k, 0.25, extra=1)
    rows, inv = rows_like(R, H, dtype=dtype, seed=k).cuda(), inv.cuda()
    w = torch.softmax(rows_like(T, k, dtype=torch.float32, seed=3), 1).cuda()
    full = torch.where((inv >= 0)[..., None], rows.double()[inv.clamp(min=0).long()], 0.0)
    out = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
    for terms in (full * w.double()[..., None], full):
        if terms is full:
            moe.moe_permute_backward(rows, inv, out)
        else:
            moe.moe_unpermute(rows, inv, w, out)
        want = terms.sum(1)
        bound = U[dtype] * want.abs() + k * 2.0 ** -24 * terms.abs().sum(1) + SMALLEST[dtype]
        assert bool(((out.double() - want).abs() <= bound).all())
        out.fill_(float("nan"))
