"""The gated product's vector form to codes, whose scale blocks are clusters of thread blocks that exchange their row
maxima: last clusters of which most blocks have no columns, reductions of one step, rows of no group (whose clusters
leave at once), and a GPU busy with other work, under which a cluster's blocks start when there is room.  Bounds as in
test_gemm_swiglu.py; a maximum does not depend on an order, so codes and scales have the same bits every time.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_fp8_block import offsets_of
from test_fp8_block_forms import VECTOR
from test_gemm_swiglu import TURN, check, problem, product
from test_rms_norm import BF16

pytestmark = pytest.mark.gpu
# dense rows, or rows of groups; two columns a warp from three grouped rows on, else one
ROWS = [([1], False), ([2], False), ([4], False), ([0, 1, 0, 1], True), ([1, 0, 2, 1], True)]


@pytest.mark.parametrize("counts,grouped", ROWS)
@pytest.mark.parametrize("I", [16, 128, 144, 1040])
@pytest.mark.parametrize("K", [16, 528, 2064])
def test_maxima_of_a_cluster(counts, grouped, I, K):
    extra = 4 - sum(counts) if grouped and sum(counts) < 4 else 0
    args = problem(sum(counts) + extra, I, K, len(counts), I + K, tame=True)
    offsets = offsets_of(counts).cuda() if grouped else None
    first, form = product(args, offsets, TURN, BF16)
    assert form == VECTOR
    check(args, first, counts, TURN, BF16)
    big = torch.randn(4096, 4096, device="cuda").to(BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(8):
            big @ big
    for _ in range(20):
        again, _ = product(args, offsets, TURN, BF16)
        for name in ("out", "codes", "scales", "gate_up"):
            assert torch.equal(again[name], first[name])
    side.synchronize()
