"""FP8 codes of values that a kernel has just computed in fp32, against the quantiser on those values: the norm, the
gated product in each of its forms and the activation's gradient leave both.  The scales are the quantiser's bit for
bit (m / 448, rounded once); a code is the one nearest to 448 v / m, either neighbour within 2^-20 of a tie."""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_fp8_block import ceil_div, offsets_of
from test_fp8_block_forms import PAIR, SINGLE, SPLIT, VECTOR
from test_gemm_swiglu import STACK, TURN, problem, product
from test_rms_norm import EPS, F32, F64, gen

pytestmark = pytest.mark.gpu


def same_as_the_quantiser(v, codes, scales):
    R, C = v.shape
    want_c, want_s = torch.empty_like(codes), torch.empty_like(scales)
    moe.moe_quantize_fp8_block(v, want_c, want_s)
    assert torch.equal(scales, want_s), f"{int((scales != want_s).sum())} of {scales.numel()} scales differ"
    p = torch.nn.functional.pad(v.to(F64), (0, -C % 128)).view(R, -1, 128)
    m = p.abs().amax(2, keepdim=True)
    q = torch.where(m < 2.0 ** -100, 0.0, 448 * p / m.clamp_min(2.0 ** -100)).view(R, -1)[:, :C]
    half = 2.0 ** (torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 4)  # half a step of q's binade
    code = codes.view(torch.float8_e4m3fn).to(F64)
    assert bool(((code - q).abs() <= half + 2.0 ** -20 * q.abs()).all())
    assert bool((torch.signbit(code) == torch.signbit(v)).all())


@pytest.mark.parametrize("H", [32, 128, 999, 1000, 5120, 8193])
@pytest.mark.parametrize("size", [1.0, 1e-25, 1e30])
def test_norm(H, size):
    T = 3000 if H <= 1000 else 400
    g = gen(H)
    x = torch.randn(T, H, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    w = size * torch.randn(H, generator=g, device="cuda")
    out, codes = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, ceil_div(H, 128), device="cuda")
    moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, codes, scales, out=out)
    same_as_the_quantiser(out, codes, scales)


@pytest.mark.parametrize("I", [64, 128, 264, 1001, 1152])
@pytest.mark.parametrize("layout", [TURN, STACK])
def test_activation_gradient(I, layout):
    if layout == STACK:
        I = 128 * ceil_div(I, 128)
    R = 1500
    g = gen(I)
    gate_up, dh = torch.randn(R, 2 * I, generator=g, device="cuda"), torch.randn(R, I, generator=g, device="cuda")
    d, codes = torch.empty_like(gate_up), torch.empty(R, 2 * I, dtype=torch.uint8, device="cuda")
    scales = torch.empty(R, ceil_div(2 * I, 128), device="cuda")
    moe.moe_swiglu_backward(gate_up, dh, d_gate_up=d, codes=codes, scales=scales, layout=layout)
    same_as_the_quantiser(d, codes, scales)


@pytest.mark.parametrize("form,counts,I,K", [(VECTOR, [4], 512, 1040), (VECTOR, [1, 0, 2], 1152, 528),
                                             (SPLIT, [100], 512, 5120), (SPLIT, [17, 16, 31], 144, 4096),
                                             (SINGLE, [37, 0, 15, 1, 64, 130, 0, 33, 5] * 9, 400, 400),
                                             (PAIR, [2092, 0, 15, 4807, 33], 528, 2064)])
@pytest.mark.parametrize("tame", [False, True])
def test_gated_product(form, counts, I, K, tame):
    args = problem(sum(counts), I, K, len(counts), I, tame)
    got, ran = product(args, offsets_of(counts).cuda() if len(counts) > 1 else None, TURN, F32, keep=False)
    assert ran == form
    same_as_the_quantiser(got["out"], got["codes"], got["scales"])
