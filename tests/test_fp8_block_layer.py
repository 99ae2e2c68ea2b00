"""The norm, the gated product and their gradients as a model uses them: examples/fp8_experts.py's Fp8Block, forward
and backward, against fp64.

The forward quantises the norm's rows and h, each with an rms of at most 2^-4 / sqrt(3) = 3.6 % (test_fp8_experts.py):
at most 5.1 % together, and 7.2 % for the experts' input gradient, plus bf16's roundings, under 1 %.  The norm's own
gradients are held to the formula on what reached them, within fp32's roundings (test_rms_norm.py).
"""
import pytest
import torch

from test_fp8_experts import example, rel, values
from test_rms_norm import BF16, F32, F64, HALF, U, backward64, near, norm64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def block(T, H, I, E, k, wtype=BF16, seed=0):
    m = example()
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    weight, router = (1 + 0.2 * n(H)).to(wtype), n(H, E) * H ** -0.5
    b = m.Fp8Block(m.make_experts(E, H, I, k, seed), weight, router, EPS)
    return b, n(T, H).to(BF16), n(T, H).to(BF16), n(T, H).to(BF16), n(T, H).to(BF16)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (2, 384, 256, 1, 1), (64, 512, 256, 16, 4),
                                       (300, 384, 640, 5, 3), (2500, 512, 384, 4, 2)])
@pytest.mark.parametrize("wtype", [BF16, F32])
def test_block_and_gradients(T, H, I, E, k, wtype):
    b, x, r, dout, dstream = block(T, H, I, E, k, wtype)
    out, stream = b.forward(x, r)
    dx, dweight, drouter = b.backward(dout, dstream)
    s, rstd, y = norm64(x, r, b.weight)
    near(stream, s, 2 * U + HALF[BF16])
    near(b.normed, y, 64 * U + HALF[BF16])
    near(b.rstd, rstd, 64 * U)
    # the experts in fp64 on the layer's own weights and selection
    layer = b.experts
    w1, w2 = values(layer.w1, layer.s1), values(layer.w2, layer.s2)
    Y = y.clone().requires_grad_()
    L = (b.normed.double() @ b.router.double()).requires_grad_()
    ids = layer.ids.long()
    w = torch.softmax(L.gather(1, ids), 1)
    h = torch.einsum("th,enh->ten", Y, w1)
    act = torch.nn.functional.silu(h[..., 0::2]) * h[..., 1::2]
    rows = torch.einsum("tei,ehi->teh", act, w2).gather(1, ids[..., None].expand(T, k, H))
    want = (rows * w[..., None]).sum(1)
    want.backward(dout.double())
    assert rel(out, want.detach()) <= 0.06
    # what reached the norm: the experts' gradient, and the logits' as the layer has it
    experts = b.dnormed.double() - drouter_part(b, dout)
    assert rel(experts, Y.grad) <= 0.082
    dx64, size, dw64, size_dw = backward64(b.dnormed, b.stream, b.weight, b.rstd, dstream)
    near(dx, dx64, HALF[BF16], 96 * U * size)
    near(dweight, dw64, 0.0, (2 + T + 304 + 64) * U * size_dw + 1e-40)
    if E > k:
        assert bool(torch.isfinite(drouter).all()) and float(drouter.abs().max()) > 0


def drouter_part(b, dout):
    """The logits' share of what reached the norm, as the layer's last backward left it."""
    _, dlogits = b.experts.backward(dout)
    return (dlogits @ b.router.t()).double()


def test_two_blocks_in_a_graph():
    """A decode step of two blocks, the second adding the first's output to the stream: captured, replayed on new
    values, the same bits as run eagerly."""
    b1, x, r, _, _ = block(5, 384, 256, 8, 2, seed=1)
    b2 = block(5, 384, 256, 8, 2, seed=2)[0]

    def step():
        return b2.forward(*b1.forward(x, r))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, stream = step()
    x.copy_(torch.randn(5, 384, device="cuda", generator=torch.Generator(device="cuda").manual_seed(77)))
    graph.replay()
    torch.cuda.synchronize()
    want, ws = step()
    assert torch.equal(out, want) and torch.equal(stream, ws)


def test_same_result_every_time():
    b, x, r, dout, dstream = block(700, 512, 256, 6, 2)
    first = [*b.forward(x, r), *b.backward(dout, dstream)]
    again = [*b.forward(x, r), *b.backward(dout, dstream)]
    for i in (0, 1, 2, 3):  # the router's gradient is torch's own product
        assert torch.equal(first[i], again[i])
