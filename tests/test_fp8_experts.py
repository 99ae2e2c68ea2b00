"""The example layer (examples/fp8_experts.py): the single operators together, forward and backward.

Against fp64 with the layer's own weight codes.  Each quantisation of activations or gradients to E4M3
rounds an element by at most 2^-4 of itself, evenly spread: an rms of at most 2^-4 / sqrt(3) = 3.6 % a
time.  The forward quantises twice, the input gradient twice more on top of it: relative errors of at
most sqrt(2) x 3.6 % = 5.1 % and sqrt(4) x 3.6 % = 7.2 % (bf16's own rounding adds under 1 %).  The
logits' gradient is a difference of dot products, whose relative error has no such bound: it is held
to the formula on the layer's own expert outputs, within the fp32 rounding of its sums (64 terms in a
row for a dot product, k + 3 roundings after it).
"""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("fp8_experts", os.path.join(ROOT, "examples", "fp8_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def values(codes, scales):
    E, N, K = codes.shape
    s = scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return codes.view(torch.float8_e4m3fn).double() * s


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (64, 512, 256, 16, 4), (300, 384, 640, 5, 3)])
def test_layer_and_gradients(T, H, I, E, k):
    m = example()
    layer = m.make_experts(E, H, I, k)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    dout = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    out = layer.forward(x, logits)
    dx, dlogits = layer.backward(dout)
    # fp64: every expert on every token, the selected ones weighted
    w1, w2 = values(layer.w1, layer.s1), values(layer.w2, layer.s2)
    X = x.double().requires_grad_()
    L = logits.double().requires_grad_()
    sel = torch.topk(L, k, dim=1).indices
    w = torch.softmax(L.gather(1, sel), 1)
    h = torch.einsum("th,enh->ten", X, w1)
    act = torch.nn.functional.silu(h[..., 0::2]) * h[..., 1::2]
    y = torch.einsum("tei,ehi->teh", act, w2)
    want = (y.gather(1, sel[..., None].expand(T, k, H)) * w[..., None]).sum(1)
    want.backward(dout.double())
    assert rel(out, want.detach()) <= 0.06
    assert rel(dx, X.grad) <= 0.082
    inv = layer.inv.long()
    dots = layer.y.double()[inv] * dout.double()[:, None]
    W, dw, size = layer.w.double(), dots.sum(2), dots.abs().sum(2)
    grad = W * (dw - (W * dw).sum(1, keepdim=True))
    bound = (64 + k + 3) * 2.0 ** -24 * W * (size + (W * size).sum(1, keepdim=True))
    ids = layer.ids.long()
    assert torch.equal(ids, sel)
    err = (dlogits.double() - torch.zeros_like(logits).double().scatter_(1, ids, grad)).abs()
    assert bool((err <= torch.zeros_like(err).scatter_(1, ids, bound)).all())


@pytest.mark.gpu
def test_router_learns():
    losses = example().train(T=256, H=256, I=128, E=8, k=2, steps=12)
    assert losses[-1] < 0.8 * losses[0]
