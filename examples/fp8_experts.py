"""A router trained through frozen FP8 experts, from the library's single operators.

The expert layer with its weights as E4M3 codes and one fp32 scale per 128x128 block:

  forward   route -> sort -> permute + quantise -> gated product (SwiGLU and its codes in the same kernel) ->
            down product -> unpermute
  backward  unpermute backward -> quantise -> down input gradient -> SwiGLU backward to codes ->
            gate/up input gradient -> permute backward, and route backward for the logits

``Fp8Block`` puts the layer behind the residual stream as a model does: residual's addition, RMS norm and quantisation
in one kernel, whose bf16 rows go to the router and whose codes go to the experts; and all of it back.

``python examples/fp8_experts.py`` trains a router (a linear map from the tokens to the logits) whose
experts stay fixed, towards the outputs that another router would give, and prints the loss.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_moe_topk_gb300 as moe  # noqa: E402


def quantize(x):
    """Rows -> (E4M3 codes, fp32 scales per 1x128 block)."""
    rows, K = x.shape
    codes = torch.empty(rows, K, dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, -(-K // 128), dtype=torch.float32, device=x.device)
    moe.moe_quantize_fp8_block(x, codes, scales)
    return codes, scales


def quantize_weights(w):
    """[E, N, K] -> (E4M3 codes, fp32 scales per 128x128 block), expert by expert."""
    E, N, K = w.shape
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=w.device)
    scales = torch.empty(E, -(-N // 128), -(-K // 128), dtype=torch.float32, device=w.device)
    for e in range(E):
        moe.moe_quantize_fp8_block(w[e], codes[e], scales[e], block_rows=128)
    return codes, scales


class Fp8Experts:
    """E SwiGLU experts [E, 2I, H] (rows 2j gate, 2j + 1 up) and [E, H, I], top-k routing."""

    def __init__(self, w1, w2, k):
        self.E, self.I, self.H, self.k = w1.shape[0], w2.shape[2], w2.shape[1], k
        self.w1, self.s1 = quantize_weights(w1)
        self.w2, self.s2 = quantize_weights(w2)
        self.device = w1.device

    def _space(self, M, N, K):
        return torch.empty(moe.moe_gemm_fp8_block_workspace_bytes(M, N, K, self.E), dtype=torch.uint8, device=self.device)

    def _gemm(self, call, x, w, scales, cols):
        codes, xs = x if isinstance(x, tuple) else quantize(x)
        out = torch.empty(codes.shape[0], cols, dtype=torch.bfloat16, device=self.device)
        call(codes, xs, w, scales, out, self._space(codes.shape[0], *w.shape[1:]), offsets=self.offsets)
        return out

    def forward(self, x, logits, quantized=None):
        """``quantized``: (codes, scales) of x's rows, where they are at hand."""
        T, dev = x.shape[0], self.device
        R, blocks = T * self.k, -(-self.H // 128)
        new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=dev)  # noqa: E731
        self.ids, self.w = new(T, self.k, dtype=torch.int32), new(T, self.k, dtype=torch.float32)
        moe.moe_topk_route(logits, self.k, self.ids, self.w)
        counts, self.offsets = new(self.E, dtype=torch.int32), new(self.E + 1, dtype=torch.int64)
        pair, self.inv = new(R, dtype=torch.int32), new(T, self.k, dtype=torch.int32)
        scratch = new(moe.moe_workspace_bytes(T, 128, 128, self.E, self.k), dtype=torch.uint8)
        moe.moe_sort_by_expert(self.ids, self.E, counts, self.offsets, pair, self.inv, scratch)
        codes, scales = new(R, self.H, dtype=torch.uint8), new(R, blocks, dtype=torch.float32)
        if quantized is None:
            moe.moe_permute_quantize_fp8_block(x, self.inv, codes, scales)
        else:
            moe.moe_permute(quantized[0], self.inv, codes)
            moe.moe_permute(quantized[1], self.inv, scales)
        h, hs = new(R, self.I, dtype=torch.uint8), new(R, -(-self.I // 128), dtype=torch.float32)
        self.gate_up = new(R, 2 * self.I, dtype=torch.bfloat16)  # the backward pass reads the products
        moe.moe_gemm_fp8_block_swiglu(codes, scales, self.w1, self.s1, self._space(R, 2 * self.I, self.H), codes=h,
                                      scales=hs, gate_up=self.gate_up, offsets=self.offsets)
        self.y = self._gemm(moe.moe_gemm_fp8_block, (h, hs), self.w2, self.s2, self.H)
        out = torch.empty_like(x)
        moe.moe_unpermute(self.y, self.inv, self.w, out)
        return out

    def backward(self, dout):
        """Gradients of x and of the logits for the last forward."""
        dy, dw = torch.empty_like(self.y), torch.empty_like(self.w)
        moe.moe_unpermute_backward(dout, self.y, self.inv, self.w, dy, dw)
        dh = self._gemm(moe.moe_gemm_fp8_block_dgrad, dy, self.w2, self.s2, self.I)
        codes = torch.empty(self.gate_up.shape, dtype=torch.uint8, device=self.device)
        scales = torch.empty(codes.shape[0], -(-codes.shape[1] // 128), dtype=torch.float32, device=self.device)
        moe.moe_swiglu_backward(self.gate_up, dh, codes=codes, scales=scales)
        drows = self._gemm(moe.moe_gemm_fp8_block_dgrad, (codes, scales), self.w1, self.s1, self.H)
        dx = torch.empty_like(dout)
        moe.moe_permute_backward(drows, self.inv, dx)
        dlogits = torch.empty(dout.shape[0], self.E, dtype=torch.float32, device=self.device)
        moe.moe_topk_route_backward(self.ids, self.w, dw, dlogits)
        return dx, dlogits


class Fp8Block:
    """out = experts(norm(stream)) with stream = x + residual, the norm's rows routed by a linear map [H, E]."""

    def __init__(self, experts, weight, router, eps=1e-6):
        self.experts, self.weight, self.router, self.eps = experts, weight, router, eps

    def forward(self, x, residual):
        """(experts' output, stream): the next block adds them up in its own norm."""
        T, H = x.shape
        self.stream, self.normed = torch.empty_like(x), torch.empty_like(x)
        self.rstd = torch.empty(T, dtype=torch.float32, device=x.device)
        codes = torch.empty(T, H, dtype=torch.uint8, device=x.device)
        scales = torch.empty(T, -(-H // 128), dtype=torch.float32, device=x.device)
        moe.moe_rms_norm_quantize_fp8_block(x, self.weight, self.eps, codes, scales, out=self.normed, residual=residual,
                                            residual_out=self.stream, rstd=self.rstd)
        return self.experts.forward(self.normed, self.normed.float() @ self.router, (codes, scales)), self.stream

    def backward(self, dout, dstream):
        """Gradients of x (and of residual, the same), of the norm's weight and of the router, from those of the two
        outputs."""
        dnormed, dlogits = self.experts.backward(dout)
        self.dnormed = (dnormed.float() + dlogits @ self.router.t()).to(dout.dtype)
        drouter = self.normed.float().t() @ dlogits
        dx, dweight = torch.empty_like(dout), torch.empty(self.weight.shape, dtype=torch.float32, device=dout.device)
        space = torch.empty(moe.moe_rms_norm_backward_workspace_bytes(*dout.shape), dtype=torch.uint8, device=dout.device)
        moe.moe_rms_norm_backward(self.dnormed, self.stream, self.weight, self.rstd, dx, dweight, space,
                                  d_residual=dstream)
        return dx, dweight, drouter


def make_experts(E, H, I, k, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    w1 = torch.randn(E, 2 * I, H, generator=g, device=device) * H ** -0.5
    w2 = torch.randn(E, H, I, generator=g, device=device) * I ** -0.5
    return Fp8Experts(w1, w2, k)


def train(T=1024, H=512, I=256, E=16, k=4, steps=40, seed=0, device="cuda"):
    """Losses of training the router by plain gradient descent."""
    experts = make_experts(E, H, I, k, seed, device)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    x = torch.randn(T, H, generator=g, device=device).to(torch.bfloat16)
    teacher = torch.randn(H, E, generator=g, device=device) * H ** -0.5
    # the student starts near the teacher: the same experts, other weights
    router = teacher + 0.7 * torch.randn(H, E, generator=g, device=device) * H ** -0.5
    target = experts.forward(x, x.float() @ teacher).float()
    losses = []
    for _ in range(steps):
        out = experts.forward(x, x.float() @ router).float()
        diff = out - target
        losses.append(float(diff.square().mean()))
        _, dlogits = experts.backward((2.0 / T * diff).to(torch.bfloat16))
        router -= 0.02 * (x.float().t() @ dlogits)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args()
    losses = train(T=args.tokens, steps=args.steps)
    for i in range(0, len(losses), max(1, len(losses) // 8)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"last       loss {losses[-1]:.5f}")
