"""A router trained through frozen FP8 experts, from the library's single operators.

The expert layer with its weights as E4M3 codes and one fp32 scale per 128x128 block:

  forward   route -> sort -> permute + quantise -> gate/up product -> SwiGLU -> quantise ->
            down product -> unpermute
  backward  unpermute backward -> quantise -> down input gradient -> SwiGLU backward -> quantise ->
            gate/up input gradient -> permute backward, and route backward for the logits

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

    def _gemm(self, call, x, w, scales, cols):
        out = torch.empty(x.shape[0], cols, dtype=torch.bfloat16, device=self.device)
        E, N, K = w.shape
        space = torch.empty(moe.moe_gemm_fp8_block_workspace_bytes(x.shape[0], N, K, E), dtype=torch.uint8,
                            device=self.device)
        codes, xs = x if isinstance(x, tuple) else quantize(x)
        call(codes, xs, w, scales, out, space, offsets=self.offsets)
        return out

    def forward(self, x, logits):
        T, dev = x.shape[0], self.device
        R = T * self.k
        new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=dev)  # noqa: E731
        self.ids, self.w = new(T, self.k, dtype=torch.int32), new(T, self.k, dtype=torch.float32)
        moe.moe_topk_route(logits, self.k, self.ids, self.w)
        counts, self.offsets = new(self.E, dtype=torch.int32), new(self.E + 1, dtype=torch.int64)
        pair, self.inv = new(R, dtype=torch.int32), new(T, self.k, dtype=torch.int32)
        scratch = new(moe.moe_workspace_bytes(T, 128, 128, self.E, self.k), dtype=torch.uint8)
        moe.moe_sort_by_expert(self.ids, self.E, counts, self.offsets, pair, self.inv, scratch)
        codes, scales = new(R, self.H, dtype=torch.uint8), new(R, -(-self.H // 128), dtype=torch.float32)
        moe.moe_permute_quantize_fp8_block(x, self.inv, codes, scales)
        h = new(R, 2 * self.I, dtype=torch.bfloat16)
        space = new(moe.moe_gemm_fp8_block_workspace_bytes(R, 2 * self.I, self.H, self.E), dtype=torch.uint8)
        moe.moe_gemm_fp8_block(codes, scales, self.w1, self.s1, h, space, offsets=self.offsets)
        self.gate, self.up = h.float()[:, 0::2], h.float()[:, 1::2]
        act = (torch.nn.functional.silu(self.gate) * self.up).to(torch.bfloat16)
        self.y = self._gemm(moe.moe_gemm_fp8_block, act, self.w2, self.s2, self.H)
        out = torch.empty_like(x)
        moe.moe_unpermute(self.y, self.inv, self.w, out)
        return out

    def backward(self, dout):
        """Gradients of x and of the logits for the last forward."""
        dy, dw = torch.empty_like(self.y), torch.empty_like(self.w)
        moe.moe_unpermute_backward(dout, self.y, self.inv, self.w, dy, dw)
        dact = self._gemm(moe.moe_gemm_fp8_block_dgrad, dy, self.w2, self.s2, self.I).float()
        sig = torch.sigmoid(self.gate)
        dgate = dact * self.up * sig * (1 + self.gate * (1 - sig))
        dup = dact * self.gate * sig
        dh = torch.stack([dgate, dup], 2).reshape(dy.shape[0], 2 * self.I).to(torch.bfloat16)
        drows = self._gemm(moe.moe_gemm_fp8_block_dgrad, dh, self.w1, self.s1, self.H)
        dx = torch.empty_like(dout)
        moe.moe_permute_backward(drows, self.inv, dx)
        dlogits = torch.empty(dout.shape[0], self.E, dtype=torch.float32, device=self.device)
        moe.moe_topk_route_backward(self.ids, self.w, dw, dlogits)
        return dx, dlogits


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
