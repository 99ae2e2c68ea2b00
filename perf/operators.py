"""The expert-row and FP8 block-scaled operators at the sizes they are timed at, with their plain forms.

A case is a dict with the operator's name (``op``) and its sizes:

  gemm        y = x W_e^T over the rows of each expert, FP8 codes with one fp32 scale per 1x128 block of x and per
              128x128 block of W
  dgrad       dx = dy W_e, the same weights
  quantize    bf16 rows -> FP8 codes and 1x128 scales, written to each token's expert rows
  permute / permute_bwd       token rows to expert rows, and the gradient
  unpermute / unpermute_bwd   weighted sum back to token rows, and the gradients of rows and weights
  route_bwd   gradient of the renormalised top-k softmax weights with respect to the logits

``run`` computes them with elementary torch operations in fp32, or through the package where ``own`` is set.
"""
import math

import torch

own = False

BLOCK = 128
MAX_E4M3 = 448.0
TINY = 2.0 ** -100  # a block whose largest magnitude is below this gets the scale 0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a dense projection (E = 1): the smallest call of the product, latency counts
        {"name": "gemm_one_token", "op": "gemm", "T": 1, "k": 1, "E": 1, "N": 2304, "K": 5120, "dtype": "bf16"},
        # a decode batch over many experts, 1-6 rows each: the weight stream counts
        {"name": "gemm_decode_64", "op": "gemm", "T": 64, "k": 6, "E": 384, "N": 1280, "K": 5120, "dtype": "bf16"},
        # prefill on one of eight expert-parallel ranks (48 of 384 experts), about 1024 rows each: the tensor cores count
        {"name": "gemm_prefill", "op": "gemm", "T": 8192, "k": 6, "E": 48, "N": 6144, "K": 7168, "dtype": "bf16"},
        # input gradient through the draft layer's gate/up projection, ragged groups of about 96 rows
        {"name": "dgrad_train", "op": "dgrad", "T": 4096, "k": 3, "E": 128, "N": 2304, "K": 5120, "dtype": "bf16"},
        # quantise + dispatch of a decode batch, and of a prefill batch
        {"name": "quantize_decode", "op": "quantize", "T": 64, "H": 5120, "E": 384, "k": 6, "dtype": "bf16"},
        {"name": "quantize_prefill", "op": "quantize", "T": 8192, "H": 7168, "E": 384, "k": 6, "dtype": "bf16"},
        # dispatch of a prefill batch; its gradient in fp32 with an odd batch and pairs dropped at a capacity
        {"name": "permute_prefill", "op": "permute", "T": 8192, "H": 7168, "E": 384, "k": 6, "dtype": "bf16"},
        {"name": "permute_bwd_dropped", "op": "permute_bwd", "T": 4095, "H": 5120, "E": 128, "k": 3, "dtype": "f32",
         "drop": 0.05, "skew": True},
        # weighted sum back: a decode batch, and the gradients of a training batch
        {"name": "unpermute_decode", "op": "unpermute", "T": 16, "H": 7168, "E": 384, "k": 6, "dtype": "bf16"},
        {"name": "unpermute_bwd_train", "op": "unpermute_bwd", "T": 8192, "H": 7168, "E": 384, "k": 6, "dtype": "bf16"},
        # the router's gradient: a small batch of the draft router, a training batch of the large one
        {"name": "route_bwd_small", "op": "route_bwd", "T": 64, "E": 128, "k": 3},
        {"name": "route_bwd_train", "op": "route_bwd", "T": 8192, "E": 384, "k": 6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "dgrad", "dgrad", "quantize", "permute", "permute_bwd", "unpermute",
                     "unpermute_bwd", "route_bwd"])
    c = {"op": op, "E": _log(rng, 1, 384)}
    c["k"] = rng.randint(1, min(8, c["E"]))
    if op in ("gemm", "dgrad"):
        c["T"] = _log(rng, 1, 16384)
        c["K"] = 16 * _log(rng, 8, 448)
        c["N"] = 16 * _log(rng, 4, 384) if op == "dgrad" else _log(rng, 64, 6144)
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c["skew"] = rng.random() < 0.3
        # no more weights and products than the listed prefill case
        c["E"] = max(c["k"], min(c["E"], int(2.1e9 / (c["N"] * c["K"]))))
        c["T"] = max(1, min(c["T"], int(2.1e12 / (c["N"] * c["K"] * c["k"]))))
        return c
    c["T"] = _log(rng, 1, 16384)
    if op == "route_bwd":
        c["E"] = max(c["k"], _log(rng, 8, 1024))
        return c
    c["H"] = _log(rng, 64, 7168)
    if op == "quantize":
        c["H"] = max(64, c["H"] // 16 * 16)
    c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if c["dtype"] == "f32":  # no more bytes than the listed 16-bit cases
        c["T"] = min(c["T"], 4096)
    c["T"] = max(1, min(c["T"], int(8192 * 7168 * 6 / (c["H"] * c["k"]))))
    c["drop"] = rng.choice([0.0, 0.0, 0.1])
    c["skew"] = rng.random() < 0.3
    return c


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, cols, dtype):
    """Rows N(0, 1) with a spread of column magnitudes, as hidden states have."""
    spread = torch.exp(0.5 * _normal(gen, cols))
    return (_normal(gen, rows, cols) * spread).to(DTYPES[dtype])


def _logits(gen, case):
    lg = _normal(gen, case["T"], case["E"])
    return lg + 1.5 * _normal(gen, case["E"]) if case.get("skew") else lg


def _routed(gen, case):
    """Top-k routing of random logits and its stable sort by expert; dropped pairs have inv = -1."""
    T, E, k = case["T"], case["E"], case["k"]
    vals, ids = torch.topk(_logits(gen, case), k, dim=1)
    key = ids.reshape(-1)
    if case.get("drop"):
        lost = torch.rand(T * k, generator=gen, device="cuda") < case["drop"]
        key = torch.where(lost, E, key)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)
    R = T * k - int(counts[E])
    inv = torch.empty(T * k, dtype=torch.int32, device="cuda")
    inv[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    inv = torch.where(key == E, -1, inv).to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts[:E], 0)
    return {"ids": ids.to(torch.int32), "w": torch.softmax(vals, 1), "inv": inv.view(T, k), "R": R,
            "pair": order[:R].to(torch.int32), "offsets": offsets, "most": int(counts[:E].max())}


def _weights(gen, E, N, K):
    """N(0, 0.02) weights as FP8 codes [E, N, K] with one scale per 128x128 block, a few experts at a time."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), dtype=torch.float32, device="cuda")
    step = max(1, int(2.5e8 // (N * K)))
    for e in range(0, E, step):
        codes[e:e + step], scales[e:e + step] = _quantize(0.02 * _normal(gen, min(step, E - e), N, K), BLOCK)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    s.update(_routed(gen, case))
    T, k, R = case["T"], case["k"], s["R"]
    if op in ("gemm", "dgrad"):
        N, K, E = case["N"], case["K"], case["E"]
        inner, outer = (K, N) if op == "gemm" else (N, K)
        s["x"], s["xs"] = _quantize(_activations(gen, R, inner, "f32")[None], 1)
        s["x"], s["xs"] = s["x"][0], s["xs"][0]
        s["weight"], s["ws"] = _weights(gen, E, N, K)
        s["out"] = torch.empty(R, outer, dtype=DTYPES[case["dtype"]], device="cuda")
        s["grouped"] = E > 1
        s["workspace"] = None
    elif op == "route_bwd":
        s["dw"] = _normal(gen, T, k)
        s["out"] = torch.empty(T, case["E"], dtype=torch.float32, device="cuda")
    else:
        H, dt = case["H"], DTYPES[case["dtype"]]
        if op in ("permute", "quantize"):
            s["x"] = _activations(gen, T, H, case["dtype"])
        if op in ("permute_bwd", "unpermute", "unpermute_bwd"):
            s["rows"] = _activations(gen, R, H, case["dtype"])
        if op == "unpermute_bwd":
            s["dout"] = _normal(gen, T, H).to(dt)
            s["dw"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        if op == "quantize":
            s["out"] = torch.empty(R, H, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(R, -(-H // BLOCK), dtype=torch.float32, device="cuda")
        else:
            s["out"] = torch.empty(R if op in ("permute", "unpermute_bwd") else T, H, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms (fp32)

def _quantize(x, block_rows):
    """fp32 [B, rows, cols] -> E4M3 codes (uint8) of 448 x / amax and fp32 scales amax / 448 per block_rows x 128 block.

    7/8 x is exact for 16-bit x and one division rounds it, so a quotient halfway between two codes stays halfway."""
    B, rows, cols = x.shape
    pr, pc = -rows % block_rows, -cols % BLOCK
    if pr or pc:
        x = torch.nn.functional.pad(x, (0, pc, 0, pr))
    v = x.view(B, (rows + pr) // block_rows, block_rows, (cols + pc) // BLOCK, BLOCK)
    amax = v.abs().amax(dim=(2, 4), keepdim=True)
    tiny = amax < TINY
    scale = torch.where(tiny, 0.0, amax / MAX_E4M3)
    codes = torch.where(tiny, v * 0.0, v * 0.875 / amax * 512.0).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape)
    return codes[:, :rows, :cols].contiguous(), scale[:, :, 0, :, 0]


def _values(codes, scales, block_rows):
    """fp32 values of codes [B, rows, cols] with scales per block_rows x 128 block."""
    B, rows, cols = codes.shape
    v = codes.view(torch.float8_e4m3fn).float()
    if rows % block_rows == 0 and cols % BLOCK == 0:
        v = v.view(B, rows // block_rows, block_rows, cols // BLOCK, BLOCK)
        return v.mul_(scales[:, :, None, :, None]).view(B, rows, cols)
    if block_rows > 1:
        scales = scales.repeat_interleave(block_rows, 1)[:, :rows]
    return v.mul_(scales.repeat_interleave(BLOCK, 2)[:, :, :cols])


def _product(s, trans):
    """Rows of each expert times its weights, as one batched product over experts padded to the longest group."""
    x = _values(s["x"][None], s["xs"][None], 1)[0]
    w = _values(s["weight"], s["ws"], BLOCK)
    if trans:
        w = w.transpose(1, 2)
    at = torch.arange(x.shape[0], device="cuda")
    e = torch.searchsorted(s["offsets"], at, right=True) - 1
    pos = at - s["offsets"][e]
    padded = torch.zeros(w.shape[0], s["most"], x.shape[1], dtype=torch.float32, device="cuda")
    padded[e, pos] = x
    return torch.bmm(padded, w)[e, pos].to(s["out"].dtype)


def _plain(s):
    op = s["op"]
    if op == "gemm":
        return _product(s, True)
    if op == "dgrad":
        return _product(s, False)
    if op == "route_bwd":
        g = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True))
        return torch.zeros_like(s["out"]).scatter_(1, s["ids"].long(), g)
    k = s["case"]["k"]
    if op == "permute":
        return s["x"][s["pair"].long() // k]
    if op == "quantize":
        codes, scales = _quantize(s["x"].float()[None], 1)
        token = s["pair"].long() // k
        return {"codes": codes[0][token].view(torch.float8_e4m3fn), "scales": scales[0][token]}
    kept = (s["inv"] >= 0)[..., None]
    rows = torch.where(kept, s["rows"].float()[s["inv"].clamp(min=0).long()], 0.0)
    if op == "permute_bwd":
        return rows.sum(1).to(s["out"].dtype)
    if op == "unpermute":
        return (rows * s["w"][..., None]).sum(1).to(s["out"].dtype)
    d = s["dout"].float()
    pair = s["pair"].long()
    drows = d[pair // k] * s["w"].reshape(-1)[pair][:, None]
    return {"drows": drows.to(s["out"].dtype), "dw": (rows * d[:, None]).sum(2)}


# ---------------------------------------------------------------- the package's operators

def _workspace(moe, s):
    """The product's scratch memory, which a program allocates once for its sizes and keeps."""
    if s["workspace"] is None:
        c = s["case"]
        n = moe.moe_gemm_fp8_block_workspace_bytes(s["R"], c["N"], c["K"], c["E"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import block_scaled_moe_topk_gb300 as moe
    op, out = s["op"], s["out"]
    if op == "gemm" or op == "dgrad":
        call = moe.moe_gemm_fp8_block if op == "gemm" else moe.moe_gemm_fp8_block_dgrad
        call(s["x"], s["xs"], s["weight"], s["ws"], out, _workspace(moe, s),
             offsets=s["offsets"] if s["grouped"] else None)
    elif op == "route_bwd":
        moe.moe_topk_route_backward(s["ids"], s["w"], s["dw"], out)
    elif op == "permute":
        moe.moe_permute(s["x"], s["inv"], out)
    elif op == "quantize":
        moe.moe_permute_quantize_fp8_block(s["x"], s["inv"], out, s["scales"])
        return {"codes": out.view(torch.float8_e4m3fn), "scales": s["scales"]}
    elif op == "permute_bwd":
        moe.moe_permute_backward(s["rows"], s["inv"], out)
    elif op == "unpermute":
        moe.moe_unpermute(s["rows"], s["inv"], s["w"], out)
    else:
        moe.moe_unpermute_backward(s["dout"], s["rows"], s["inv"], s["w"], out, s["dw"])
        return {"drows": out, "dw": s["dw"]}
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the least work, and 64-bit results

def work(case):
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    R = T * k * (1.0 - case.get("drop", 0.0))
    if op == "route_bwd":
        return {"bytes": 4.0 * T * E + 12.0 * T * k, "flops": 4.0 * T * k}
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if op in ("gemm", "dgrad"):
        N, K = case["N"], case["K"]
        active = E * (1.0 - (1.0 - k / E) ** T)  # experts with a row, under even routing
        inner, outer = (K, N) if op == "gemm" else (N, K)
        blocks = -(-N // BLOCK) * -(-K // BLOCK)
        return {"bytes": active * (N * K + 4.0 * blocks) + R * (inner + 4.0 * -(-inner // BLOCK) + size * outer),
                "flops": 2.0 * R * N * K}
    H = case["H"]
    index = 4.0 * T * k
    if op == "quantize":
        return {"bytes": size * T * H + index + R * (H + 4.0 * -(-H // BLOCK)), "flops": 3.0 * T * H}
    if op == "unpermute":
        return {"bytes": size * (R * H + T * H) + 2 * index, "flops": 2.0 * R * H}
    if op == "unpermute_bwd":
        return {"bytes": size * (T * H + 2 * R * H) + 3 * index, "flops": 3.0 * R * H}
    return {"bytes": size * (T * H + R * H) + index, "flops": R * H if op == "permute_bwd" else 0.0}


def _e4m3_nearest(v):
    """The E4M3 value nearest to each fp64 value, |v| <= 448; halfway between two codes, the even one."""
    table = torch.arange(127, device=v.device).to(torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)
    middle = (table[1:] + table[:-1]) / 2
    mag = v.abs()
    i = torch.searchsorted(middle, mag)
    tie = (mag == middle[i.clamp(max=125)]) & (i % 2 == 1)
    return torch.copysign(table[i + tie.long()], v)


def exact(case, seed):
    s = prepare(case, seed)
    op, k = case["op"], case["k"]
    f64 = torch.float64
    if op in ("gemm", "dgrad"):
        if 2.0 * s["R"] * case["N"] * case["K"] > 1e13:
            return None
        out = torch.empty(s["out"].shape, dtype=f64, device="cuda")
        off = s["offsets"].tolist()
        inner = torch.arange(s["x"].shape[1], device="cuda") // BLOCK
        n, c = (torch.arange(case[d], device="cuda") // BLOCK for d in ("N", "K"))
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            w = s["weight"][e].view(torch.float8_e4m3fn).to(f64) * s["ws"][e].to(f64)[n][:, c]
            x = s["x"][a:b].view(torch.float8_e4m3fn).to(f64) * s["xs"][a:b].to(f64)[:, inner]
            out[a:b] = x @ (w.t() if op == "gemm" else w)
        return out
    if op == "route_bwd":
        w, dw = s["w"].to(f64), s["dw"].to(f64)
        out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
        rows = torch.arange(case["T"], device="cuda")
        mean = (w * dw).sum(1)
        for j in range(k):
            out[rows, s["ids"][:, j].long()] += w[:, j] * (dw[:, j] - mean)
        return out
    T, H, inv = case["T"], case["H"], s["inv"].long()
    if op == "quantize":
        x = torch.zeros(T, -(-H // BLOCK) * BLOCK, dtype=f64, device="cuda")
        x[:, :H] = s["x"].to(f64)
        v = x.view(T, -1, BLOCK)
        amax = v.abs().amax(2, keepdim=True)
        q = _e4m3_nearest(v * MAX_E4M3 / amax).view(T, -1)[:, :H]
        codes = torch.empty(s["R"], H, dtype=f64, device="cuda")
        scales = torch.empty(s["R"], v.shape[1], dtype=f64, device="cuda")
        for j in range(k):
            on = inv[:, j] >= 0
            codes[inv[on, j]] = q[on]
            scales[inv[on, j]] = amax[on, :, 0] / MAX_E4M3
        return {"codes": codes, "scales": scales}
    if op == "permute":
        out = torch.empty(s["R"], H, dtype=f64, device="cuda")
        for j in range(k):
            on = inv[:, j] >= 0
            out[inv[on, j]] = s["x"][on].to(f64)
        return out
    w = s["w"].to(f64)
    if op in ("permute_bwd", "unpermute"):
        out = torch.zeros(T, H, dtype=f64, device="cuda")
        for j in range(k):
            on = inv[:, j] >= 0
            row = s["rows"][inv[on, j]].to(f64)
            out[on] += row if op == "permute_bwd" else row * w[on, j][:, None]
        return out
    d = s["dout"].to(f64)
    drows = torch.empty(s["R"], H, dtype=f64, device="cuda")
    dw = torch.zeros(T, k, dtype=f64, device="cuda")
    for j in range(k):
        on = inv[:, j] >= 0
        drows[inv[on, j]] = d[on] * w[on, j][:, None]
        dw[on, j] = (d[on] * s["rows"][inv[on, j]].to(f64)).sum(1)
    return {"drows": drows, "dw": dw}
