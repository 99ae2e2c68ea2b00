"""The norm before an expert layer and its gated product at the sizes they are timed at, with their plain forms.

A case is a dict with the operator's name (``op``) and its sizes:

  norm            y = w (x + r) / sqrt(mean((x + r)^2) + eps) of each row, with the sum x + r written too
  norm_quantize   the same, leaving as FP8 codes with a scale per 1x128 block ("fp8": fp32, "mx": 1x32, power of two),
                  and as y itself for the router
  norm_bwd        gradients of the norm with respect to its rows and its weight
  swiglu          h = silu(x G_e^T) * (x U_e^T) over the rows of each expert, FP8 codes with one fp32 scale per 1x128
                  block of x and per 128x128 block of the weights; h as codes with 1x128 scales or as it is, the two
                  products kept for the gradient where a case says so
  swiglu_bwd      gradients of the two products, as codes with 1x128 scales or as they are

``run`` computes them with elementary torch operations in fp32, or through the package where ``own`` is set.
"""
import math

import torch

own = False

BLOCK = 128
MX_BLOCK = 32
MAX_E4M3 = 448.0
TINY = 2.0 ** -100  # a 1x128 block whose largest magnitude is below this gets the scale 0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the norm of one decoded token with its residual: the smallest call, latency counts
        {"name": "norm_one_token", "op": "norm", "T": 1, "H": 5120, "dtype": "bf16", "residual": True, "train": False},
        # a training batch's norm with its residual, the rows' 1/rms kept: bandwidth counts
        {"name": "norm_train", "op": "norm", "T": 8192, "H": 7168, "dtype": "bf16", "residual": True, "train": True},
        # before the experts of a decode batch: FP8 rows for the experts and bf16 rows for the router
        {"name": "norm_fp8_decode", "op": "norm_quantize", "T": 64, "H": 5120, "dtype": "bf16", "residual": True,
         "fmt": "fp8", "keep": True},
        # before the MX layer of a prefill batch
        {"name": "norm_mx_prefill", "op": "norm_quantize", "T": 8192, "H": 7168, "dtype": "bf16", "residual": True,
         "fmt": "mx", "keep": True},
        # the norm's gradients: a training batch on the residual stream, and an odd batch in fp32
        {"name": "norm_bwd_train", "op": "norm_bwd", "T": 8192, "H": 7168, "dtype": "bf16", "residual": True},
        {"name": "norm_bwd_f32", "op": "norm_bwd", "T": 4095, "H": 5120, "dtype": "f32", "residual": False},
        # one token through a dense gated block (E = 1)
        {"name": "swiglu_one_token", "op": "swiglu", "T": 1, "k": 1, "E": 1, "I": 1152, "K": 5120, "dtype": "bf16",
         "quantized": True, "save": False, "stacked": False},
        # a decode batch over many experts, 1-6 rows each: the weight stream counts
        {"name": "swiglu_decode_64", "op": "swiglu", "T": 64, "k": 6, "E": 384, "I": 640, "K": 5120, "dtype": "bf16",
         "quantized": True, "save": False, "stacked": False},
        # prefill on one of eight expert-parallel ranks, about 1024 rows an expert: the tensor cores count
        {"name": "swiglu_prefill", "op": "swiglu", "T": 8192, "k": 6, "E": 48, "I": 2048, "K": 7168, "dtype": "bf16",
         "quantized": True, "save": False, "stacked": True},
        # training forward of the draft layer, ragged groups of about 96 rows, both products kept
        {"name": "swiglu_train", "op": "swiglu", "T": 4096, "k": 3, "E": 128, "I": 1152, "K": 5120, "dtype": "bf16",
         "quantized": True, "save": True, "stacked": False},
        # the gated block's gradient: a small batch, and a training batch whose result goes into the next FP8 product
        {"name": "swiglu_bwd_small", "op": "swiglu_bwd", "R": 96, "I": 1152, "dtype": "bf16", "quantized": True,
         "stacked": False},
        {"name": "swiglu_bwd_train", "op": "swiglu_bwd", "R": 49152, "I": 2048, "dtype": "bf16", "quantized": True,
         "stacked": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_quantize", "norm_bwd", "swiglu", "swiglu", "swiglu", "swiglu_bwd"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op.startswith("norm"):
        c["H"] = _log(rng, 32, 8192)
        if op == "norm_quantize":
            c["fmt"], c["keep"] = rng.choice(["fp8", "mx"]), rng.random() < 0.7
            if c["fmt"] == "mx":
                c["H"] = max(32, c["H"] // 32 * 32)
        # rows of many short heads too; no more bytes than the listed 16-bit cases
        most = 8192 * 7168 // (2 if c["dtype"] == "f32" else 1)
        c["T"] = max(1, min(_log(rng, 1, 65536), most // c["H"]))
        c["residual"] = rng.random() < 0.6
        if op == "norm":
            c["train"] = rng.random() < 0.5
        return c
    c["quantized"] = rng.random() < 0.6
    c["stacked"] = rng.random() < 0.4
    c["I"] = 128 * _log(rng, 1, 20) if c["stacked"] else 16 * _log(rng, 2, 160) if c["quantized"] else _log(rng, 32, 2560)
    if op == "swiglu_bwd":
        most = 49152 * 2048 // (2 if c["dtype"] == "f32" or not c["quantized"] else 1)
        c["R"] = max(1, min(_log(rng, 1, 65536), most // c["I"]))
        return c
    c["E"] = _log(rng, 1, 384)
    c["k"] = rng.randint(1, min(8, c["E"]))
    c["T"] = _log(rng, 1, 16384)
    c["K"] = 16 * _log(rng, 8, 448)
    c["save"] = rng.random() < 0.3
    # no more weights and products than the listed prefill case
    per_row = 2 * c["I"] * c["K"]
    c["E"] = max(c["k"], min(c["E"], int(1.4e9 / per_row)))
    c["T"] = max(1, min(c["T"], int(1.4e12 / (per_row * c["k"])), int(3e8 / (c["I"] * c["k"]))))
    return c


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, cols, dtype):
    """Rows N(0, 1) with a spread of column magnitudes, as hidden states have."""
    spread = torch.exp(0.5 * _normal(gen, cols))
    return (_normal(gen, rows, cols) * spread).to(DTYPES[dtype])


def _groups(gen, case):
    """int64 [E + 1]: where each expert's rows start when random logits route the tokens, and the longest group."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = torch.topk(_normal(gen, T, E), k, dim=1).indices
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, int(counts.max())


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
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "case": dict(case), "dtype": dt}

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op.startswith("norm"):
        T, H = case["T"], case["H"]
        s["x"] = _activations(gen, T, H, case["dtype"])
        s["weight"] = (1.0 + 0.1 * _normal(gen, H)).to(dt)
        residual = case["residual"]
        if op == "norm_bwd":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = _normal(gen, T, H).to(dt)
            s["dres"] = _normal(gen, T, H).to(dt) if residual else None
            s["dx"], s["dw"], s["workspace"] = empty(T, H), empty(H, dtype=torch.float32), None
            return s
        s["res"] = _activations(gen, T, H, case["dtype"]) if residual else None
        s["sum"] = empty(T, H) if residual else None
        s["out"] = empty(T, H) if op == "norm" or case["keep"] else None
        s["rstd"] = empty(T, dtype=torch.float32) if case.get("train") else None
        if op == "norm_quantize":
            s["codes"] = empty(T, H, dtype=torch.uint8)
            s["scales"] = (empty(T, H // MX_BLOCK, dtype=torch.uint8) if case["fmt"] == "mx"
                           else empty(T, -(-H // BLOCK), dtype=torch.float32))
        return s
    inner = case["I"]
    s["stacked"] = case["stacked"]
    if op == "swiglu_bwd":
        R = case["R"]
        s["gate_up"] = (1.5 * _normal(gen, R, 2 * inner)).to(dt)
        s["dh"] = _normal(gen, R, inner).to(dt)
        width = 2 * inner
    else:
        K, E = case["K"], case["E"]
        s["offsets"], s["most"] = _groups(gen, case)
        s["grouped"], s["workspace"] = E > 1, None
        R = s["R"] = case["T"] * case["k"]
        x, xs = _quantize(_activations(gen, R, K, "f32")[None], 1)
        s["x"], s["xs"] = x[0], xs[0]
        s["weight"], s["ws"] = _weights(gen, E, 2 * inner, K)
        s["gate_up"] = empty(R, 2 * inner) if case["save"] else None
        width = inner
    if case["quantized"]:
        s["codes"], s["scales"] = empty(R, width, dtype=torch.uint8), empty(R, -(-width // BLOCK), dtype=torch.float32)
        s["out"] = None
    else:
        s["codes"], s["scales"], s["out"] = None, None, empty(R, width)
    return s


# ---------------------------------------------------------------- plain forms (fp32)

def _quantize(x, block_rows):
    """fp32 [B, rows, cols] -> E4M3 codes (uint8) of 448 x / amax and fp32 scales amax / 448 per block_rows x 128 block."""
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


def _quantize_mx(x):
    """fp32 [rows, cols] -> E4M3 codes and E8M0 scales 2^(floor(log2 amax) - 8) per 1x32 block, saturating at 448."""
    v = x.view(x.shape[0], -1, MX_BLOCK)
    exponent = (v.abs().amax(2).view(torch.int32) >> 23) - 8  # with fp32's bias of 127, which is E8M0's
    codes = torch.ldexp(v, 127 - exponent[..., None]).clamp(-MAX_E4M3, MAX_E4M3).to(torch.float8_e4m3fn)
    return codes.view(x.shape), exponent.to(torch.uint8).view(torch.float8_e8m0fnu)


def _codes(x):
    codes, scales = _quantize(x[None], 1)
    return {"codes": codes[0].view(torch.float8_e4m3fn), "scales": scales[0]}


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


def _product(s):
    """Rows of each expert times its weights, as one batched product over experts padded to the longest group."""
    x = _values(s["x"][None], s["xs"][None], 1)[0]
    w = _values(s["weight"], s["ws"], BLOCK)
    at = torch.arange(x.shape[0], device="cuda")
    e = torch.searchsorted(s["offsets"], at, right=True) - 1
    pos = at - s["offsets"][e]
    padded = torch.zeros(w.shape[0], s["most"], x.shape[1], dtype=torch.float32, device="cuda")
    padded[e, pos] = x
    return torch.bmm(padded, w.transpose(1, 2))[e, pos]


def _halves(v, stacked):
    """The gate's and the up projection's columns of [rows, 2 I]: one half after the other, or in turn."""
    inner = v.shape[1] // 2
    return (v[:, :inner], v[:, inner:]) if stacked else (v[:, 0::2], v[:, 1::2])


def _together(gate, up, stacked):
    return torch.cat([gate, up], 1) if stacked else torch.stack([gate, up], 2).view(gate.shape[0], -1)


def _plain_norm(s):
    v = s["x"].float()
    out = {}
    if s["res"] is not None:
        v = v + s["res"].float()
        out["sum"] = v.to(s["dtype"])
    rstd = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    y = v * rstd * s["weight"].float()
    if s["out"] is not None:
        out["y"] = y.to(s["dtype"])
    if s["rstd"] is not None:
        out["rstd"] = rstd[:, 0]
    if s["op"] == "norm_quantize":
        if s["case"]["fmt"] == "mx":
            out["codes"], out["scales"] = _quantize_mx(y)
        else:
            out.update(_codes(y))
    return out


def _plain_norm_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = s["x"].float() * rstd
    g = dy * s["weight"].float()
    dx = (g - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dtype"]), "dw": (dy * xhat).sum(0)}


def _plain_swiglu(s):
    v = _product(s)
    gate, up = _halves(v, s["stacked"])
    h = gate / (1.0 + torch.exp(-gate)) * up
    out = {"h": h.to(s["dtype"])} if s["out"] is not None else _codes(h)
    if s["gate_up"] is not None:
        out["gate_up"] = v.to(s["dtype"])
    return out


def _plain_swiglu_bwd(s):
    gate, up = _halves(s["gate_up"].float(), s["stacked"])
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    d = _together(dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig, s["stacked"])
    return {"d": d.to(s["dtype"])} if s["out"] is not None else _codes(d)


_PLAIN = {"norm": _plain_norm, "norm_quantize": _plain_norm, "norm_bwd": _plain_norm_bwd, "swiglu": _plain_swiglu,
          "swiglu_bwd": _plain_swiglu_bwd}


# ---------------------------------------------------------------- the package's operators

def _own_codes(s):
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def _own_norm(moe, s):
    x, w, out = s["x"], s["weight"], {}
    if s["op"] == "norm":
        moe.moe_rms_norm(x, w, EPS, s["out"], residual=s["res"], residual_out=s["sum"], rstd=s["rstd"])
    elif s["case"]["fmt"] == "mx":
        moe.moe_rms_norm_quantize_mx(x, w, EPS, moe.MOE_ACT_MXFP8, s["codes"], s["scales"], out=s["out"],
                                     residual=s["res"], residual_out=s["sum"])
        out = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"].view(torch.float8_e8m0fnu)}
    else:
        moe.moe_rms_norm_quantize_fp8_block(x, w, EPS, s["codes"], s["scales"], out=s["out"], residual=s["res"],
                                            residual_out=s["sum"])
        out = _own_codes(s)
    for name, key in (("sum", "sum"), ("y", "out"), ("rstd", "rstd")):
        if s[key] is not None:
            out[name] = s[key]
    return out


def _workspace(s, n):
    """Scratch memory, which a program allocates once for its sizes and keeps."""
    if s["workspace"] is None:
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import block_scaled_moe_topk_gb300 as moe
    op, c = s["op"], s["case"]
    if op in ("norm", "norm_quantize"):
        return _own_norm(moe, s)
    if op == "norm_bwd":
        space = _workspace(s, moe.moe_rms_norm_backward_workspace_bytes(c["T"], c["H"]))
        moe.moe_rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], s["dw"], space,
                                  d_residual=s["dres"])
        return {"dx": s["dx"], "dw": s["dw"]}
    layout = moe.MOE_GATE_UP_STACKED if s["stacked"] else moe.MOE_GATE_UP_INTERLEAVED
    if op == "swiglu":
        space = _workspace(s, moe.moe_gemm_fp8_block_workspace_bytes(s["R"], 2 * c["I"], c["K"], c["E"]))
        moe.moe_gemm_fp8_block_swiglu(s["x"], s["xs"], s["weight"], s["ws"], space, out=s["out"], codes=s["codes"],
                                      scales=s["scales"], gate_up=s["gate_up"], layout=layout,
                                      offsets=s["offsets"] if s["grouped"] else None)
        out = {"h": s["out"]} if s["out"] is not None else _own_codes(s)
        if s["gate_up"] is not None:
            out["gate_up"] = s["gate_up"]
        return out
    moe.moe_swiglu_backward(s["gate_up"], s["dh"], d_gate_up=s["out"], codes=s["codes"], scales=s["scales"],
                            layout=layout)
    return {"d": s["out"]} if s["out"] is not None else _own_codes(s)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- the least work, and 64-bit results

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if op.startswith("norm"):
        T, H = case["T"], case["H"]
        n = float(T) * H
        if op == "norm_bwd":
            return {"bytes": n * size * (4 if case["residual"] else 3) + 4.0 * T + (size + 4.0) * H, "flops": 10.0 * n}
        rows = 1 + (2 if case["residual"] else 0) + (1 if op == "norm" or case["keep"] else 0)
        least = n * size * rows + size * H + (4.0 * T if case.get("train") else 0.0)
        if op == "norm_quantize":
            least += n + (n / MX_BLOCK if case["fmt"] == "mx" else 4.0 * T * -(-H // BLOCK))
        return {"bytes": least, "flops": 5.0 * n}
    inner = case["I"]
    if op == "swiglu_bwd":
        n = float(case["R"]) * inner
        result = 2 * n + 4.0 * case["R"] * -(-2 * inner // BLOCK) if case["quantized"] else 2 * n * size
        return {"bytes": 3 * n * size + result, "flops": 12.0 * n}
    T, k, E, K = case["T"], case["k"], case["E"], case["K"]
    R = float(T * k)
    active = E * (1.0 - (1.0 - k / E) ** T)  # experts with a row, under even routing
    weights = 2.0 * inner * K + 4.0 * -(-2 * inner // BLOCK) * -(-K // BLOCK)
    result = inner + 4.0 * -(-inner // BLOCK) if case["quantized"] else size * inner
    if case["save"]:
        result += 2 * size * inner
    return {"bytes": active * weights + R * (K + 4.0 * -(-K // BLOCK) + result), "flops": 4.0 * R * inner * K}


def _e4m3_nearest(v):
    """The E4M3 value nearest to each fp64 value, at most 448 in magnitude; halfway between two codes, the even one."""
    table = torch.arange(127, device=v.device).to(torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)
    middle = (table[1:] + table[:-1]) / 2
    mag = v.abs()
    i = torch.searchsorted(middle, mag)
    tie = (mag == middle[i.clamp(max=125)]) & (i % 2 == 1)
    return torch.copysign(table[i + tie.long()], v)


def _exact_codes(v):
    """E4M3 values and 1x128 scales of fp64 rows, some rows at a time."""
    rows, cols = v.shape
    blocks = -(-cols // BLOCK)
    codes = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
    scales = torch.empty(rows, blocks, dtype=torch.float64, device="cuda")
    step = max(1, int(2e8 // cols))
    for r in range(0, rows, step):
        part = torch.zeros(min(step, rows - r), blocks * BLOCK, dtype=torch.float64, device="cuda")
        part[:, :cols] = v[r:r + step]
        part = part.view(part.shape[0], blocks, BLOCK)
        amax = part.abs().amax(2, keepdim=True)
        tiny = amax < TINY
        q = torch.where(tiny, 0.0, part * MAX_E4M3 / torch.where(tiny, 1.0, amax))
        codes[r:r + step] = _e4m3_nearest(q).view(part.shape[0], -1)[:, :cols]
        scales[r:r + step] = torch.where(tiny, 0.0, amax / MAX_E4M3)[..., 0]
    return {"codes": codes, "scales": scales}


def _exact_norm(s, case):
    f64 = torch.float64
    v = s["x"].to(f64)
    out = {}
    if s["res"] is not None:
        v = v + s["res"].to(f64)
        out["sum"] = v
    rms = (v.square().sum(1, keepdim=True) / case["H"] + EPS).sqrt()
    y = v / rms * s["weight"].to(f64)
    if s["out"] is not None:
        out["y"] = y
    if s["rstd"] is not None:
        out["rstd"] = 1.0 / rms[:, 0]
    if case["op"] == "norm":
        return out
    if case["fmt"] == "fp8":
        out.update(_exact_codes(y))
        return out
    b = y.view(case["T"], -1, MX_BLOCK)
    scale = torch.ldexp(torch.ones((), dtype=f64, device="cuda"), torch.frexp(b.abs().amax(2)).exponent - 9)
    out["codes"] = _e4m3_nearest((b / scale[..., None]).clamp(-MAX_E4M3, MAX_E4M3)).view(y.shape)
    out["scales"] = scale
    return out


def _exact_gated(v, stacked):
    g, u = (v[:, :v.shape[1] // 2], v[:, v.shape[1] // 2:]) if stacked else (v[:, ::2], v[:, 1::2])
    return g, u, torch.sigmoid(g)


def exact(case, seed):
    op, f64 = case["op"], torch.float64
    if op == "swiglu" and 4.0 * case["T"] * case["k"] * case["I"] * case["K"] > 1e13:
        return None
    s = prepare(case, seed)
    if op in ("norm", "norm_quantize"):
        return _exact_norm(s, case)
    if op == "norm_bwd":
        # the rows' 1/rms is an input: fp32 as the forward pass keeps it
        x, dy, w, r = s["x"].to(f64), s["dy"].to(f64), s["weight"].to(f64), s["rstd"].to(f64)[:, None]
        dot = (dy * w * x).sum(1, keepdim=True)
        dx = r * dy * w - r ** 3 / case["H"] * dot * x
        return {"dx": dx if s["dres"] is None else dx + s["dres"].to(f64), "dw": (dy * x * r).sum(0)}
    if op == "swiglu_bwd":
        g, u, sig = _exact_gated(s["gate_up"].to(f64), s["stacked"])
        dh = s["dh"].to(f64)
        d = torch.empty(case["R"], 2 * case["I"], dtype=f64, device="cuda")
        dg, du, _ = _exact_gated(d, s["stacked"])
        dg.copy_(dh * u * (sig + g * sig * (1.0 - sig)))
        du.copy_(dh * g * sig)
        return {"d": d} if s["out"] is not None else _exact_codes(d)
    v = torch.empty(s["R"], 2 * case["I"], dtype=f64, device="cuda")
    off = s["offsets"].tolist()
    n, c = (torch.arange(d, device="cuda") // BLOCK for d in (2 * case["I"], case["K"]))
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        w = s["weight"][e].view(torch.float8_e4m3fn).to(f64) * s["ws"][e].to(f64)[n][:, c]
        v[a:b] = s["x"][a:b].view(torch.float8_e4m3fn).to(f64) * s["xs"][a:b].to(f64)[:, c] @ w.t()
    g, u, sig = _exact_gated(v, s["stacked"])
    h = g * sig * u
    out = {"h": h} if s["out"] is not None else _exact_codes(h)
    if s["gate_up"] is not None:
        out["gate_up"] = v
    return out
