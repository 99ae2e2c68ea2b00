"""What the norm's and the gated block's calls refuse, without a GPU: the bindings check by check (tensors that only say
that they are on a GPU), and the C entry points' own checks, which come before any launch."""
import ctypes

import pytest
import torch

import block_scaled_moe_topk_gb300 as moe
from test_binding_refusals import Accepted, BF16, END, F32, I64, U8, elsewhere, fake, fakes, host

EPS = 1e-6


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    def current():
        raise Accepted
    monkeypatch.setattr(moe, "_current_device", current)


def norm(**a):
    moe.moe_rms_norm(eps=EPS, **a)


def norm_fp8(**a):
    moe.moe_rms_norm_quantize_fp8_block(eps=EPS, **a)


def norm_mx(**a):
    moe.moe_rms_norm_quantize_mx(eps=EPS, fmt=moe.MOE_ACT_MXFP8, **a)


def norm_mx4(**a):
    moe.moe_rms_norm_quantize_mx(eps=EPS, fmt=moe.MOE_ACT_MXFP4, **a)


def rows_of(*names):
    return {n: ((6, 288), BF16) for n in names}


CALLS = {
    "norm": (norm, lambda: fakes(**rows_of("x"), weight=((288,), BF16), **rows_of("out", "residual", "residual_out"),
                                 rstd=((6,), F32))),
    "norm_fp8": (norm_fp8, lambda: fakes(**rows_of("x"), weight=((288,), F32), codes=((6, 288), U8),
                                         scales=((6, 3), F32), **rows_of("out", "residual", "residual_out"),
                                         rstd=((6,), F32))),
    "norm_mx": (norm_mx, lambda: fakes(**rows_of("x"), weight=((288,), BF16), codes=((6, 288), U8), scales=((6, 9), U8),
                                       **rows_of("out", "residual", "residual_out"))),
    "norm_mx4": (norm_mx4, lambda: fakes(**rows_of("x"), weight=((288,), BF16), codes=((6, 144), U8),
                                         scales=((6, 9), U8))),
    "norm_backward": (moe.moe_rms_norm_backward,
                      lambda: fakes(**rows_of("dy", "x"), weight=((288,), BF16), rstd=((6,), F32), **rows_of("dx"),
                                    d_weight=((288,), F32), workspace=((6 * 288 * 4,), U8), **rows_of("d_residual"))),
    "swiglu_backward": (moe.moe_swiglu_backward,
                        lambda: fakes(gate_up=((6, 288), BF16), d_h=((6, 144), BF16), d_gate_up=((6, 288), BF16),
                                      codes=((6, 288), U8), scales=((6, 3), F32))),
    "gemm_swiglu": (moe.moe_gemm_fp8_block_swiglu,
                    lambda: fakes(x=((7, 144), U8), x_scale=((7, 2), F32), w=((3, 416, 144), U8),
                                  w_scale=((3, 4, 2), F32), workspace=((256,), U8), out=((7, 208), BF16),
                                  codes=((7, 208), U8), scales=((7, 2), F32), gate_up=((7, 416), BF16),
                                  offsets=((4,), I64))),
}
STRIDED = {"x", "out", "residual", "residual_out", "dy", "dx", "d_residual", "gate_up", "d_h", "d_gate_up"}
ARGS = [(c, a) for c, (_, make) in CALLS.items() for a in make()]
TYPED = [(c, a) for c, a in ARGS if a != "workspace"]


def refused(call, args, match):
    with pytest.raises(moe.MoeError, match=match) as ei:
        CALLS[call][0](**args)
    assert ei.value.status == 1


@pytest.mark.parametrize("call", list(CALLS))
def test_right_arguments_pass(call):
    with pytest.raises(Accepted):
        CALLS[call][0](**CALLS[call][1]())


@pytest.mark.parametrize("call,arg", ARGS)
def test_host_tensor_and_another_gpu(call, arg):
    args = CALLS[call][1]()
    refused(call, {**args, arg: host(args[arg])}, "must be on the GPU" + END)
    elsewhere(args[arg])
    refused(call, args, r" is on cuda:\d, expected cuda:\d" + END)


def test_another_current_device(monkeypatch):
    monkeypatch.setattr(moe, "_current_device", lambda: 1)
    for fn, make in CALLS.values():
        with pytest.raises(moe.MoeError, match="the tensors are on cuda:0, the current device is cuda:1" + END):
            fn(**make())


@pytest.mark.parametrize("call,arg", TYPED)
def test_wrong_type(call, arg):
    args = CALLS[call][1]()
    refused(call, {**args, arg: fake(*args[arg].shape, dtype=torch.float64)},
            f"{arg} |has the unsupported type torch.|must be (bf16|torch)")


@pytest.mark.parametrize("call,arg,dim", [(c, a, d) for c, a in TYPED for d in range(CALLS[c][1]()[a].dim())])
def test_wrong_size(call, arg, dim):
    args = CALLS[call][1]()
    shape = list(args[arg].shape)
    shape[dim] += 256  # more than a scale block
    refused(call, {**args, arg: fake(*shape, dtype=args[arg].dtype)}, " has shape ")


@pytest.mark.parametrize("call,arg", TYPED)
def test_wrong_rank(call, arg):
    args = CALLS[call][1]()
    for shape in ((1,) + tuple(args[arg].shape), (args[arg].numel(),), ()):
        if len(shape) != args[arg].dim():
            refused(call, {**args, arg: fake(*shape, dtype=args[arg].dtype)}, " has shape | must be a matrix")


@pytest.mark.parametrize("call,arg", TYPED)
def test_wrong_strides(call, arg):
    args = CALLS[call][1]()
    t = args[arg]
    if arg not in STRIDED or call == "gemm_swiglu":
        apart = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2].as_subclass(type(t))
        refused(call, {**args, arg: apart}, f"{arg} must be contiguous" + END)
        return
    refused(call, {**args, arg: fake(*reversed(t.shape), dtype=t.dtype).t()}, f"{arg} must have unit column stride" + END)
    wide = torch.zeros(t.shape[0], t.shape[1] + 5, dtype=t.dtype).as_subclass(type(t))[:, :t.shape[1]]
    with pytest.raises(Accepted):
        CALLS[call][0](**{**args, arg: wide})


OPTIONAL = {"norm": ("residual", "residual_out", "rstd"), "norm_fp8": ("out", "residual", "residual_out", "rstd"),
            "norm_mx": ("out", "residual", "residual_out"), "norm_mx4": (), "norm_backward": ("d_weight", "d_residual"),
            "swiglu_backward": ("d_gate_up",), "gemm_swiglu": ("out", "gate_up", "offsets")}
NEEDED = ("x", "d_h", "w", "x_scale", "w_scale", "workspace")  # left out they raise as any missing argument does


@pytest.mark.parametrize("call,arg", [(c, a) for c, a in ARGS if a not in NEEDED or (c, a) == ("norm_backward", "workspace")])
def test_left_out(call, arg):
    args = {**CALLS[call][1](), arg: None}
    if arg in OPTIONAL[call]:
        with pytest.raises(Accepted):
            CALLS[call][0](**args)
    else:
        refused(call, args, "need|must be a matrix|come together")


def test_values():
    args = CALLS["swiglu_backward"][1]()
    refused("swiglu_backward", {**args, "layout": 2}, "unknown layout" + END)
    refused("swiglu_backward", {**args, "d_gate_up": None, "codes": None, "scales": None}, "d_gate_up or codes are needed" + END)
    gated = CALLS["gemm_swiglu"][1]()
    refused("gemm_swiglu", {**gated, "layout": 2}, "unknown layout" + END)
    refused("gemm_swiglu", {**gated, "out": None, "codes": None, "scales": None}, "out or codes are needed" + END)
    refused("gemm_swiglu", {**gated, "w": fake(3, 415, 144, dtype=U8)}, "w has 415 rows")
    with pytest.raises(Accepted):
        moe.moe_gemm_fp8_block_swiglu(**{**gated, "codes": None, "scales": None})
    with pytest.raises(Accepted):
        moe.moe_gemm_fp8_block_swiglu(**{**gated, "out": None, "gate_up": None})
    odd = fakes(x=((6, 100), BF16), weight=((100,), BF16), codes=((6, 100), U8), scales=((6, 3), U8))
    refused("norm_mx", odd, "multiple of 32" + END)
    with pytest.raises(moe.MoeError, match="fmt must be"):
        moe.moe_rms_norm_quantize_mx(eps=EPS, fmt=7, **CALLS["norm_mx4"][1]())


# ---------------------------------------------------------------- the C entry points
A, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)  # never followed: every call below is refused


def norm_c(x=A, xs=64, r=None, rs=0, dt=0, w=A, wt=0, eps=EPS, T=4, H=64, out=A, os=64, ro=None, ros=0, rstd=None):
    return moe.lib().moe_rms_norm(x, xs, r, rs, dt, w, wt, eps, T, H, out, os, ro, ros, rstd, None)


@pytest.mark.parametrize("status,args", [
    (1, dict(x=None)), (1, dict(xs=63)), (1, dict(dt=3)), (1, dict(dt=9)), (1, dict(w=None)), (1, dict(wt=1)),
    (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (1, dict(T=-1)), (1, dict(H=0)), (1, dict(out=None)),
    (1, dict(os=10)), (1, dict(r=A, rs=1)), (1, dict(ro=A, ros=1)), (2, dict(H=32769, xs=40000, os=40000)),
    (2, dict(T=(1 << 30) + 1)), (7, dict(x=ODD)), (7, dict(out=ODD)), (7, dict(w=ODD)), (7, dict(rstd=ODD)),
    (7, dict(r=ODD, rs=64)), (7, dict(ro=ODD, ros=64))])
def test_norm_refuses(status, args):
    assert norm_c(**args) == status


def test_quantised_norm_refuses():
    fp8, mx = moe.lib().moe_rms_norm_quantize_fp8_block, moe.lib().moe_rms_norm_quantize_mx
    rest = (None, 0, None, 0, None, None)
    head = (A, 64, None, 0, 0, A, 0, EPS, 4, 64)
    assert fp8(*head, None, A, *rest) == 1 and fp8(*head, A, None, *rest) == 1 and fp8(*head, A, ODD, *rest) == 7
    assert mx(*head, 5, A, A, *rest) == 1 and mx(*head, 0, None, A, *rest) == 1 and mx(*head, 0, A, None, *rest) == 1
    assert mx(A, 64, None, 0, 0, A, 0, EPS, 4, 48, 0, A, A, *rest) == 2


def backward_c(dy=A, dys=64, x=A, xs=64, r=None, rs=0, dt=0, w=A, wt=0, rstd=A, T=4, H=64, dx=A, dxs=64, dw=A, space=A,
               size=None):
    size = moe.moe_rms_norm_backward_workspace_bytes(T, H) if size is None else size
    return moe.lib().moe_rms_norm_backward(dy, dys, x, xs, r, rs, dt, w, wt, rstd, T, H, dx, dxs, dw, space, size, None)


@pytest.mark.parametrize("status,args", [
    (1, dict(dy=None)), (1, dict(x=None)), (1, dict(dx=None)), (1, dict(rstd=None)), (1, dict(w=None)),
    (1, dict(space=None)), (1, dict(dt=3)), (1, dict(wt=1)), (1, dict(T=-1)), (1, dict(H=-3)), (1, dict(dys=63)),
    (1, dict(xs=63)), (1, dict(dxs=63)), (1, dict(r=A, rs=63)), (2, dict(H=32769)), (4, dict(size=4 * 64 * 4 - 1)),
    (7, dict(dy=ODD)), (7, dict(x=ODD)), (7, dict(dx=ODD)), (7, dict(r=ODD, rs=64)), (7, dict(w=ODD)),
    (7, dict(rstd=ODD)), (7, dict(dw=ODD)), (7, dict(space=ctypes.c_void_p((1 << 20) + 128)))])
def test_norm_backward_refuses(status, args):
    assert backward_c(**args) == status


def test_norm_backward_workspace():
    f = moe.moe_rms_norm_backward_workspace_bytes
    assert f(1, 100) == 400 and f(0, 100) == 400 and f(1 << 20, 7168) == 304 * 7168 * 4
    assert f(1 << 20, 100) == 456 * 100 * 4
    assert f(-1, 100) == 0 and f(5, 0) == 0 and f(5, 40000) == 0


def swiglu_c(gu=A, gus=256, dh=A, dhs=128, dt=0, layout=0, R=4, I=128, d=A, ds=256, codes=A, scales=A):
    return moe.lib().moe_swiglu_backward(gu, gus, dh, dhs, dt, layout, R, I, d, ds, codes, scales, None)


@pytest.mark.parametrize("status,args", [
    (1, dict(gu=None)), (1, dict(dh=None)), (1, dict(gus=255)), (1, dict(dhs=127)), (1, dict(ds=255)), (1, dict(dt=3)),
    (1, dict(layout=2)), (1, dict(layout=-1)), (1, dict(R=-1)), (1, dict(I=0)), (1, dict(d=None, codes=None, scales=None)),
    (1, dict(scales=None)), (1, dict(codes=None)), (2, dict(I=32769, gus=70000, dhs=70000, ds=70000)),
    (2, dict(layout=1, I=64)), (2, dict(R=(1 << 30) + 1)), (7, dict(gu=ODD)), (7, dict(dh=ODD)), (7, dict(d=ODD)),
    (7, dict(scales=ODD))])
def test_swiglu_backward_refuses(status, args):
    assert swiglu_c(**args) == status


def gated_c(x=A, xs=A, w=A, ws=A, layout=0, off=A, M=5, I=128, K=256, E=2, out=A, gu=A, dt=0, codes=A, scales=A, space=A,
            size=256):
    return moe.lib().moe_gemm_fp8_block_swiglu(x, xs, w, ws, layout, off, M, I, K, E, out, gu, dt, codes, scales, space,
                                               size, None)


A8 = ctypes.c_void_p((1 << 20) + 8)


@pytest.mark.parametrize("status,args", [
    (1, dict(x=None)), (1, dict(xs=None)), (1, dict(w=None)), (1, dict(ws=None)), (1, dict(off=None)),
    (1, dict(out=None, codes=None, scales=None)), (1, dict(codes=None)), (1, dict(scales=None)), (1, dict(space=None)),
    (1, dict(layout=2)), (1, dict(dt=3)), (1, dict(M=-1)), (1, dict(I=0)), (1, dict(K=0)), (1, dict(E=0)),
    (2, dict(K=264)), (2, dict(E=1025)), (2, dict(I=40000)), (2, dict(I=136)), (2, dict(layout=1, I=192)),
    (2, dict(M=(1 << 30) + 1)), (4, dict(size=255)), (7, dict(x=A8)), (7, dict(w=A8)), (7, dict(codes=A8)),
    (7, dict(out=ODD)), (7, dict(gu=ODD)), (7, dict(scales=ODD)), (7, dict(xs=ODD)), (7, dict(ws=ODD)),
    (7, dict(off=ODD)), (7, dict(space=ctypes.c_void_p((1 << 20) + 128)))])
def test_gated_product_refuses(status, args):
    assert gated_c(**args) == status
