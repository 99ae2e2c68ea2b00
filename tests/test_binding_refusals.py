"""What the bindings of the single operators refuse, check by check, without a GPU.

The tensors say that they are on a GPU (a subclass of torch.Tensor over host memory), so that a call gets as far as
the check that is meant, and the message says which one it was.  Every call is refused before the library sees it: a
binding that lets one through asks for the current device, and that fails the test.
"""
import pytest
import torch

import block_scaled_moe_topk_gb300 as moe


class Fake(torch.Tensor):
    """A host tensor that claims to be on cuda:0, or on cuda:1 where ``other`` is set."""
    other = False

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return 1 if self.other else 0


def fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Fake)


def elsewhere(t):
    t.other = True
    return t


def host(t):
    return torch.zeros(t.shape, dtype=t.dtype)


class Accepted(Exception):
    pass


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    def current():
        raise Accepted
    monkeypatch.setattr(moe, "_current_device", current)


I32, I64, U8, F32, BF16 = torch.int32, torch.int64, torch.uint8, torch.float32, torch.bfloat16


def fakes(**spec):
    return {k: (fake(*v[0], dtype=v[1]) if isinstance(v, tuple) else v) for k, v in spec.items()}


CALLS = {
    "permute": (moe.moe_permute, lambda: fakes(x=((4, 64), BF16), inv=((4, 2), I32), rows=((9, 64), BF16))),
    "permute_backward": (moe.moe_permute_backward,
                         lambda: fakes(d_rows=((9, 64), BF16), inv=((4, 2), I32), d_x=((4, 64), BF16))),
    "unpermute": (moe.moe_unpermute, lambda: fakes(rows=((9, 64), BF16), inv=((4, 2), I32), topk_w=((4, 2), F32),
                                                   out=((4, 64), BF16))),
    "unpermute_backward": (moe.moe_unpermute_backward,
                           lambda: fakes(d_out=((4, 64), BF16), rows=((9, 64), BF16), inv=((4, 2), I32),
                                         topk_w=((4, 2), F32), d_rows=((9, 64), BF16), d_topk_w=((4, 2), F32))),
    "route_backward": (moe.moe_topk_route_backward,
                       lambda: fakes(topk_ids=((4, 2), I32), topk_w=((4, 2), F32), d_topk_w=((4, 2), F32),
                                     d_logits=((4, 8), F32))),
    "quantize": (moe.moe_quantize_fp8_block,
                 lambda: fakes(x=((200, 300), BF16), codes=((200, 300), U8), scales=((200, 3), F32))),
    "quantize_weights": (lambda **a: moe.moe_quantize_fp8_block(block_rows=128, **a),
                         lambda: fakes(x=((200, 300), BF16), codes=((200, 300), U8), scales=((2, 3), F32))),
    "permute_quantize": (moe.moe_permute_quantize_fp8_block,
                         lambda: fakes(x=((4, 300), BF16), inv=((4, 2), I32), codes=((9, 300), U8),
                                       scales=((9, 3), F32))),
    "gemm": (moe.moe_gemm_fp8_block,
             lambda: fakes(x=((7, 144), U8), x_scale=((7, 2), F32), w=((3, 208, 144), U8), w_scale=((3, 2, 2), F32),
                           out=((7, 208), BF16), workspace=((256,), U8), offsets=((4,), I64))),
    "dgrad": (moe.moe_gemm_fp8_block_dgrad,
              lambda: fakes(dy=((7, 208), U8), dy_scale=((7, 2), F32), w=((3, 208, 144), U8),
                            w_scale=((3, 2, 2), F32), dx=((7, 144), BF16), workspace=((256,), U8),
                            offsets=((4,), I64))),
}

# What a message calls an argument, where it is not by its name.
NAMES = {("gemm", "x"): "the codes", ("gemm", "x_scale"): "the codes' scales", ("gemm", "out"): "the output",
         ("dgrad", "dy"): "the codes", ("dgrad", "dy_scale"): "the codes' scales", ("dgrad", "dx"): "the output",
         ("gemm", "workspace"): "the workspace", ("dgrad", "workspace"): "the workspace"}
# Matrices with a row stride of their own; the other tensors are contiguous.
STRIDED = {"permute": ("x", "rows"), "permute_backward": ("d_rows", "d_x"), "unpermute": ("rows", "out"),
           "unpermute_backward": ("d_out", "rows", "d_rows"), "quantize": ("x",), "quantize_weights": ("x",),
           "permute_quantize": ("x",)}
# Tensors whose size of dimension d no other argument fixes, so that a wrong one shows at another tensor.
FREE = {("permute", "x", 0): "x", ("permute", "x", 1): "rows", ("permute", "inv", 0): "x", ("permute", "inv", 1): None,
        ("permute", "rows", 0): None, ("permute_backward", "d_rows", 0): None, ("permute_backward", "d_rows", 1): "d_x",
        ("permute_backward", "inv", 0): "d_x", ("permute_backward", "inv", 1): None,
        ("unpermute", "rows", 0): None, ("unpermute", "rows", 1): "out", ("unpermute", "inv", 0): "out",
        ("unpermute", "inv", 1): "topk_w", ("unpermute_backward", "d_out", 1): "d_rows",
        ("unpermute_backward", "inv", 0): "d_out", ("unpermute_backward", "inv", 1): "topk_w",
        ("unpermute_backward", "d_rows", 0): "rows", ("route_backward", "topk_ids", 0): "topk_w",
        ("route_backward", "topk_ids", 1): "topk_w", ("route_backward", "d_logits", 1): None,
        ("quantize", "x", 0): "codes", ("quantize", "x", 1): "codes", ("quantize_weights", "x", 0): "codes",
        ("quantize_weights", "x", 1): "codes", ("permute_quantize", "x", 1): "codes",
        ("permute_quantize", "inv", 0): "x", ("permute_quantize", "inv", 1): None,
        ("permute_quantize", "codes", 0): "scales",
        ("gemm", "x", 0): "x_scale", ("gemm", "w", 0): "w_scale", ("gemm", "w", 1): "out", ("gemm", "w", 2): "x",
        ("dgrad", "dy", 0): "dy_scale", ("dgrad", "w", 0): "w_scale", ("dgrad", "w", 1): "dy", ("dgrad", "w", 2): "dx"}
ARGS = [(c, a) for c, (_, make) in CALLS.items() for a in make()]
DIMS = [(c, a, d) for c, (_, make) in CALLS.items() for a, t in make().items() if a != "workspace"
        for d in range(t.dim())]


END = ": MOE_ERR_INVALID_ARG$"


def refused(call, args, match):
    with pytest.raises(moe.MoeError, match=match) as ei:
        CALLS[call][0](**args)
    assert ei.value.status == 1


def name_of(call, arg):
    return NAMES.get((call, arg), arg)


@pytest.mark.parametrize("call", list(CALLS))
def test_right_arguments_pass(call):
    with pytest.raises(Accepted):
        CALLS[call][0](**CALLS[call][1]())


@pytest.mark.parametrize("call,arg", ARGS)
def test_host_tensor(call, arg):
    args = CALLS[call][1]()
    args[arg] = host(args[arg])
    refused(call, args, f"{name_of(call, arg)} must be on the GPU{END}")


@pytest.mark.parametrize("call,arg", ARGS)
def test_tensor_on_another_gpu(call, arg):
    args = CALLS[call][1]()
    elsewhere(args[arg])
    refused(call, args, r" is on cuda:\d, expected cuda:\d" + END)


def test_another_current_device(monkeypatch):
    monkeypatch.setattr(moe, "_current_device", lambda: 1)
    for fn, make in CALLS.values():
        with pytest.raises(moe.MoeError, match="the tensors are on cuda:0, the current device is cuda:1" + END) as ei:
            fn(**make())
        assert ei.value.status == 1


@pytest.mark.parametrize("call,arg", [(c, a) for c, a in ARGS if a != "workspace"])
def test_wrong_type(call, arg):
    args = CALLS[call][1]()
    args[arg] = fake(*args[arg].shape, dtype=torch.float64)
    refused(call, args, f"{name_of(call, arg)} |unsupported type torch.float64{END}")


@pytest.mark.parametrize("call,arg,dim", DIMS)
def test_wrong_size(call, arg, dim):
    args = CALLS[call][1]()
    shape = list(args[arg].shape)
    shape[dim] += 1
    shown = FREE.get((call, arg, dim), arg)
    args[arg] = fake(*shape, dtype=args[arg].dtype)
    if shown is None:  # a size of its own: any is right
        with pytest.raises(Accepted):
            CALLS[call][0](**args)
    else:
        refused(call, args, f": {name_of(call, shown)} has shape ")


@pytest.mark.parametrize("call,arg", [(c, a) for c, a in ARGS if a != "workspace"])
def test_wrong_rank(call, arg):
    args = CALLS[call][1]()
    for shape in ((1,) + tuple(args[arg].shape), (args[arg].numel(),), ()):
        if len(shape) == args[arg].dim():
            continue
        bad = dict(args)
        bad[arg] = fake(*shape, dtype=args[arg].dtype)
        refused(call, bad, "ha(s|ve) shape|must be a matrix" + END)


@pytest.mark.parametrize("call,arg", [(c, a) for c, a in ARGS if a != "workspace"])
def test_wrong_strides(call, arg):
    """Transposed storage: no unit column stride; tables and codes have to be contiguous as a whole."""
    args = CALLS[call][1]()
    t = args[arg]
    strided = arg in STRIDED.get(call, ())
    if strided:
        args[arg] = fake(*reversed(t.shape), dtype=t.dtype).t()
        refused(call, args, f"{name_of(call, arg)} must have unit column stride{END}")
        wide = torch.zeros(t.shape[0], t.shape[1] + 5, dtype=t.dtype).as_subclass(Fake)
        args[arg] = wide[:, :t.shape[1]]  # padded rows are right
        with pytest.raises(Accepted):
            CALLS[call][0](**args)
    else:
        args[arg] = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2].as_subclass(Fake)
        refused(call, args, f"{name_of(call, arg)} must be contiguous{END}")


def test_optional_arguments():
    fn, make = CALLS["unpermute_backward"]
    for drop in ({"d_rows": None}, {"d_topk_w": None}, {"d_topk_w": None, "rows": None}):
        with pytest.raises(Accepted):
            fn(**{**make(), **drop})
    refused("unpermute_backward", {**make(), "rows": None}, "d_topk_w needs rows" + END)
    with pytest.raises(moe.MoeError, match="block_rows must be 1 or 128" + END):
        moe.moe_quantize_fp8_block(**CALLS["quantize"][1](), block_rows=64)
    for call in ("gemm", "dgrad"):
        with pytest.raises(Accepted):
            CALLS[call][0](**{**CALLS[call][1](), "offsets": None})


@pytest.mark.parametrize("call", list(CALLS))
def test_all_on_the_host(call):
    refused(call, {k: host(t) for k, t in CALLS[call][1]().items()}, f"must be on the GPU{END}")


@pytest.mark.parametrize("call", list(STRIDED))
def test_wrong_type_throughout(call):
    args = CALLS[call][1]()
    for name in STRIDED[call]:
        args[name] = fake(*args[name].shape, dtype=torch.float64)
    refused(call, args, f"{STRIDED[call][0]} has the unsupported type torch.float64{END}")
    if call != "permute":  # bytes can be moved, not summed or quantised
        for name in STRIDED[call]:
            args[name] = fake(*args[name].shape, dtype=U8)
        refused(call, args, f"{STRIDED[call][0]} has the unsupported type torch.uint8{END}")


@pytest.mark.parametrize("call,names", [("unpermute", ("inv", "topk_w")), ("unpermute_backward", ("inv", "topk_w", "d_topk_w")),
                                        ("route_backward", ("topk_ids", "topk_w", "d_topk_w"))])
def test_wrong_rank_throughout(call, names):
    for shape in ((4,), (4, 2, 1)):
        args = CALLS[call][1]()
        for name in names:
            args[name] = fake(*shape, dtype=args[name].dtype)
        refused(call, args, f": {names[0]} has shape ")


def test_missing_weights():
    for call in ("unpermute", "unpermute_backward"):
        refused(call, {**CALLS[call][1](), "topk_w": None}, "topk_w must be torch.float32" + END)
