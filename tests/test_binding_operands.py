"""CPU tests of how the bindings of qlinear_block_norm and qlinear_adapters take
what is no tensor: a TypeError that names the operand, as the other entry
points give, and None where the C call accepts NULL. The library and torch's
device side are the stand-ins of test_binding_streams."""
import numpy as np
import pytest

from group_wise_affine_qlinear_amd import qlinear as ql
from test_binding_streams import Tensor, taken, torch  # noqa: F401

M, D, N, K, RANK, ADAPTERS = 8, 64, 96, 128, 16, 2
NO_TENSORS = [[1.0, 2.0], 3.0, np.zeros((M, D), dtype=np.float32), "residual"]


def block_norm(**kw):
    f32, bf16 = torch.float32, torch.bfloat16
    args = dict(y=Tensor((M, D), f32), post_weight=Tensor((D,), f32), post_bias=Tensor((D,), f32), gate=None,
                residual_out=Tensor((M, D), bf16), pre_weight=Tensor((D,), f32), pre_bias=Tensor((D,), f32),
                h=Tensor((M, D), bf16), x16=Tensor((M, D), torch.float16), rowscale=Tensor((M,), f32),
                row_sample=Tensor((M,), torch.int32), samples=3)
    args.update(kw)
    ql.qlinear_block_norm(args.pop("residual", Tensor((M, D), bf16)), M, D, **args)


def adapters(n=ADAPTERS, k=K, **kw):
    f32, bf16 = torch.float32, torch.bfloat16
    args = dict(x=Tensor((M, k), bf16), a=Tensor((n, RANK, k), bf16), b=Tensor((n, N, RANK), bf16),
                row_adapter=Tensor((M,), torch.int32), out=Tensor((M, N), f32), y=Tensor((M, N), f32),
                ranks=Tensor((n,), torch.int32), scaling=Tensor((n,), f32), residual=Tensor((M, N), f32),
                gate=Tensor((M, N), f32), gate_rows=1, epilogue=ql.QL_EPI_GATE_RESIDUAL, workspace=Tensor((4096,), torch.uint8))
    args.update(kw)
    ql.qlinear_adapters(args.pop("x"), args.pop("a"), args.pop("b"), args.pop("row_adapter"), M, N, k, args.pop("out"), **args)


@pytest.mark.parametrize("name", ["residual", "y", "post_weight", "post_bias", "gate", "residual_out", "pre_weight", "pre_bias",
                                  "scale", "shift", "h", "x16", "rowscale", "row_sample"])
def test_block_norm(taken, name):  # noqa: F811
    block_norm()
    for bad in NO_TENSORS:
        with pytest.raises(TypeError):
            block_norm(**{name: bad})
        if name in ("gate", "scale", "shift"):
            with pytest.raises(TypeError):
                block_norm(**{name: bad, "samples": None})


@pytest.mark.parametrize("name", ["x", "a", "b", "row_adapter", "out", "y", "ranks", "scaling", "residual", "gate", "workspace"])
def test_adapters(taken, name):  # noqa: F811
    adapters()
    for bad in NO_TENSORS:
        # a text as the workspace names where to take it from
        with pytest.raises(ValueError if name == "workspace" and isinstance(bad, str) else TypeError):
            adapters(**{name: bad})


def test_adapters_without_what_is_not_read(taken):  # noqa: F811
    adapters(n=0, x=None)
    adapters(n=0, x=None, b=None)
    adapters(k=0, x=None)
    for kw in (dict(x=None), dict(b=None), dict(k=0, b=None), dict(a=None), dict(n=0, a=None), dict(row_adapter=None)):
        with pytest.raises(TypeError):
            adapters(**kw)
