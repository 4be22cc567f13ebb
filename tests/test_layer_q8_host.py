"""Argument checks of the layer on quantised activations in Python (no GPU: every call is refused
before a pointer is read)."""
import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def call(ops, **change):
    cfg = ops.make_config(64, 256, 8, 2, 128, wdtype=ops.W8A8_FP8)
    a = {"x": torch.zeros(4, 256, dtype=BF16), "xq": torch.zeros(4, 256, dtype=torch.uint8), "xq_scale": torch.zeros(4, 2),
         "out": torch.zeros(4, 256, dtype=BF16), "workspace": torch.zeros(256, dtype=torch.uint8),
         "dev_status": torch.zeros(1, dtype=torch.int32)}
    a.update(change)
    ops.layer_q8(cfg, a["x"], a["xq"], a["xq_scale"], ops.Weights(), a["out"], a["workspace"], a["dev_status"])


@pytest.mark.parametrize("name,other", [
    ("x", torch.zeros(4, 256)), ("x", torch.zeros(4, 256, dtype=torch.uint8)),
    ("xq", torch.zeros(4, 256, dtype=BF16)), ("xq", torch.zeros(4, 256, dtype=torch.int32)),
    ("xq_scale", torch.zeros(4, 2, dtype=torch.float64)), ("xq_scale", torch.zeros(4, 2, dtype=BF16)),
    ("out", torch.zeros(4, 256)), ("out", torch.zeros(4, 256, dtype=torch.float16)),
    ("workspace", torch.zeros(256)), ("dev_status", torch.zeros(1, dtype=torch.int64))])
def test_layer_q8_refuses_other_types(ops, name, other):
    with pytest.raises(ValueError, match=f"^{name}: .*expected"):
        call(ops, **{name: other})


@pytest.mark.parametrize("name,other", [
    ("x", torch.zeros(256, 4, dtype=BF16).t()), ("xq", torch.zeros(256, 4, dtype=torch.uint8).t()),
    ("xq", torch.zeros(4, 512, dtype=torch.float8_e4m3fn)[:, ::2]), ("xq_scale", torch.zeros(2, 4).t()),
    ("out", torch.zeros(4, 512, dtype=BF16)[:, :256]), ("workspace", torch.zeros(512, dtype=torch.uint8)[::2])])
def test_layer_q8_refuses_strides(ops, name, other):
    with pytest.raises(ValueError, match=f"^{name}: a contiguous tensor"):
        call(ops, **{name: other})


@pytest.mark.parametrize("name,other", [("xq", torch.zeros(3, 256, dtype=torch.uint8)), ("xq_scale", torch.zeros(4, 3)),
                                        ("out", torch.zeros(5, 256, dtype=BF16)),
                                        ("dev_status", torch.zeros(2, dtype=torch.int32))])
def test_layer_q8_refuses_sizes(ops, name, other):
    with pytest.raises(ValueError, match=f"^{name}: .* values expected"):
        call(ops, **{name: other})


def test_layer_q8_refuses_tensors_of_the_host(ops):
    with pytest.raises(ValueError, match="^x: a tensor on the GPU"):
        call(ops)


@pytest.mark.parametrize("wdtype", ["W_BF16", "W8A8_FP8"])
@pytest.mark.parametrize("out", [torch.zeros(4, 256), torch.zeros(3, 256, dtype=BF16), torch.zeros(4, 256, dtype=torch.uint8),
                                 torch.zeros(256, 4, dtype=BF16).t(), torch.zeros(4, 256, dtype=BF16)])
def test_block_refuses_an_output_that_it_cannot_fill(ops, wdtype, out):
    cfg = ops.make_config(64, 256, 8, 2, 128, wdtype=getattr(ops, wdtype))
    block = ops.MoEBlock(cfg, {}, torch.ones(256, dtype=BF16), device="cpu")
    with pytest.raises(ValueError, match="^out: "):
        block(torch.zeros(4, 256, dtype=BF16), out=out)
