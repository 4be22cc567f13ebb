"""Whose routing MoELayer.experts_backward takes (no GPU: the library's calls are stubs)."""
import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod

BF16 = torch.bfloat16


@pytest.fixture
def ops(monkeypatch):
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    for name in ("layer", "layer_q8", "add_rmsnorm"):
        monkeypatch.setattr(o, name, lambda *a, **kw: None)
    o.taken = []
    monkeypatch.setattr(o, "experts_backward", lambda dout, *a, **kw: o.taken.append(dout.shape[0]))
    yield o
    del o.taken


def rows(T, H=256):
    return torch.zeros(T, H, dtype=BF16)


def layer_of(ops, **kw):
    cfg = ops.make_config(64, 256, 8, 2, 128, **kw)
    w = {n: torch.zeros(1, dtype=BF16) for n in ("w1", "w3", "w2")}
    return ops.MoELayer(cfg, w, device="cpu"), cfg, w


def test_the_gradient_takes_as_many_tokens_as_the_last_call_had(ops):
    layer, _, _ = layer_of(ops)
    scratch = torch.zeros(256, dtype=torch.uint8)
    for T in (24, 64, 0, 1):
        layer(rows(T))
        for other in {T - 1, T + 1, 40} - {T, -1}:
            with pytest.raises(ValueError, match=f"^dout: {other} tokens.* {T}"):
                layer.experts_backward(rows(other), scratch, x=rows(other), dx=rows(other))
        layer.experts_backward(rows(T), scratch, x=rows(T), dx=rows(T))
    assert ops.taken == [24, 64, 0, 1]


def test_there_is_no_gradient_before_the_first_call(ops):
    layer, _, _ = layer_of(ops)
    with pytest.raises(ValueError, match="^dout: 24 tokens"):
        layer.experts_backward(rows(24), torch.zeros(256, dtype=torch.uint8), x=rows(24), dx=rows(24))
    assert not ops.taken


def test_a_refused_call_leaves_the_routing_of_the_one_before(ops, monkeypatch):
    layer, _, _ = layer_of(ops)
    layer(rows(24))

    def refuse(*a, **kw):
        raise ops.MoEError(1, "moe_layer")

    monkeypatch.setattr(ops, "layer", refuse)
    with pytest.raises(ops.MoEError):
        layer(rows(30))
    layer.experts_backward(rows(24), torch.zeros(256, dtype=torch.uint8), x=rows(24), dx=rows(24))
    assert ops.taken == [24]


@pytest.mark.parametrize("wdtype", ["W_BF16", "W8A8_FP8"])
def test_a_block_calls_its_layer(ops, wdtype):
    _, cfg, w = layer_of(ops, wdtype=getattr(ops, wdtype))
    block = ops.MoEBlock(cfg, w, torch.ones(256, dtype=BF16), device="cpu")
    scratch = torch.zeros(256, dtype=torch.uint8)
    for T in (24, 9):
        block(rows(T))
        with pytest.raises(ValueError, match=f"^dout: {T + 1} tokens.* {T}"):
            block.layer.experts_backward(rows(T + 1), scratch, x=rows(T + 1), dx=rows(T + 1))
        block.layer.experts_backward(rows(T), scratch, x=rows(T), dx=rows(T))
    assert ops.taken == [24, 9]


def test_a_replayed_call_is_told_by_its_number_of_tokens(ops):
    layer, _, _ = layer_of(ops)
    layer(rows(24))
    layer(rows(60))
    layer.tokens = 24  # a graph that holds the first call ran again
    layer.experts_backward(rows(24), torch.zeros(256, dtype=torch.uint8), x=rows(24), dx=rows(24))
    assert ops.taken == [24]
