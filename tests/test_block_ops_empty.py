"""Calls without a token: empty tensors have no address, and there is nothing to refuse."""
import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod

BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def ops():
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def test_c_calls_without_tokens(ops):
    L, n = ops.lib(), None
    assert L.moe_add_rmsnorm(n, n, 0x1000, 0, 0, 256, 1e-6, n, n, n, n, n, 128, n) == 0
    assert L.moe_unpermute_backward(n, n, n, n, 0, 2, 256, n, n, n, n, n, n, n) == 0
    assert L.moe_route_backward(n, 8, n, n, n, n, n, 0, 8, 2, 1, 0, 1.0, 0x1000, 0x1000, 0x1000, n, 8, n, n) == 0
    # sizes are checked all the same
    assert L.moe_add_rmsnorm(n, n, n, 0, 0, 24, 1e-6, n, n, n, n, n, 128, n) == 1
    assert L.moe_add_rmsnorm(n, n, n, 0, 0, 256, 0.0, n, n, n, n, n, 128, n) == 1
    assert L.moe_unpermute_backward(n, n, n, n, 0, 2, 12, n, n, n, n, n, n, n) == 1


@pytest.mark.gpu
def test_python_calls_without_tokens(ops):
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    x, w = e(0, 256, dt=BF16), torch.ones(256, dtype=BF16, device="cuda")
    ops.add_rmsnorm(x, w, 1e-6, x, rstd=e(0))
    ops.add_rmsnorm(x, w, 1e-6, e(0, 256, dt=BF16), residual=x, h=e(0, 256, dt=BF16), yq=e(0, 256, dt=torch.uint8),
                    yq_scale=e(0, 2))
    ops.add_rmsnorm(x, w, 1e-6, None, yq=e(0, 256, dt=torch.uint8), yq_scale=e(0), q_group=0)
    ops.unpermute_backward(x, e(0, dt=I32), e(0, 2), 0, 2, 256, y=x, dy=x, d_weights=e(0, 2), shared_y=x,
                           shared_gate=e(0), d_shared_y=x, d_shared_gate=e(0))
    ops.route_backward(e(0, 8), e(0, 2, dt=I32), 8, e(0, 8), weights=e(0, 2), d_weights=e(0, 2), n_seq=1,
                       counts=e(1, 8, dt=I32), valid=e(3, dt=I32), grad_losses=e(2))
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["W_BF16", "W8A8_FP8"])
@pytest.mark.parametrize("residual", [False, True])
def test_block_without_tokens(ops, wdtype, residual):
    cfg = ops.make_config(64, 256, 8, 2, 128, wdtype=getattr(ops, wdtype))
    block = ops.MoEBlock(cfg, {}, torch.ones(256, dtype=BF16, device="cuda"))
    x = torch.empty(0, 256, dtype=BF16, device="cuda")
    out, h = block(x, x if residual else None)
    assert out.shape == h.shape == x.shape
