"""GPU: the experts' gradient through a layer and a block, on the routing of their last call."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixture_experts_layer_07_gb300 import build
    build.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def test_routing_of_a_call_of_another_size_is_refused(ops):
    from mixture_experts_layer_07_gb300 import synth
    from tests import gpu_util as gu
    spec = synth.SPECS["tiny"]
    t = gu.layer_tensors(synth.host_inputs(spec, 64, seed=5))
    block = ops.MoEBlock(gu.config_for(ops, spec, 64), t, torch.ones(spec.H, dtype=BF16, device="cuda"))
    layer, E, K = block.layer, spec.E, spec.K
    scratch = torch.empty(ops.experts_backward_scratch_bytes(64, spec.H, E, K, spec.I), dtype=torch.uint8,
                          device="cuda")
    g = torch.Generator("cuda").manual_seed(0)
    for T, call in ((24, layer), (40, block), (64, layer), (3, block)):
        call(t["x"][:T])
        x = block.y[:T] if call is block else t["x"][:T]
        dout = torch.randn(64, spec.H, device="cuda", generator=g).to(BF16)
        dx, dw = torch.empty(T, spec.H, dtype=BF16, device="cuda"), torch.empty(T, K, device="cuda")
        for other in (T - 1, T + 1):
            if other <= 64:
                with pytest.raises(ValueError, match=f"^dout: {other} tokens"):
                    layer.experts_backward(dout[:other], scratch, x=t["x"][:other], dx=dx)
        layer.experts_backward(dout[:T], scratch, x=x, dx=dx, d_weights=dw)
        view = lambda n, dt, *s: layer.view(n, dt, s).clone()  # noqa: E731
        want, w_want = torch.empty_like(dx), torch.empty_like(dw)
        ops.experts_backward(dout[:T], view("offsets", I32, E + 1), view("row_to_flat", I32, T * K),
                             view("flat_to_row", I32, T * K), view("weights", F32, T, K), t["w1"], t["w3"], t["w2"],
                             scratch, x=x, dx=want, d_weights=w_want)
        assert torch.equal(dx, want) and torch.equal(dw, w_want)
    assert int(layer.dev_status) == 0
