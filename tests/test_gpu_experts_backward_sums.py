"""GPU: how near the routing weights' gradient comes to 64 bits, whatever H is.

d_weights is fp32 and behind no rounding to bf16, so it shows the errors of the sums a, g and u over
H.  The tensor cores cut their running fp32 sum once per 16 of K: 0.72 x 2^-24 of it on the average
(half an ulp, over a binade), always towards zero.  A sum of n such steps in one go, whose terms have
no common sign, ends n / 2 times that too short (step j meets j / n of what the end has); taken out
every 256 of H, n is 16, and 32 for the first 512 where H takes 24 stages of 64 or more:

    H = 512, 1472   16 / 2 x 4.3e-8                              3.4e-7
    H = 1520, 1536  a third of it with n = 32                    4.6e-7
    H = 2880        a sixth                                      4.0e-7
    H = 8192        a sixteenth                                  3.6e-7

a and u enter the product once, g with silu's slope over its value, about 1.2 in this norm: 3.2 times
that, 1.5e-6 at the most.  Additions in registers (2^-24 each, either sign), the exponential and the
reciprocal (2^-22 each) add less than 0.5e-6.  In one go H = 1472 would give 6.3e-6, 2880 1.2e-5.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, I32, D = torch.bfloat16, torch.float32, torch.int32, torch.float64


@pytest.mark.parametrize("H", [512, 1472, 1520, 1536, 2880, 8192])
def test_d_weights_near_64_bits(H):
    from mixture_experts_layer_07_gb300 import build
    build.build()
    from mixture_experts_layer_07_gb300 import ops
    T, I = 400, 256
    g = torch.Generator("cuda").manual_seed(H)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dout = rand(T, H).to(BF16), (rand(T, H) * 0.01).to(BF16)
    w1, w3 = ((rand(1, I, H) * H ** -0.5).to(BF16) for _ in range(2))
    w2 = (rand(1, H, I) * I ** -0.5).to(BF16)
    at = torch.arange(T, dtype=I32, device="cuda")
    off = torch.tensor([0, T], dtype=I32, device="cuda")
    weights, d = torch.rand(T, 1, device="cuda", generator=g), torch.empty(T, 1, device="cuda")
    scratch = torch.empty(ops.experts_backward_scratch_bytes(T, H, 1, 1, I), dtype=torch.uint8, device="cuda")
    ops.experts_backward(dout, off, at, at, weights, w1, w3, w2, scratch, x=x, d_weights=d)
    gate, up, a = x.to(D) @ w1[0].to(D).t(), x.to(D) @ w3[0].to(D).t(), dout.to(D) @ w2[0].to(D)
    want = (a * gate * torch.sigmoid(gate) * up).sum(1, keepdim=True)
    rel = float((d.to(D) - want).norm() / want.norm())
    assert rel < 2e-6, rel
