"""GPU: the operators around the layer used together -- the W8A8 layer on
quantised activations, the pre-norm block, and a training step of a block."""
import ctypes
import importlib.util
import os

import numpy as np
import pytest
import torch

from mixture_experts_layer_07_gb300 import synth
from tests import gpu_util as gu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    from mixture_experts_layer_07_gb300 import build
    build.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def test_layer_q8_refusals(ops):
    w = ops.Weights(0x1000, None, None, 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, None, None, None)
    by = ctypes.byref

    def f(cfg, T=8, x=0x1000, xq=0x1000, xs=0x1000, n=None, ws=0x10000):
        n = ops.workspace_bytes(cfg) if n is None else n
        return ops.lib().moe_layer_q8(by(cfg), T, x, xq, xs, by(w), 0x1000, ws, n, None, None)

    cfg = ops.make_config(64, 256, 8, 2, 128, wdtype=ops.W8A8_FP8)
    assert f(ops.make_config(64, 256, 8, 2, 128, wdtype=ops.W_FP8)) == 2
    assert f(ops.make_config(64, 256, 8, 2, 128)) == 2
    assert f(cfg, xq=None) == 1 and f(cfg, xs=None) == 1 and f(cfg, x=None) == 1
    assert f(cfg, T=65) == 1 and f(cfg, T=-1) == 1 and f(cfg, T=0) == 0
    assert f(cfg, xq=0x1008) == 4 and f(cfg, xs=0x1002) == 4 and f(cfg, ws=0x10080) == 4
    assert f(cfg, n=ops.workspace_bytes(cfg) - 1) == 3


def test_layer_q8_refuses_other_sizes(ops):
    cfg = ops.make_config(64, 256, 8, 2, 128, wdtype=ops.W8A8_FP8)
    x, q, s = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for args, name in (((x[:, :128], q, s, x), "x"), ((x, q[:3], s, x), "xq"), ((x, q, s[:, :1], x), "xq_scale"),
                       ((x, q, s, x[:2]), "out")):
        with pytest.raises(ValueError, match=f"^{name}: "):
            ops.layer_q8(cfg, args[0], args[1], args[2], None, args[3], None)


def quantise(y):
    """Codes and scales per row and 128 columns, as the W8A8 path quantises bf16 rows."""
    T, H = y.shape
    n = -(-H // 128)
    p = torch.zeros(T, n * 128, device="cuda")
    p[:, :H] = y.float()
    m = p.view(T, n, 128).abs().amax(2)
    s = m / torch.full_like(m, 448.0)  # a division: by a plain number torch would multiply by 1 / 448
    q = torch.where(s[..., None] > 0, p.view(T, n, 128) / s[..., None], 0.0)
    return q.view(T, n * 128)[:, :H].to(torch.float8_e4m3fn).contiguous(), s


def w8a8_case(H=272, E=8, K=2, I=160, T=64, has_shared=False):
    spec = synth.SPECS["tiny"].with_(H=H, E=E, K=K, I=I, wdtype="fp8", act="fp8", has_shared=has_shared,
                                     I_shared=128 if has_shared else 0)
    inp = synth.host_inputs(spec, T, seed=3)
    return spec, gu.layer_tensors(inp)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 33, 300])
@pytest.mark.parametrize("shared", [False, True])
def test_layer_q8_is_the_layer_bit_for_bit(ops, T, shared):
    spec, t = w8a8_case(T=T, has_shared=shared)
    cfg = gu.config_for(ops, spec, T)
    layer = ops.MoELayer(cfg, t)
    want = layer(t["x"]).clone()
    xq, xs = quantise(t["x"])
    got = torch.empty_like(want)
    ops.layer_q8(cfg, t["x"], xq, xs, layer.weights, got, layer.workspace, layer.dev_status)
    torch.cuda.synchronize()
    assert int(layer.dev_status) == 0 and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 200])
@pytest.mark.parametrize("residual", [False, True])
def test_block_is_its_parts(ops, T, residual):
    g = torch.Generator("cuda").manual_seed(T)
    for spec, t in (w8a8_case(T=T), (synth.SPECS["tiny"], gu.layer_tensors(synth.host_inputs(synth.SPECS["tiny"], T, seed=4)))):
        H = spec.H
        norm = (1 + 0.1 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16)
        x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
        r = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16) if residual else None
        cfg = gu.config_for(ops, spec, 256)
        block = ops.MoEBlock(cfg, t, norm)
        out, h = block(x, r)
        y = torch.empty_like(x)
        hh = torch.empty_like(x) if residual else None
        yq, ys = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
        ops.add_rmsnorm(x, norm, 1e-6, y, residual=r, h=hh, yq=yq, yq_scale=ys)
        assert torch.equal(h, hh if residual else x)
        layer = ops.MoELayer(cfg, t)
        ref = torch.empty_like(x)
        if block.q8:
            ops.layer_q8(cfg, y, yq, ys, layer.weights, ref, layer.workspace, layer.dev_status)
        else:
            ref = layer(y)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
def test_block_gradients_match_64_bit_autograd(ops):
    m = example()
    b = m.Block(n_seq=3, L=20, H=128, E=6, K=2, I=64, seed=2, alpha=0.5, beta=0.05)
    g = torch.Generator("cuda").manual_seed(7)
    T, H, E = b.T, b.H, b.E
    x, r = (torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    mask = torch.rand(T, device="cuda", generator=g) < 0.7
    d_out = torch.randn(T, H, device="cuda", generator=g) * mask[:, None] / T
    b.norm.add_(0.1 * torch.randn(H, device="cuda", generator=g))
    b.forward(x, r, mask)
    dx, d_gate, d_norm = (t.double() for t in b.backward(d_out, mask))
    D = torch.float64
    leaf = lambda t: t.to(D).requires_grad_()  # noqa: E731
    xd, wg, nw = leaf(x), leaf(b.wg), leaf(b.norm)
    h = xd + r.to(D)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + m.EPS) * nw
    logits = y @ wg.t()
    ids = b.ids.long()
    w = torch.softmax(logits.gather(1, ids), 1)
    moe = torch.zeros(T, H, dtype=D, device="cuda")
    for e in range(E):
        a = torch.nn.functional.silu(y @ b.w1[e].to(D).t()) * (y @ b.w3[e].to(D).t())
        moe = moe + (w * (ids == e)).sum(1, keepdim=True) * (a @ b.w2[e].to(D).t())
    p = torch.softmax(logits, 1).view(3, 20, E)
    k = mask.view(3, 20).to(D)
    n = k.sum(1)
    counts = torch.nn.functional.one_hot(ids, E).sum(1).view(3, 20, E).to(D)
    f = E * (counts * k[..., None]).sum(1) / (b.K * n[:, None])
    balance = (f * (p * k[..., None]).sum(1) / n[:, None]).sum(1).mean()
    z = (torch.logsumexp(logits, 1).square() * k.reshape(-1)).sum() / k.sum()
    total = ((h + moe) * d_out.to(torch.bfloat16).to(D)).sum() + 0.5 * balance + 0.05 * z
    want = torch.autograd.grad(total, (xd, wg, nw))
    # bf16 rounds y, the expert rows and their gradients (2^-8 each); six such roundings
    for got, ref, name in zip((dx, d_gate, d_norm), want, ("dx", "d_gate", "d_norm")):
        rel = float((got - ref).norm() / ref.norm())
        assert rel < 6 * 2 ** -8, (name, rel)


@pytest.mark.gpu
def test_block_learns(ops):
    m = example()
    b, hist = m.train(steps=30)
    (t0, b0, z0), (t1, b1, z1) = hist[0], hist[-1]
    assert np.isfinite(hist).all() and t1 < t0 and z1 < z0 and b1 < b0
    assert int(b.counts.sum()) == int(b.valid[-2]) * b.K
