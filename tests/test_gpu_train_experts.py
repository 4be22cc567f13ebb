"""GPU: a training step of a block whose experts learn and whose activations are kept in 8 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D = torch.float64


@pytest.fixture(scope="module")
def example():
    from mixture_experts_layer_07_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def step(m, **kw):
    b = m.Block(n_seq=3, L=20, H=128, E=6, K=2, I=64, seed=2, alpha=0.5, beta=0.05, **kw)
    g = torch.Generator("cuda").manual_seed(7)
    T, H = b.T, b.H
    x, r = (torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    mask = torch.rand(T, device="cuda", generator=g) < 0.7
    d_out = torch.randn(T, H, device="cuda", generator=g) * mask[:, None] / T
    b.norm.add_(0.1 * torch.randn(H, device="cuda", generator=g))
    b.forward(x, r, mask)
    got = [t.double() for t in (*b.backward(d_out, mask), *b.d_experts)]
    torch.cuda.synchronize()
    assert int(b.status) == 0
    return b, x, r, mask, d_out, got


def wanted(m, b, x, r, mask, d_out):
    """The same gradients in 64 bits."""
    E = b.E
    leaf = lambda t: t.to(D).requires_grad_()  # noqa: E731
    xd, wg, nw = leaf(x), leaf(b.wg), leaf(b.norm)
    ws = [leaf(w) for w in (b.w1, b.w3, b.w2)]
    h = xd + r.to(D)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + m.EPS) * nw
    logits = y @ wg.t()
    ids = b.ids.long()
    w = torch.softmax(logits.gather(1, ids), 1)
    moe = torch.zeros_like(h)
    for e in range(E):
        act = torch.nn.functional.silu(y @ ws[0][e].t()) * (y @ ws[1][e].t())
        moe = moe + (w * (ids == e)).sum(1, keepdim=True) * (act @ ws[2][e].t())
    p = torch.softmax(logits, 1).view(b.n_seq, -1, E)
    k = mask.view(b.n_seq, -1).to(D)
    n = k.sum(1)
    counts = torch.nn.functional.one_hot(ids, E).sum(1).view(b.n_seq, -1, E).to(D)
    f = E * (counts * k[..., None]).sum(1) / (b.K * n[:, None])
    balance = (f * (p * k[..., None]).sum(1) / n[:, None]).sum(1).mean()
    z = (torch.logsumexp(logits, 1).square() * k.reshape(-1)).sum() / k.sum()
    total = ((h + moe) * d_out.to(torch.bfloat16).to(D)).sum() + 0.5 * balance + 0.05 * z
    return torch.autograd.grad(total, (xd, wg, nw, *ws))


NAMES = ("dx", "d_gate", "d_norm", "dw1", "dw3", "dw2")


def test_experts_gradients_match_64_bit_autograd(example):
    b, x, r, mask, d_out, got = step(example)
    # bf16 rounds y, act, the products' gradients and the sums (2^-8 each); six such roundings
    for g, w, name in zip(got, wanted(example, b, x, r, mask, d_out), NAMES):
        rel = float((g - w).norm() / w.norm())
        assert rel < 6 * 2 ** -8, (name, rel)


def test_gradients_from_8_bit_activations(example):
    b, x, r, mask, d_out, got = step(example, q8=True)
    # on top of the roundings above: y and h are off by half a step of e4m3, 2^-4 relative to each
    # value at most.  Every gradient is of first order in y (the matrices', the gate's and the norm's
    # weight's) or depends on it through the recomputed g and u: their derivative along y is
    # O(1) times the relative change, three factors of it at the most (x, silu', u)
    for g, w, name in zip(got, wanted(example, b, x, r, mask, d_out), NAMES):
        rel = float((g - w).norm() / w.norm())
        assert rel < 6 * 2 ** -8 + 3 * 2 ** -4, (name, rel)
    # and the same outputs, bit for bit, from the unpacked codes
    T, H = x.shape
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    example.ops.unpack_q8(b.yq, b.ys, y)
    dx, dw = torch.empty_like(y), [torch.empty_like(t) for t in b.d_experts]
    example.ops.experts_backward(d_out.to(torch.bfloat16), b.offsets, b.r2f, b.f2r, b.weights, b.w1, b.w3, b.w2,
                                 b.s_experts, x=y, dx=dx, d_weights=None, dw1=dw[0], dw3=dw[1], dw2=dw[2])
    assert torch.equal(dx, b.dy)
    for a, c in zip(dw, b.d_experts):
        assert torch.equal(a, c)


@pytest.mark.parametrize("q8", [False, True])
def test_training_runs(example, q8):
    b, hist = example.train(steps=3, n_seq=2, L=33, H=144, E=5, K=2, I=80, q8=q8)
    assert np.isfinite(hist).all() and len(hist) == 3
    assert int(b.counts.sum()) == int(b.valid[-2]) * b.K
