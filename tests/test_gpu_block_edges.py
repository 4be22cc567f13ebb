"""GPU: the operators around the layer where a value is small beside its parts,
where an input is not finite, and at the ends of their ranges.

Tolerances as in test_gpu_block_ops: u = 2^-24 per fp32 rounding.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests.test_gpu_block_ops import U, balance, f32, f64, i32, ops, row_range, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 1 - sigmoid
# every tier of the logit gradient, whole and ragged
@pytest.mark.parametrize("E,K", [(7, 2), (16, 3), (32, 4), (50, 4), (64, 6), (128, 8), (200, 8), (256, 8), (300, 8),
                                 (512, 10), (800, 16), (896, 16), (1000, 32), (1024, 32)])
@pytest.mark.parametrize("centre", [-8.0, 0.0, 4.0, 8.0, 14.0, 20.0, 40.0])
@pytest.mark.parametrize("part", ["losses", "weights"])
def test_sigmoid_gradient_keeps_its_digits(ops, E, K, centre, part):  # noqa: F811
    """Every column against its own size, the factor 1 - sigmoid included: a row of large logits
    has nothing but terms with that factor when the z-loss is off."""
    S, L, scale = 2, 9, 2.5
    T = S * L
    g = np.random.default_rng(E + abs(int(centre)))
    l = (g.normal(size=(T, E)) * 0.5 + centre).astype(np.float32)
    ids = np.argsort(-(l + g.normal(size=(T, E))), axis=1)[:, :K].astype(np.int32)
    w = bo.routing_weights(l, ids, 1, scale).astype(np.float32)
    gl = np.array([0.6, 0.0], np.float32) if part == "losses" else None
    gw = g.normal(size=(T, K)).astype(np.float32) if part == "weights" else None
    dl, di = f32(l), i32(ids)
    c, _, v, _ = balance(ops, dl, di, None, E, S, 1)
    out = torch.empty(T, E, device="cuda")
    ops.route_backward(dl, di, E, out, mode=1, scale=scale, weights=f32(w), d_weights=None if gw is None else f32(gw),
                       n_seq=S, counts=c, valid=v, grad_losses=None if gl is None else f32(gl))
    torch.cuda.synchronize()
    ref = bo.route_backward(l, ids, w, gw, None, None, E, S, 1, scale, gl)
    tail = 1.0 / (1.0 + np.exp(l.astype(np.float64)))
    mag = np.zeros((T, E))
    if part == "losses":
        cc = c.cpu().numpy()
        for t in range(T):
            a = gl[0] * E * cc[t // L] / (K * L * L * S)
            p = bo.probabilities(l[t:t + 1], 1)[0]
            mag[t] = p * (a + (a * p).sum()) * tail[t]
    else:
        for t in range(T):
            tot = (w[t] * np.abs(gw[t])).sum()
            for k in range(K):
                mag[t, ids[t, k]] += w[t, k] * (abs(gw[t, k]) + tot / scale) * tail[t, ids[t, k]]
    # as for the probabilities: e^-l is off by 2 |l| u (its argument's product and
    # constant), the sums by 160 u; row_range holds the largest |l|
    rel = (3 * row_range(l, E, np.ones(T, bool)) + 256) * U
    within(f64(out), ref, rel * mag, "dlogits")
