"""Argument checks of the experts' gradient and of the 8-bit activations (no GPU: every call
fails validation, or has nothing to do, before anything is queued), and the oracle's gradient
against difference quotients."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod
from oracle import block_oracle as bo

A = 0x1000  # an aligned address that no call reaches
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def ops():
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def test_pack_and_unpack_refusals(ops):
    L = ops.lib()
    for T, H, want in ((-1, 256, 1), (4, 0, 1), (4, 24, 1), (0, 256, 0)):
        assert L.moe_pack_q8(A, T, H, A, A, None) == want and L.moe_unpack_q8(A, A, T, H, A, None) == want
    assert L.moe_pack_q8(None, 0, 256, None, None, None) == 0
    for k in range(3):
        p = [A, A, A]
        p[k] = None
        assert L.moe_pack_q8(p[0], 4, 256, p[1], p[2], None) == 1
        assert L.moe_unpack_q8(p[1], p[2], 4, 256, p[0], None) == 1
        p[k] = A + (2 if k == 2 else 8)
        assert L.moe_pack_q8(p[0], 4, 256, p[1], p[2], None) == 4
        assert L.moe_unpack_q8(p[1], p[2], 4, 256, p[0], None) == 4


def test_norm_backward_q8_refusals(ops):
    need = ops.add_rmsnorm_backward_scratch_bytes(64, 256)

    def f(dy=A, dh=None, hq=A, hs=A, rstd=A, w=A, wdt=0, T=64, H=256, dx=A, dw=A, s=A, n=need):
        return ops.lib().moe_add_rmsnorm_backward_q8(dy, dh, hq, hs, rstd, w, wdt, T, H, dx, dw, s, n, None)

    assert f(T=-1) == 1 and f(H=8) == 1 and f(wdt=2) == 1 and f(H=65536) == 2
    for k in ("dy", "hq", "hs", "rstd", "w", "dx", "dw", "s"):
        assert f(**{k: None}) == 1, k
    for k in ("dy", "dh", "hq", "w", "dx"):
        assert f(**{k: A + 8}) == 4, k
    assert f(hs=A + 2) == 4 and f(rstd=A + 2) == 4 and f(n=need - 1) == 3


def test_experts_backward_refusals(ops):
    need = ops.experts_backward_scratch_bytes(64, 256, 8, 2, 128)
    assert need % 256 == 0

    def f(x=A, xq=None, xs=None, dout=A, off=A, r2f=A, f2r=A, wt=A, T=64, H=256, E=8, K=2, I=128, w1=A, w3=A, w2=A,
          add=A, dx=A, dwt=A, dw1=A, dw3=A, dw2=A, dt=0, acc=0, s=A, n=need, st=None):
        return ops.lib().moe_experts_backward(x, xq, xs, dout, off, r2f, f2r, wt, T, H, E, K, I, w1, w3, w2, add, dx,
                                              dwt, dw1, dw3, dw2, dt, acc, s, n, st, None)

    for bad in (dict(T=-1), dict(H=0), dict(H=24), dict(E=0), dict(E=1025), dict(K=0), dict(K=9), dict(E=64, K=33),
                dict(I=0), dict(I=24), dict(T=2 ** 30, K=8), dict(dt=2), dict(dt=-1), dict(acc=2)):
        assert f(**bad) == 1, bad
    for k in ("x", "dout", "off", "r2f", "f2r", "wt", "w1", "w3", "w2", "s"):
        assert f(**{k: None}) == 1, k
    assert f(x=A, xq=A, xs=A) == 1 and f(x=None, xq=A) == 1 and f(x=A, xs=A) == 1  # one form of the tokens
    for k in ("dw1", "dw3", "dw2"):                                               # the three together
        assert f(**{k: None}) == 1, k
    assert f(dx=None, dwt=None, dw1=None, dw3=None, dw2=None) == 1                # no output
    assert f(acc=1) == 2                                                          # bf16 sums lose what is added
    assert f(n=need - 1) == 3
    for k in ("x", "dout", "w1", "w3", "w2", "add", "dx", "dw1", "dw3", "dw2"):
        assert f(**{k: A + 8}) == 4, k
    assert f(x=None, xq=A + 8, xs=A) == 4 and f(x=None, xq=A, xs=A + 2) == 4
    for k in ("off", "r2f", "f2r", "wt", "dwt", "st"):
        assert f(**{k: A + 2}) == 4, k
    assert f(s=A + 128) == 4
    empty = dict(T=0, x=None, dout=None, r2f=None, f2r=None, wt=None, add=None, dx=None, dwt=None)
    assert f(**empty, dw1=None, dw3=None, dw2=None) == 0
    assert f(**empty, dt=1, acc=1) == 0


def test_experts_backward_scratch(ops):
    f = ops.experts_backward_scratch_bytes
    # x's and dout's rows, dg, du and w act, dx's rows in fp32; at most 15 padding rows per expert
    rows = 2048 * 8 + 15 * 128
    assert rows * (8 * 2048 + 6 * 768) <= f(2048, 2048, 128, 8, 768) < 1.05 * rows * (8 * 2048 + 6 * 768)
    assert f(0, 256, 8, 2, 128) > 0
    for bad in ((4, 24, 8, 2, 128), (4, 256, 8, 9, 128), (4, 256, 8, 2, 100), (-1, 256, 8, 2, 128)):
        with pytest.raises(ops.MoEError):
            f(*bad)


def test_python_calls_refuse_other_types_sizes_and_places(ops):
    x, q, s = torch.zeros(4, 256, dtype=BF16), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for args, name in (((x.float(), q, s), "x"), ((x[:, ::2], q, s), "x"), ((x, q[:3], s), "xq"), ((x, x, s), "xq"),
                       ((x, q, s[:, :1]), "xq_scale"), ((x, q, s.double()), "xq_scale")):
        with pytest.raises(ValueError, match=f"^{name}: "):
            ops.pack_q8(*args)
    with pytest.raises(ValueError, match="x: a tensor on the GPU"):
        ops.pack_q8(x, q, s)
    with pytest.raises(ValueError, match="xq_scale: "):
        ops.unpack_q8(q, s[:2], x)
    with pytest.raises(ValueError, match="hq: torch.bfloat16"):
        ops.add_rmsnorm_backward_q8(x, x, s, torch.zeros(4), x[0], x, torch.zeros(256), q)

    z = lambda *n, dt=F32: torch.zeros(*n, dtype=dt)  # noqa: E731
    w = z(3, 32, 256, dt=BF16)
    good = dict(dout=x, offsets=z(4, dt=I32), row_to_flat=z(8, dt=I32), flat_to_row=z(8, dt=I32), weights=z(4, 2),
                w1=w, w3=w.clone(), w2=z(3, 256, 32, dt=BF16), scratch=z(512, dt=torch.uint8), x=x, dx=x.clone(),
                dx_add=x.clone(), d_weights=z(4, 2), dw1=w.clone(), dw3=w.clone(), dw2=w.clone())
    for name, t in (("offsets", z(3, dt=I32)), ("offsets", z(4, dt=torch.int64)), ("row_to_flat", z(7, dt=I32)),
                    ("flat_to_row", z(8)), ("weights", z(5, 2)), ("w1", z(3, 32, 240, dt=BF16)), ("w3", z(3, 32, 256)),
                    ("w2", z(2, 256, 32, dt=BF16)), ("scratch", z(512)), ("x", z(4, 240, dt=BF16)),
                    ("dx", z(4, 256)), ("dx_add", z(3, 256, dt=BF16)), ("d_weights", z(4, 2, dt=BF16)),
                    ("dw1", z(3, 32, 240)), ("dw3", z(3, 32, 256)), ("dw2", z(3, 32, 256)),
                    ("dw1", z(3, 32, 512, dt=BF16)[:, :, ::2])):
        with pytest.raises(ValueError, match=f"^{name}: "):
            ops.experts_backward(**{**good, name: t})
    with pytest.raises(ValueError, match="^w1: a stack of matrices"):
        ops.experts_backward(**{**good, "w1": z(96, 256, dt=BF16)})
    with pytest.raises(ValueError, match="a tensor on the GPU expected"):
        ops.experts_backward(**good)
    with pytest.raises(ValueError, match="^xq: "):
        ops.experts_backward(**{**good, "x": None, "xq": x, "xq_scale": s})


def forward(x, ids, weights, w1, w3, w2):
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = ids[t, k]
            if e >= 0:
                g, u = w1[e] @ x[t], w3[e] @ x[t]
                out[t] += weights[t, k] * (w2[e] @ (g / (1 + np.exp(-g)) * u))
    return out


@pytest.mark.parametrize("name", ["x", "weights", "w1", "w3", "w2"])
def test_oracle_gradient_against_differences(name):
    g = np.random.default_rng(0)
    T, H, E, K, I = 5, 6, 4, 2, 3
    ids = np.stack([g.permutation(E)[:K] for _ in range(T)])
    ids[1, 0] = -1
    p = {"x": g.normal(size=(T, H)), "weights": g.random((T, K)), "w1": g.normal(size=(E, I, H)),
         "w3": g.normal(size=(E, I, H)), "w2": g.normal(size=(E, H, I))}
    dout = g.normal(size=(T, H))
    got = bo.experts_backward(p["x"], dout, ids, p["weights"], p["w1"], p["w3"], p["w2"])
    got = got["d_weights" if name == "weights" else "d" + name]
    loss = lambda q: (forward(q["x"], ids, q["weights"], q["w1"], q["w3"], q["w2"]) * dout).sum()  # noqa: E731
    eps = 1e-5
    for at in np.ndindex(p[name].shape):
        up, down = p[name].copy(), p[name].copy()
        up[at] += eps
        down[at] -= eps
        slope = (loss({**p, name: up}) - loss({**p, name: down})) / (2 * eps)
        # third derivatives of order 10 times eps^2, and the difference's cancellation
        assert abs(got[at] - slope) < 1e-7 * (1 + abs(slope)), (at, got[at], slope)


def test_oracle_pack_keeps_zero_groups_and_scales():
    x = np.zeros((2, 200))
    x[0, :128] = np.linspace(-3, 3, 128)
    q, s = bo.pack_q8(x)
    assert s.shape == (2, 2) and s[0, 1] == s[1, 0] == 0 and np.isclose(s[0, 0], 3 / 448)
    assert np.isclose(np.abs(q).max(), 448) and not q[1].any() and not q[0, 128:].any()
