"""Argument checks of the operators around the layer (no GPU: every call fails
validation, or has nothing to do, before anything is queued)."""
import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod

A = 0x1000  # an aligned address that no call reaches


@pytest.fixture(scope="module")
def ops():
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def test_add_rmsnorm_refusals(ops):
    def f(x=A, res=2 * A, w=A, wdt=0, T=4, H=256, eps=1e-6, h=3 * A, y=4 * A, rstd=A, yq=A, ys=A,
          g=128):
        return ops.lib().moe_add_rmsnorm(x, res, w, wdt, T, H, eps, h, y, rstd, yq, ys, g, None)

    assert f(T=-1) == 1 and f(H=0) == 1 and f(H=24) == 1 and f(wdt=2) == 1
    assert f(H=32784) == 2 and f(g=64) == 2
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert f(eps=eps) == 1
    assert f(x=None) == 1 and f(w=None) == 1
    assert f(res=None) == 1                      # h without a residual
    assert f(y=None, yq=None, ys=None) == 1      # no output
    assert f(yq=None) == 1 and f(ys=None) == 1   # codes and scales come together
    assert f(y=3 * A) == 1 and f(y=2 * A) == 1   # y over h, y over the residual
    for k in ("x", "res", "w", "h", "y", "yq"):
        assert f(**{k: A + 8}) == 4, k
    assert f(rstd=A + 2) == 4 and f(ys=A + 2) == 4
    assert f(T=0) == 0


def test_add_rmsnorm_backward_refusals(ops):
    need = ops.add_rmsnorm_backward_scratch_bytes(64, 256)
    assert need > 0 and need % 256 == 0
    assert ops.add_rmsnorm_backward_scratch_bytes(1 << 20, 8192) < (1 << 26)

    def f(dy=A, dh=None, h=A, rstd=A, w=A, wdt=0, T=64, H=256, dx=A, dw=A, s=A, n=need):
        return ops.lib().moe_add_rmsnorm_backward(dy, dh, h, rstd, w, wdt, T, H, dx, dw, s, n, None)

    assert f(T=-1) == 1 and f(H=8) == 1 and f(wdt=-1) == 1 and f(H=65536) == 2
    for k in ("dy", "h", "rstd", "w", "dx", "dw", "s"):
        assert f(**{k: None}) == 1, k
    assert f(n=need - 1) == 3
    for k in ("dy", "dh", "h", "w", "dx"):
        assert f(**{k: A + 8}) == 4, k
    assert f(s=A + 128) == 4 and f(dw=A + 1) == 4
    with pytest.raises(ops.MoEError):
        ops.add_rmsnorm_backward_scratch_bytes(4, 20)


def test_balance_loss_refusals(ops):
    need = ops.balance_loss_scratch_bytes(64, 8, 4)

    def f(l=A, ld=8, ids=A, mask=None, T=64, E=8, K=2, S=4, mode=0, c=A, mp=A, v=A, lo=A, s=A,
          n=need, st=None):
        return ops.lib().moe_balance_loss(l, ld, ids, mask, T, E, K, S, mode, c, mp, v, lo, s, n, st,
                                          None)

    assert f(T=-4) == 1 and f(E=0) == 1 and f(E=1025, ld=1025) == 1 and f(K=0) == 1 and f(K=9) == 1
    assert f(E=64, K=33, ld=64) == 1 and f(S=0) == 1 and f(S=3) == 1 and f(mode=2) == 1
    assert f(ld=7) == 1
    for k in ("l", "ids", "c", "mp", "v", "lo", "s"):
        assert f(**{k: None}) == 1, k
    assert f(n=need - 1) == 3
    assert f(s=A + 128) == 4 and f(l=A + 2) == 4 and f(lo=A + 2) == 4 and f(st=A + 2) == 4
    with pytest.raises(ops.MoEError):
        ops.balance_loss_scratch_bytes(10, 8, 3)
    # more blocks and more sequences never need less
    assert ops.balance_loss_scratch_bytes(1 << 16, 128, 1) >= ops.balance_loss_scratch_bytes(64, 128, 1)
    assert ops.balance_loss_scratch_bytes(1 << 16, 128, 64) >= 64 * 128 * 12


def test_route_backward_refusals(ops):
    def f(l=A, ld=9, ids=A, w=A, dw=A, ds=None, mask=None, T=64, E=8, K=2, S=4, mode=0, c=A, v=A,
          gl=A, dl=2 * A, ldd=9, st=None):
        return ops.lib().moe_route_backward(l, ld, ids, w, dw, ds, mask, T, E, K, S, mode, 1.0, c, v,
                                            gl, dl, ldd, st, None)

    assert f(T=-4) == 1 and f(E=1025) == 1 and f(K=9) == 1 and f(S=5) == 1 and f(mode=3) == 1
    assert f(ld=7) == 1 and f(ldd=7) == 1
    assert f(ds=A, ld=8) == 1 and f(ds=A, ldd=8) == 1
    assert f(w=None) == 1 and f(ids=None) == 1 and f(c=None) == 1 and f(v=None) == 1
    assert f(l=None) == 1 and f(dl=None) == 1 and f(dl=A) == 1
    assert f(dl=A + 2) == 4 and f(gl=A + 1) == 4 and f(dw=A + 1) == 4
    assert f(T=0) == 0


def test_unpermute_backward_refusals(ops):
    def f(d=A, y=A, f2r=A, w=A, T=4, K=2, H=256, sy=A, sg=A, dy=A, dw=A, dsy=A, dsg=A):
        return ops.lib().moe_unpermute_backward(d, y, f2r, w, T, K, H, sy, sg, dy, dw, dsy, dsg, None)

    assert f(T=-1) == 1 and f(K=0) == 1 and f(H=12) == 1 and f(H=32776) == 2
    assert f(T=1 << 30, K=4) == 1
    assert f(dy=None, dw=None, dsy=None, dsg=None) == 1
    assert f(y=None) == 1 and f(w=None) == 1 and f(sy=None) == 1 and f(sg=None) == 1
    assert f(d=None) == 1 and f(f2r=None) == 1
    for k in ("d", "y", "dy", "sy", "dsy"):
        assert f(**{k: A + 8}) == 4, k
    for k in ("f2r", "w", "dw", "sg", "dsg"):
        assert f(**{k: A + 2}) == 4, k
    assert f(T=0) == 0


def test_binding_refuses_other_types_shapes_and_strides(ops):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w, y = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf), torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="x"):
        ops.add_rmsnorm(x.float(), w, 1e-6, y)
    with pytest.raises(ValueError, match="weight"):
        ops.add_rmsnorm(x, w[:32], 1e-6, y)
    with pytest.raises(ValueError, match="y"):
        ops.add_rmsnorm(x, w, 1e-6, torch.zeros(64, 4, dtype=bf).t())
    with pytest.raises(ValueError, match="yq_scale"):
        ops.add_rmsnorm(x, w, 1e-6, y, yq=torch.zeros(4, 64, dtype=torch.uint8), yq_scale=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="rstd"):
        ops.add_rmsnorm_backward(x, x, torch.zeros(3), w, y, torch.zeros(64), torch.zeros(8))
    l, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32)
    out = [torch.zeros(8, dtype=i32), torch.zeros(8), torch.zeros(3, dtype=i32), torch.zeros(2)]
    with pytest.raises(ValueError, match="ids"):
        ops.balance_loss(l, ids.long(), 8, *out, torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="token_mask"):
        ops.balance_loss(l, ids, 8, *out, torch.zeros(4096, dtype=torch.uint8), token_mask=torch.ones(4))
    with pytest.raises(ValueError, match="d_weights"):
        ops.route_backward(l, ids, 8, torch.zeros(4, 8), weights=torch.zeros(4, 2), d_weights=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="dy"):
        ops.unpermute_backward(x, torch.zeros(8, dtype=i32), torch.zeros(4, 2), 4, 2, 64,
                               dy=torch.zeros(4, 64, dtype=bf))


def test_binding_refuses_tensors_of_the_host(ops):
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf)
    with pytest.raises(ValueError, match="x: a tensor on the GPU"):
        ops.add_rmsnorm(x, w, 1e-6, torch.zeros(4, 64, dtype=bf))
    with pytest.raises(ValueError, match="x: a matrix"):
        ops.add_rmsnorm(x[0], w, 1e-6, x)
    with pytest.raises(TypeError):
        ops.add_rmsnorm(x, w, "eps", x)
    with pytest.raises(AttributeError):
        ops.add_rmsnorm([1.0], w, 1e-6, x)
