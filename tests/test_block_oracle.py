"""The oracle of the operators around the layer: its gradients against central
differences of its forward passes, its definitions against closed forms."""
import numpy as np
import pytest

from oracle import block_oracle as bo

EPS = 1e-6


def numeric_grad(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


# a central difference of step d errs by about d^2 |f'''| / 6 + 2^-53 |f| / d:
# below 1e-9 relative to values of order one
TOL = 1e-8


def test_rmsnorm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(0)
    h, w, dy, dh = rng.normal(size=(3, 16)), rng.normal(size=16), rng.normal(size=(3, 16)), rng.normal(size=(3, 16))
    dx, dw = bo.rmsnorm_backward(dy, dh, h, w, EPS)
    f = lambda hh, ww: (bo.rmsnorm(hh, None, ww, EPS)[1] * dy).sum() + (hh * dh).sum()  # noqa: E731
    assert np.abs(dx - numeric_grad(lambda v: f(v, w), h)).max() < TOL
    assert np.abs(dw - numeric_grad(lambda v: f(h, v), w)).max() < TOL


def test_group_scales_follow_the_last_narrow_group():
    y = np.arange(1, 2 * 160 + 1, dtype=float).reshape(2, 160)
    s = bo.group_scales(y, 128)
    assert s.shape == (2, 2)
    assert np.allclose(s, np.array([[128, 160], [288, 320]]) / 448)


@pytest.mark.parametrize("mode", [0, 1])
def test_balanced_batch_has_loss_one(mode):
    E, K, T = 4, 2, 8
    ids = np.array([[t % 4, (t + 2) % 4] for t in range(T)], np.int32)
    r = bo.balance(np.full((T, E), 0.3), ids, None, E, 1, mode)
    assert np.allclose(r["mean_prob"], 0.25) and (r["counts"] == 4).all()
    assert r["losses"][0] == pytest.approx(1.0)
    assert r["losses"][1] == pytest.approx((0.3 + np.log(4)) ** 2)
    assert list(r["valid"]) == [8, 8, 1]


@pytest.mark.parametrize("mode", [0, 1])
def test_masked_tokens_and_empty_rows_leave_no_trace(mode):
    rng = np.random.default_rng(1)
    l = rng.normal(size=(6, 5))
    ids = np.array([[0, 1]] * 6, np.int32)
    mask = np.array([1, 1, 0, 0, 0, 0], np.uint8)
    l[2:] = np.nan
    r = bo.balance(l, ids, mask, 5, 2, mode)
    assert np.isfinite(r["losses"]).all() and list(r["valid"]) == [2, 0, 2, 1]
    assert (r["counts"][1] == 0).all() and (r["mean_prob"][1] == 0).all()
    l[0] = -np.inf
    r = bo.balance(l, ids, mask, 5, 2, mode)
    assert r["mean_prob"][0].sum() == pytest.approx(0.5)  # one of two kept rows is empty
    d = bo.route_backward(l, ids, np.ones((6, 2)) / 2, None, None, mask, 5, 2, mode, 1.0, [1.0, 1.0])
    assert (d[0] == 0).all() and (d[2:] == 0).all() and np.isfinite(d).all()


@pytest.mark.parametrize("mode,scale", [(0, 1.0), (1, 2.5)])
def test_route_gradient_is_the_difference_quotient(mode, scale):
    rng = np.random.default_rng(2)
    T, E, K, S = 6, 5, 3, 2
    l = rng.normal(size=(T, E + 1))
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    mask = np.array([1, 1, 0, 1, 0, 0], np.uint8)
    gw, gs, gl = rng.normal(size=(T, K)), rng.normal(size=T), [0.7, 0.3]

    def f(v):
        w = bo.routing_weights(v, ids, mode, scale)
        b = bo.balance(v, ids, mask, E, S, mode)["losses"]
        per = (w * gw).sum(axis=1) + gs / (1 + np.exp(-v[:, E]))
        return per[mask.astype(bool)].sum() + gl[0] * b[0] + gl[1] * b[1]

    w = bo.routing_weights(l, ids, mode, scale)
    d = bo.route_backward(l, ids, w, gw, gs, mask, E, S, mode, scale, gl)
    assert np.abs(d - numeric_grad(f, l)).max() < TOL


def test_combine_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(3)
    T, K, H = 3, 2, 8
    y, w, sy, sg, dout = (rng.normal(size=s) for s in ((T * K, H), (T, K), (T, H), (T,), (T, H)))
    f2r = rng.permutation(T * K)

    def f(y, w, sy, sg):
        return (((y[f2r].reshape(T, K, H) * w[:, :, None]).sum(1) + sg[:, None] * sy) * dout).sum()

    r = bo.unpermute_backward(dout, y, f2r, w, sy, sg)
    assert np.abs(r["dy"] - numeric_grad(lambda v: f(v, w, sy, sg), y)).max() < TOL
    assert np.abs(r["d_weights"] - numeric_grad(lambda v: f(y, v, sy, sg), w)).max() < TOL
    assert np.abs(r["d_shared_y"] - numeric_grad(lambda v: f(y, w, v, sg), sy)).max() < TOL
    assert np.abs(r["d_shared_gate"] - numeric_grad(lambda v: f(y, w, sy, v), sg)).max() < TOL
