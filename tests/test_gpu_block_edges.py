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


# ------------------------------------------------------------------ norm: rows that are not finite
@pytest.mark.parametrize("H", [16, 256, 2880, 8208])
@pytest.mark.parametrize("T", [9, 400])
def test_norm_of_rows_that_are_not_finite_group_by_group(ops, T, H):  # noqa: F811
    """As the header has it: a NaN takes its whole row, an infinity its own group, and a finite row
    whose squares overflow comes out as zeros; the rows beside them are as without them."""
    g = torch.Generator("cuda").manual_seed(H)
    x, r = (torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16)
    clean = x.clone(), r.clone()
    col = {1: H // 2, 2: H - 1, 3: 0, 5: H // 3}
    x[1, col[1]] = float("nan")
    r[2, col[2]] = float("inf")
    x[3, col[3]] = -float("inf")
    x[4] = 3e19 * (1 + torch.arange(H, device="cuda") % 5)
    x[5, col[5]], r[5, col[5]] = float("inf"), -float("inf")  # their sum is a NaN
    odd = [1, 2, 3, 4, 5]
    even = [t for t in range(T) if t not in odd]
    for q in (128, 0):
        def norm(a, b):
            o = [torch.empty_like(a), torch.empty_like(a), torch.empty(T, device="cuda"),
                 torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda"),
                 torch.empty(T, -(-H // 128) if q else 1, device="cuda")]
            ops.add_rmsnorm(a, w, 1e-6, o[0], residual=b, h=o[1], rstd=o[2], yq=o[3], yq_scale=o[4], q_group=q)
            return o[0].float(), o[1].float(), o[2], o[3].float(), o[4]
        y, h, rstd, code, scale = norm(x, r)
        for a, b in zip((y, h, rstd, code, scale), norm(*clean)):
            assert torch.equal(a[even], b[even])
        assert torch.equal(h.nan_to_num(1.0, 2.0, 3.0), (x.float() + r.float()).to(torch.bfloat16).float().nan_to_num(1.0, 2.0, 3.0))
        for t in (1, 5):
            assert rstd[t].isnan() and y[t].isnan().all() and code[t].isnan().all() and scale[t].isnan().all()
        for t in (2, 3):
            assert rstd[t] == 0
            rest = torch.arange(H, device="cuda") != col[t]
            assert y[t, col[t]].isnan() and (y[t, rest] == 0).all()
            group = (torch.arange(H, device="cuda") // (q or H)) == col[t] // (q or H)
            assert code[t, group].isnan().all() and (code[t, ~group] == 0).all()
            mine = torch.arange(scale.shape[1], device="cuda") == col[t] // (q or H)
            assert scale[t, mine].isnan().all() and (scale[t, ~mine] == 0).all()
        assert rstd[4] == 0 and (y[4] == 0).all() and (code[4] == 0).all() and (scale[4] == 0).all()
        assert h[4].isfinite().all()


# ------------------------------------------------------------------ combine: dropped replicas
@pytest.mark.parametrize("T,K,H", [(1, 3, 64), (7, 5, 272), (400, 4, 2880), (3, 2, 32768)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_dropped_replica_has_no_gradient_where_dout_is_not_finite(ops, T, K, H, value):  # noqa: F811
    g = torch.Generator("cuda").manual_seed(T + K)
    b = torch.bfloat16
    dout, y = torch.randn(T, H, device="cuda", generator=g).to(b), torch.randn(T * K, H, device="cuda", generator=g).to(b)
    w = torch.randn(T, K, device="cuda", generator=g)
    f2r = torch.randperm(T * K, device="cuda", generator=g).to(torch.int32)
    dropped = torch.zeros(T, K, dtype=torch.bool, device="cuda")
    dropped[0, 1] = dropped[T - 1, 0] = True
    f2r.view(T, K)[0, 1], f2r.view(T, K)[T - 1, 0] = -1, T * K
    dout[[0, T - 1], H - 1] = value
    dy, dw = torch.full_like(y, 3.0), torch.full_like(w, 3.0)
    ops.unpermute_backward(dout, f2r, w, T, K, H, y=y, dy=dy, d_weights=dw)
    assert (dw[dropped] == 0).all()
    kept = dw[~dropped]
    assert (~kept.isfinite()).sum() == (~dropped[[0, T - 1]]).sum() // (2 if T == 1 else 1)
    bad = ~dy.isfinite().all(1)
    rows = f2r.view(T, K)[[0, T - 1]][~dropped[[0, T - 1]]].unique().long()
    assert bad[rows].all() and bad.sum() == len(rows)


@pytest.mark.parametrize("T,K,H", [(1, 262141, 8), (2, 300001, 16), (1, 131071, 32768)])
def test_combine_gradient_of_more_replicas_than_a_grid_has_rows(ops, T, K, H):  # noqa: F811
    """Few tokens spread their replicas over the grid's second axis, which ends at 65535 blocks."""
    g = torch.Generator("cuda").manual_seed(K)
    b = torch.bfloat16
    dout, sy = torch.randn(T, H, device="cuda", generator=g).to(b), torch.randn(T, H, device="cuda", generator=g).to(b)
    y = torch.randint(-2, 3, (T * K, H), device="cuda", generator=g, dtype=torch.int8).to(b)
    w, sg = torch.randn(T, K, device="cuda", generator=g), torch.randn(T, device="cuda", generator=g)
    f2r = torch.randperm(T * K, device="cuda", generator=g).to(torch.int32)
    dy, dw = torch.full_like(y, 3.0), torch.full_like(w, 3.0)
    dsy, dsg = torch.empty_like(sy), torch.empty_like(sg)
    ops.unpermute_backward(dout, f2r, w, T, K, H, y=y, dy=dy, d_weights=dw, shared_y=sy, shared_gate=sg,
                           d_shared_y=dsy, d_shared_gate=dsg)
    token, rows = torch.arange(T, device="cuda").repeat_interleave(K), f2r.long()
    for i in range(0, T * K, 1 << 14):  # a product's one rounding, and bf16's
        part = slice(i, i + (1 << 14))
        d = dout[token[part]]
        assert torch.equal(dy[rows[part]], (w.view(-1, 1)[part] * d.float()).to(b))
        yd = y[rows[part]].double() * d.double()
        assert ((dw.view(-1)[part] - yd.sum(1)).abs() <= 96 * U * yd.abs().sum(1)).all()
    assert torch.equal(dsy, (sg[:, None] * dout.float()).to(b))
    sd = sy.double() * dout.double()
    assert ((dsg - sd.sum(1)).abs() <= 96 * U * sd.abs().sum(1)).all()


# ------------------------------------------------------------------ the largest counts
def test_norm_gradient_of_the_most_rows(ops):  # noqa: F811
    """T = 2^31 - 1: the number of row groups has to be formed without T + rows - 1."""
    torch.cuda.empty_cache()
    T, H = 2 ** 31 - 1, 16
    g = torch.Generator("cuda").manual_seed(0)
    h = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    dx = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")  # dy, and dx over it
    rstd = torch.ones(T, device="cuda")
    rows = [0, 5, 1 << 20, (1 << 30) + 3, T - 17, T - 2, T - 1]
    sh, sdy = (torch.randn(len(rows), H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.ones(H, device="cuda")
    h[rows], dx[rows] = sh, sdy
    dw, dw2, sdx = torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty_like(sh)
    scratch = torch.empty(ops.add_rmsnorm_backward_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")
    ops.add_rmsnorm_backward(dx, h, rstd, w, dx, dw, scratch)
    ops.add_rmsnorm_backward(sdy, sh, torch.ones(len(rows), device="cuda"), w, sdx, dw2, scratch)
    assert torch.equal(dx[rows], sdx)
    # seven products and their sum, in either order
    terms = (sdy.double() * sh.double()).abs().sum(0)
    assert ((dw.double() - dw2.double()).abs() <= 16 * U * terms).all()
    del h, dx, rstd
    torch.cuda.empty_cache()


def test_losses_of_the_most_empty_sequences(ops):  # noqa: F811
    """n_seq = 2^31 - 1 without a token: valid has n_seq + 2 entries, past the largest int."""
    torch.cuda.empty_cache()
    S = 2 ** 31 - 1
    c, p = torch.full((S,), -9, dtype=torch.int32, device="cuda"), torch.full((S,), -9.0, device="cuda")
    v, lo = torch.full((S + 2,), -9, dtype=torch.int32, device="cuda"), torch.full((2,), -9.0, device="cuda")
    scratch = torch.empty(ops.balance_loss_scratch_bytes(0, 1, S), dtype=torch.uint8, device="cuda")  # not read at T = 0
    ops.balance_loss(torch.empty(0, 1, device="cuda"), torch.empty(0, 1, dtype=torch.int32, device="cuda"), 1, c, p, v,
                     lo, scratch, n_seq=S)
    for t in (c, p, v, lo):
        for part in t.split(1 << 28):
            assert not part.any()
    del c, p, v, scratch, t, part
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ router: an infinite logit
@pytest.mark.parametrize("E", [5, 40, 600])
def test_router_row_with_an_infinite_logit(ops, E):  # noqa: F811
    """+inf is a NaN to the softmax and a sigmoid of 1; the other sequence does not see it."""
    S, L, K = 2, 16, 3
    g = np.random.default_rng(E)
    l = g.normal(size=(S * L, E)).astype(np.float32)
    ids = np.argsort(-l, axis=1)[:, :K].astype(np.int32)
    big, inf = l.copy(), l.copy()
    big[5, 2], inf[5, 2] = 200.0, np.inf
    for mode in (0, 1):
        c0, p0, v0, lo0 = balance(ops, f32(big), i32(ids), None, E, S, mode)
        c1, p1, v1, lo1 = balance(ops, f32(inf), i32(ids), None, E, S, mode)
        assert torch.equal(c0, c1) and torch.equal(v0, v1) and torch.equal(p0[1], p1[1]) and lo1[1].isnan()
        if mode == 0:
            assert p1[0].isnan().all() and lo1[0].isnan()
        else:
            assert torch.equal(p0, p1) and lo0[0] == lo1[0]
        out = [torch.empty(S * L, E, device="cuda") for _ in range(2)]
        for o, a in zip(out, (big, inf)):
            ops.route_backward(f32(a), i32(ids), E, o, mode=mode, n_seq=S, counts=c0, valid=v0, grad_losses=f32([1.0, 0.0]))
        rest = [t for t in range(S * L) if t != 5]
        assert torch.equal(out[0][rest], out[1][rest])
        assert torch.equal(out[0][5], out[1][5]) if mode else out[1][5].isnan().all()
