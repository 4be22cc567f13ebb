"""GPU: the operators around the layer against the float64 oracle.

Tolerances, in units of u = 2^-24 (fp32 half step) and B = 2^-8 (bf16 half
step, relative), derived from how the values come about:
* an fp32 sum of n terms in chains of at most c additions and a tree errs by at
  most (c + 16) u times the sum of the terms' magnitudes; the kernels' chains
  are at most 64 columns per thread and, over tokens, the rows one thread or
  one block slot takes (T / 152 + 64 covers both);
* rstd: half the relative error of the mean square, (64 + 16) u / 2, and its own
  rounding: 2^-18 covers it; y adds two products, then B |y|;
* exp(l - max): |l - max| u for the difference's rounding scaled by the
  argument, and 4 u; a probability has that twice (numerator, sum) plus the
  sum's own error: (2 range + 160) u with range = max |l - max| over the row;
* e4m3: half a step is 2^-4 relative, 2^-10 for subnormal codes; the value
  before rounding carries y's and the scale's 2^-17.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixture_experts_layer_07_gb300 import build
    build.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()}/{bad.size} out of tolerance, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g}x")


# ------------------------------------------------------------------ norm
def norm_inputs(T, H, residual, seed, wdt=torch.bfloat16):
    g = np.random.default_rng(seed)
    x = bf(g.normal(size=(T, H)) * np.exp(g.normal(size=(T, 1))))
    r = bf(g.normal(size=(T, H))) if residual else None
    w = f32(1 + 0.2 * g.normal(size=H)).to(wdt)
    return x, r, w


def run_norm(ops, x, r, w, q=None, eps=EPS):
    T, H = x.shape
    o = {"y": torch.empty_like(x), "rstd": torch.empty(T, device="cuda")}
    o["h"] = torch.empty_like(x) if r is not None else None
    o["yq"] = o["yq_scale"] = None
    if q is not None:
        o["yq"] = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        o["yq_scale"] = torch.full((T, -(-H // 128) if q else 1), -1.0, device="cuda")
    ops.add_rmsnorm(x, w, eps, o["y"], residual=r, h=o["h"], rstd=o["rstd"], yq=o["yq"],
                    yq_scale=o["yq_scale"], q_group=128 if q is None else q)
    torch.cuda.synchronize()
    return o


def check_norm(o, x, r, w, q=None):
    h, y, rstd = bo.rmsnorm(f64(x), None if r is None else f64(r), f64(w), EPS)
    within(f64(o["rstd"]), rstd, 2.0 ** -18 * rstd, "rstd")
    within(f64(o["y"]), y, (B + 2.0 ** -16) * np.abs(y) + 1e-38, "y")
    if r is not None:
        within(f64(o["h"]), h, (B + 2.0 ** -16) * np.abs(h) + 1e-38, "h")
    if q is not None:
        H = x.shape[1]
        group = q or H
        s = bo.group_scales(y, group)
        within(f64(o["yq_scale"]), s, 2.0 ** -17 * s, "yq_scale")
        u = y / np.repeat(s, group, axis=1)[:, :H]
        within(f64(o["yq"].float()), u, (2.0 ** -4 + 2.0 ** -14) * np.abs(u) + 2.0 ** -10, "yq")


# H around every change of shape: one warp, half groups, several warps, eight vectors per thread
SIZES = [(1, 16), (1, 2048), (3, 128), (7, 144), (9, 256), (17, 272), (5, 512), (33, 528), (2, 1024),
         (5, 1040), (257, 2048), (31, 2880), (4, 7168), (3, 8192), (2, 8208), (1, 16400), (2, 32768)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_matches_oracle(ops, T, H, residual):
    for q, wdt in ((None, torch.bfloat16), (128, torch.float32), (0, torch.bfloat16)):
        x, r, w = norm_inputs(T, H, residual, T + H, wdt)
        check_norm(run_norm(ops, x, r, w, q), x, r, w, q)


@pytest.mark.parametrize("H", [256, 2880])
def test_norm_zero_nan_and_infinite_rows(ops, H):
    x, r, w = norm_inputs(5, H, True, 3)
    x[1], r[1] = 0, 0
    x[2, 7] = float("nan")
    x[3, H - 1] = float("inf")
    clean_x, clean_r = x[[0, 4]].contiguous(), r[[0, 4]].contiguous()
    for q in (128, 0):
        o = run_norm(ops, x, r, w, q)
        ref = run_norm(ops, clean_x, clean_r, w, q)
        for k in ("y", "h", "rstd", "yq_scale"):
            assert torch.equal(o[k][[0, 4]], ref[k]), k
        assert (o["y"][1] == 0).all() and (o["yq_scale"][1] == 0).all() and (o["yq"][1].float() == 0).all()
        for row in (2, 3):
            assert o["yq_scale"][row].isnan().any() and o["yq"][row].float().isnan().any()
            assert o["y"][row].isnan().any()


def test_norm_in_place_and_single_outputs(ops):
    x, r, w = norm_inputs(37, 2880, True, 4)
    ref = run_norm(ops, x, r, w, 128)
    # h over the residual, y over x
    x2, r2 = x.clone(), r.clone()
    ops.add_rmsnorm(x2, w, EPS, x2, residual=r2, h=r2)
    assert torch.equal(x2, ref["y"]) and torch.equal(r2, ref["h"])
    # h over x
    x3 = x.clone()
    y = torch.empty_like(x)
    ops.add_rmsnorm(x3, w, EPS, y, residual=r, h=x3)
    assert torch.equal(x3, ref["h"]) and torch.equal(y, ref["y"])
    # codes alone
    yq, ys = torch.empty(37, 2880, dtype=torch.uint8, device="cuda"), torch.empty(37, 23, device="cuda")
    ops.add_rmsnorm(x, w, EPS, None, residual=r, yq=yq, yq_scale=ys)
    assert torch.equal(yq, ref["yq"].view(torch.uint8)) and torch.equal(ys, ref["yq_scale"])


@pytest.mark.parametrize("magnitude", [1.0, 1e-30, 1e28])
@pytest.mark.parametrize("q", [128, 0])
def test_norm_codes_are_those_of_ieee_division(ops, magnitude, q):
    # the kernel's own fp32 operations, one by one: y = (h s) w, scale = amax / 448, y / scale
    T, H = 67, 2000
    x, r, w = norm_inputs(T, H, True, 21, torch.float32)
    w = w * magnitude  # scales far outside 2^+-80 take the division itself
    o = run_norm(ops, x, r, w, q)
    y = ((x.float() + r.float()) * o["rstd"][:, None]) * w
    group = q or H
    n = -(-H // group)
    p = torch.zeros(T, n * group, device="cuda")
    p[:, :H] = y
    m = p.view(T, n, group).abs().amax(2)
    scale = m / torch.full_like(m, 448.0)
    assert torch.equal(o["yq_scale"], scale)
    code = (p.view(T, n, group) / scale[..., None].expand(T, n, group)).view(T, n * group)[:, :H]
    assert torch.equal(o["yq"].view(torch.uint8), code.to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("H", [256, 272, 528, 1040, 2048, 2880, 8192, 8208, 16400, 32768])
def test_norm_of_a_row_does_not_depend_on_the_batch(ops, H):
    x, r, w = norm_inputs(400, H, True, H)
    whole = run_norm(ops, x, r, w, 128)
    for a, b in ((0, 1), (17, 20), (100, 400)):
        part = run_norm(ops, x[a:b].contiguous(), r[a:b].contiguous(), w, 128)
        for k in ("y", "h", "rstd", "yq_scale"):
            assert torch.equal(part[k], whole[k][a:b]), k
        assert torch.equal(part["yq"].view(torch.uint8), whole["yq"][a:b].view(torch.uint8))


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_backward_matches_oracle(ops, T, H, with_dh):
    for wdt in (torch.bfloat16, torch.float32):
        g = np.random.default_rng(T * H)
        h, _, w = norm_inputs(T, H, False, T + H + 1, wdt)
        dy = bf(g.normal(size=(T, H)))
        dh = bf(g.normal(size=(T, H))) if with_dh else None
        run_norm_backward(ops, h, w, dy, dh)


def run_norm_backward(ops, h, w, dy, dh):
    T, H = h.shape
    hh = f64(h)
    rstd64 = 1 / np.sqrt((hh * hh).mean(axis=1) + EPS)
    rstd = f32(rstd64)
    dx, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    s = torch.full((ops.add_rmsnorm_backward_scratch_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.add_rmsnorm_backward(dy, h, rstd, w, dx, dw, s, dh=dh)
    first = dx.clone(), dw.clone()
    ops.add_rmsnorm_backward(dy, h, rstd, w, dx, dw, s, dh=dh)
    torch.cuda.synchronize()
    assert torch.equal(first[0], dx) and torch.equal(first[1], dw)  # the same order every time
    rx, rw = bo.rmsnorm_backward(f64(dy), None if dh is None else f64(dh), hh, f64(w), EPS)
    n, gw = hh * rstd64[:, None], f64(dy) * f64(w)
    c_abs = np.abs(gw * n).mean(axis=1, keepdims=True)
    terms = rstd64[:, None] * (np.abs(gw) + np.abs(n) * c_abs) + (0 if dh is None else np.abs(f64(dh)))
    within(f64(dx), rx, B * np.abs(rx) + 96 * U * terms, "dx")
    within(f64(dw), rw, (T / 152 + 64 + 16) * U * (np.abs(f64(dy) * n)).sum(axis=0) + 1e-30, "dweight")


def test_norm_backward_many_rows_and_in_place(ops):
    h, _, w = norm_inputs(3001, 528, False, 8)
    g = np.random.default_rng(1)
    dy, dh = bf(g.normal(size=(3001, 528))), bf(g.normal(size=(3001, 528)))
    run_norm_backward(ops, h, w, dy, dh)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    s = torch.empty(ops.add_rmsnorm_backward_scratch_bytes(3001, 528), dtype=torch.uint8, device="cuda")
    dw = torch.empty(528, device="cuda")
    ref = torch.empty_like(h)
    ops.add_rmsnorm_backward(dy, h, rstd, w, ref, dw, s, dh=dh)
    a, b = dy.clone(), dh.clone()
    ops.add_rmsnorm_backward(a, h, rstd, w, a, dw, s, dh=dh)
    ops.add_rmsnorm_backward(dy, h, rstd, w, b, dw, s, dh=b)
    assert torch.equal(a, ref) and torch.equal(b, ref)


def test_norm_backward_without_rows_clears_dweight(ops):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64,), 7.0, device="cuda")
    ops.add_rmsnorm_backward(e, e, torch.empty(0, device="cuda"), torch.ones(64, device="cuda"), e, dw,
                             torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert (dw == 0).all()


def test_norm_gradient_is_the_difference_quotient(ops):
    # the oracle's forward in 64 bits, the kernel's gradient: the bf16 rounding
    # of dx (B) dominates the difference quotient's own error
    g = np.random.default_rng(5)
    h, _, w = norm_inputs(2, 32, False, 6, torch.float32)
    dy = bf(g.normal(size=(2, 32)))
    dx, dw = torch.empty_like(h), torch.empty(32, device="cuda")
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    ops.add_rmsnorm_backward(dy, h, rstd, w, dx, dw,
                             torch.empty(ops.add_rmsnorm_backward_scratch_bytes(2, 32), dtype=torch.uint8,
                                         device="cuda"))
    f = lambda hh, ww: (bo.rmsnorm(hh, None, ww, EPS)[1] * f64(dy)).sum()  # noqa: E731
    hh, ww, step = f64(h), f64(w), 1e-5
    nx, nw = np.zeros_like(hh), np.zeros_like(ww)
    for i in np.ndindex(hh.shape):
        a, b = hh.copy(), hh.copy()
        a[i] += step
        b[i] -= step
        nx[i] = (f(a, ww) - f(b, ww)) / (2 * step)
    for i in range(32):
        a, b = ww.copy(), ww.copy()
        a[i] += step
        b[i] -= step
        nw[i] = (f(hh, a) - f(hh, b)) / (2 * step)
    within(f64(dx), nx, B * np.abs(nx) + 1e-5, "dx")
    within(f64(dw), nw, 1e-5 * np.abs(nw) + 1e-5, "dweight")


def test_norm_offsets_past_32_bits(ops):
    T, H = 300000, 8192  # 2.4e9 elements
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rows = [0, 131072, 262144, 262145, T - 1]
    some, _, w = norm_inputs(len(rows), H, False, 9)
    x[rows] = some
    y, yq = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device="cuda")
    ys, rstd = torch.empty(T, 64, device="cuda"), torch.empty(T, device="cuda")
    ops.add_rmsnorm(x, w, EPS, y, rstd=rstd, yq=yq, yq_scale=ys)
    ref = run_norm(ops, some, None, w, 128)
    assert torch.equal(y[rows], ref["y"]) and torch.equal(ys[rows], ref["yq_scale"])
    assert torch.equal(yq[rows], ref["yq"].view(torch.uint8)) and torch.equal(rstd[rows], ref["rstd"])
    dw = torch.empty(H, device="cuda")
    s = torch.empty(ops.add_rmsnorm_backward_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")
    ops.add_rmsnorm_backward(x, x, rstd, w, y, dw, s)
    d2, w2 = torch.empty_like(some), torch.empty(H, device="cuda")
    ops.add_rmsnorm_backward(some, some, rstd[rows].contiguous(), w, d2, w2, s)
    assert torch.equal(y[rows], d2)
    n = f64(some) * f64(rstd[rows])[:, None]
    within(f64(dw), (f64(some) * n).sum(0), (T / 152 + 80) * U * np.abs(f64(some) * n).sum(0), "dweight")


# ------------------------------------------------------------------ router
def router_case(S, L, E, K, mode, shared, mask, seed, kind="plain"):
    g = np.random.default_rng(seed)
    T = S * L
    l = (g.normal(size=(T, E + shared)) * 2).astype(np.float32)
    if kind == "masked":        # experts switched off: -inf, and the type's lowest value
        l[:, : E // 2] = np.where(g.random((T, E // 2)) < 0.5, -np.inf, l[:, : E // 2])
        if E > 2:
            l[::3, E - 1] = np.finfo(np.float32).min
    elif kind == "very_negative":
        l -= 300.0
    elif kind == "large":
        l *= 40.0
    sel = l[:, :E] if mode == 0 else l[:, :E] + 0.1 * g.normal(size=(T, E)).astype(np.float32)
    ids = np.argsort(-sel, axis=1, kind="stable")[:, :K].astype(np.int32)
    m = None
    if mask == "tail":
        m = (np.arange(L)[None] < g.integers(0, L + 1, size=(S, 1))).astype(np.uint8).ravel()
    elif mask == "scattered":
        m = (g.random(T) < 0.5).astype(np.uint8) * 255
    elif mask == "none_left":
        m = np.zeros(T, np.uint8)
    elif mask == "one_sequence":
        m = np.zeros((S, L), np.uint8)
        m[S - 1, L - 1] = 1
        m = m.ravel()
    if m is not None:  # what the mask leaves out may hold anything
        l[m == 0] = np.nan
        ids[m == 0] = -77
    return l, ids, m


def balance(ops, l, ids, m, E, S, mode, scratch=None, status=None):
    T = l.shape[0]
    c, p = torch.full((S, E), -9, dtype=torch.int32, device="cuda"), torch.full((S, E), -9.0, device="cuda")
    v, lo = torch.full((S + 2,), -9, dtype=torch.int32, device="cuda"), torch.full((2,), -9.0, device="cuda")
    if scratch is None:
        scratch = torch.zeros(ops.balance_loss_scratch_bytes(T, E, S), dtype=torch.uint8, device="cuda")
    ops.balance_loss(l, ids, E, c, p, v, lo, scratch, n_seq=S, mode=mode, token_mask=m, dev_status=status)
    torch.cuda.synchronize()
    assert not scratch.any(), "the scratch is zero again"
    return c, p, v, lo


def row_range(l, E, keep):
    with np.errstate(invalid="ignore"):
        x = l[keep, :E].astype(np.float64)
        x = np.where(np.isfinite(x) & (x > -1e30), x, np.nan)
        r = np.nanmax(x, axis=1) - np.nanmin(x, axis=1) if x.size else np.zeros(1)
    return float(np.nanmax(r, initial=0.0)) + float(np.nanmax(np.abs(x), initial=0.0) if x.size else 0.0)


ROUTER = [  # S, L, E, K, mode, shared, mask, kind
    (1, 1, 1, 1, 0, 0, None, "plain"), (1, 1, 8, 2, 1, 1, None, "plain"), (3, 1, 33, 32, 0, 0, "scattered", "plain"),
    (4, 25, 8, 2, 0, 1, "tail", "plain"), (2, 77, 17, 4, 1, 0, "tail", "plain"), (5, 40, 64, 6, 0, 0, "one_sequence", "plain"),
    (1, 300, 128, 8, 0, 1, None, "plain"), (1, 300, 127, 8, 1, 0, "scattered", "plain"),
    (7, 13, 256, 8, 0, 0, "tail", "plain"), (2, 64, 257, 9, 1, 1, "none_left", "plain"),
    (3, 50, 512, 10, 0, 1, "tail", "plain"), (2, 30, 896, 16, 1, 0, "scattered", "plain"),
    (1, 40, 1024, 32, 0, 0, None, "plain"), (1, 2, 1023, 3, 1, 1, None, "plain"),
    (2, 40, 32, 4, 0, 0, "scattered", "masked"), (2, 40, 128, 8, 1, 0, None, "masked"),
    (2, 40, 64, 4, 0, 1, "tail", "very_negative"), (2, 40, 64, 4, 1, 0, None, "very_negative"),
    (1, 60, 128, 8, 0, 0, None, "large"), (1, 60, 128, 8, 1, 0, "tail", "large"),
    (700, 3, 16, 2, 0, 0, "scattered", "plain")]


@pytest.mark.parametrize("S,L,E,K,mode,shared,mask,kind", ROUTER)
def test_balance_loss_matches_oracle(ops, S, L, E, K, mode, shared, mask, kind):
    l, ids, m = router_case(S, L, E, K, mode, shared, mask, S * L + E, kind)
    keep = np.ones(S * L, bool) if m is None else m != 0
    ref = bo.balance(l, ids, m, E, S, mode)
    dm = None if m is None else torch.from_numpy(m).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c, p, v, lo = balance(ops, f32(l), i32(ids), dm, E, S, mode, status=st)
    assert int(st) == 0
    assert np.array_equal(c.cpu().numpy(), ref["counts"]) and np.array_equal(v.cpu().numpy(), ref["valid"])
    rel = (2 * row_range(l, E, keep) + 160 + S * L / 152) * U
    # the fixed-point sum of a block is off by at most half of 2^-(61 - 31)
    within(f64(p), ref["mean_prob"], rel * ref["mean_prob"] + 2.0 ** -30, "mean_prob")
    within(f64(lo)[0], ref["losses"][0], rel * ref["losses"][0] + E * 2.0 ** -30, "balance loss")
    # lse = m + log(sum): a half step of its own and the sum's relative error
    z = ref["losses"][1]
    within(f64(lo)[1], z, 4 * U * z + 2 * rel * np.sqrt(z) + S * L / 152 * U * z + rel * rel, "z loss")


@pytest.mark.parametrize("S,L,E,K,mode,shared,mask,kind", ROUTER)
@pytest.mark.parametrize("parts", ["all", "losses", "weights", "gate"])
def test_route_backward_matches_oracle(ops, S, L, E, K, mode, shared, mask, kind, parts):
    l, ids, m = router_case(S, L, E, K, mode, shared, mask, S * L + E + 1, kind)
    T = S * L
    g = np.random.default_rng(E)
    scale = 1.0 if mode == 0 else 2.5
    keep = np.ones(T, bool) if m is None else m != 0
    w = np.full((T, K), np.nan, np.float32)
    w[keep] = bo.routing_weights(l[keep], ids[keep], mode, scale)
    gw = g.normal(size=(T, K)).astype(np.float32) if parts in ("all", "weights") else None
    gs = g.normal(size=T).astype(np.float32) if shared and parts in ("all", "gate") else None
    gl = np.array([0.6, 0.05], np.float32) if parts in ("all", "losses") else None
    dm = None if m is None else torch.from_numpy(m).cuda()
    dl, di = f32(l), i32(ids)
    c, _, v, _ = balance(ops, dl, di, dm, E, S, mode)
    ld = E + shared + 3  # wider rows: the rest stays as it is
    out = torch.full((T, ld), -5.0, device="cuda")
    opt = lambda a: None if a is None else f32(a)  # noqa: E731
    ops.route_backward(dl, di, E, out, mode=mode, scale=scale, weights=f32(w), d_weights=opt(gw),
                       d_shared_gate=opt(gs), token_mask=dm, n_seq=S, counts=c, valid=v, grad_losses=opt(gl))
    torch.cuda.synchronize()
    cols = E + (gs is not None)
    assert (out[:, cols:] == -5.0).all()
    got = f64(out)[:, :cols]
    ref = bo.route_backward(l, ids, w, gw, gs, m, E, S, mode, scale, gl)
    # magnitudes of the terms that a row adds up
    mag = np.zeros((T, cols))
    if gl is not None:
        vv = v.cpu().numpy()
        for t in np.flatnonzero(keep):
            n = vv[t // L]
            a = abs(gl[0]) * E * c.cpu().numpy()[t // L] / (K * n * n * vv[-1])
            p = bo.probabilities(l[t:t + 1, :E], mode)[0]
            q, lse = bo._normalise(l[t:t + 1, :E].astype(np.float64))
            mag[t, :E] = p * (a + (a * p).sum()) + 2 * gl[1] * (np.abs(lse[0]) + 1) * q[0] / vv[-2]
    if gw is not None:
        for t in np.flatnonzero(keep):
            tot = (w[t] * np.abs(gw[t])).sum()
            for k in range(K):
                mag[t, ids[t, k]] += abs(w[t, k]) * (abs(gw[t, k]) + tot / scale)
    if gs is not None:
        mag[:, E] = np.abs(gs)
    rel = (3 * row_range(l, E, keep) + 256) * U
    within(got, ref, rel * mag + 1e-30, "dlogits")
    assert (got[~keep] == 0).all()


@pytest.mark.parametrize("mode", [0, 1])
def test_route_gradient_is_the_difference_quotient(ops, mode):
    S, L, E, K, scale = 2, 4, 6, 3, (1.0 if mode == 0 else 1.7)
    g = np.random.default_rng(11)
    l = g.normal(size=(S * L, E + 1)).astype(np.float32)
    ids = np.argsort(-l[:, :E], axis=1)[:, :K].astype(np.int32)
    m = np.array([1, 1, 1, 0, 1, 0, 0, 0], np.uint8)
    gw, gs = g.normal(size=(S * L, K)).astype(np.float32), g.normal(size=S * L).astype(np.float32)
    gl = np.array([0.8, 0.1], np.float32)

    def f(v):
        w = bo.routing_weights(v, ids, mode, scale)
        b = bo.balance(v, ids, m, E, S, mode)["losses"]
        return ((w * gw).sum(1) + gs / (1 + np.exp(-v[:, E])))[m != 0].sum() + (gl * b).sum()

    x = l.astype(np.float64)
    num = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += 1e-5
        b[i] -= 1e-5
        num[i] = (f(a) - f(b)) / 2e-5
    dl, di, dm = f32(l), i32(ids), torch.from_numpy(m).cuda()
    c, _, v, _ = balance(ops, dl, di, dm, E, S, mode)
    out = torch.empty(S * L, E + 1, device="cuda")
    ops.route_backward(dl, di, E, out, mode=mode, scale=scale, weights=f32(bo.routing_weights(l, ids, mode, scale)),
                       d_weights=f32(gw), d_shared_gate=f32(gs), token_mask=dm, n_seq=S, counts=c, valid=v,
                       grad_losses=f32(gl))
    within(f64(out), num, np.full(num.shape, 1e-6), "dlogits")


@pytest.mark.parametrize("mode", [0, 1])
def test_router_rows_without_an_expert_and_nan_rows(ops, mode):
    E, K = 40, 4
    l, ids, _ = router_case(2, 16, E, K, mode, 0, None, 5)
    l[3] = -np.inf
    ref = bo.balance(l, ids, None, E, 2, mode)
    c, p, v, lo = balance(ops, f32(l), i32(ids), None, E, 2, mode)
    within(f64(p), ref["mean_prob"], 400 * U * ref["mean_prob"] + 2.0 ** -30, "mean_prob")
    within(f64(lo), ref["losses"], 400 * U * np.abs(ref["losses"]), "losses")
    out = torch.empty(32, E, device="cuda")
    ops.route_backward(f32(l), i32(ids), E, out, mode=mode, n_seq=2, counts=c, valid=v, grad_losses=f32([1, 1]))
    assert (out[3] == 0).all() and out.isfinite().all()
    l[20, 7] = np.nan  # a kept NaN reaches its sequence and the losses, and no other sequence
    c, p, v, lo = balance(ops, f32(l), i32(ids), None, E, 2, mode)
    assert p[1].isnan().all() and p[0].isfinite().all() and lo.isnan().all()


def test_router_ids_out_of_range_are_dropped_and_reported(ops):
    l, ids, _ = router_case(1, 50, 16, 3, 0, 0, None, 6)
    ids[7, 1], ids[30, 0] = 16, -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c, p, v, lo = balance(ops, f32(l), i32(ids), None, 16, 1, 0, status=st)
    ref = bo.balance(l, ids, None, 16, 1, 0)
    assert int(st) == ops.DEV_BAD_EXPERT_ID and np.array_equal(c.cpu().numpy(), ref["counts"])
    g = np.random.default_rng(0).normal(size=(50, 3)).astype(np.float32)
    w = np.full((50, 3), 1 / 3, np.float32)
    st.zero_()
    out = torch.empty(50, 16, device="cuda")
    ops.route_backward(f32(l), i32(ids), 16, out, weights=f32(w), d_weights=f32(g), dev_status=st)
    within(f64(out), bo.route_backward(l, ids, w, g, None, None, 16, 1, 0, 1.0, None), 64 * U * 10, "dlogits")
    assert int(st) == ops.DEV_BAD_EXPERT_ID


def test_router_repeated_ids_add_up(ops):
    l, ids, _ = router_case(1, 9, 8, 6, 0, 0, None, 7)
    ids[:, 1:5] = ids[:, :1]
    g = np.random.default_rng(1).normal(size=(9, 6)).astype(np.float32)
    w = np.full((9, 6), 1 / 6, np.float32)
    out = [torch.empty(9, 8, device="cuda") for _ in range(2)]
    for o in out:
        ops.route_backward(f32(l), i32(ids), 8, o, weights=f32(w), d_weights=f32(g))
    assert torch.equal(*out)
    within(f64(out[0]), bo.route_backward(l, ids, w, g, None, None, 8, 1, 0, 1.0, None), 64 * U * 10, "dlogits")


def test_balance_of_no_tokens_and_of_shared_scratch(ops):
    E = 24
    e = torch.empty(0, E, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    c, p, v, lo = balance(ops, *e, None, E, 3, 0)
    assert not c.any() and not p.any() and not v.any() and not lo.any()
    # calls of other sizes on one scratch, each as on its own
    cases = [router_case(S, L, E2, 2, mode, 0, "scattered", S + L) + (E2, S, mode)
             for S, L, E2, mode in ((1, 5000, 128, 0), (9, 70, 16, 1), (3, 1, 1000, 0), (1, 5000, 128, 1))]
    big = torch.zeros(max(ops.balance_loss_scratch_bytes(len(l), E2, S) for l, _, _, E2, S, _ in cases),
                      dtype=torch.uint8, device="cuda")
    for l, ids, m, E2, S, mode in cases:
        args = (f32(l), i32(ids), torch.from_numpy(m).cuda(), E2, S, mode)
        for a, b in zip(balance(ops, *args, scratch=big), balance(ops, *args)):
            assert torch.equal(a, b)


def test_balance_is_the_same_every_time(ops):
    g = torch.Generator("cuda").manual_seed(1)
    l = torch.randn(20000, 200, device="cuda", generator=g)
    ids = l.topk(6, dim=1).indices.to(torch.int32)
    first = balance(ops, l, ids, None, 200, 4, 1)
    for _ in range(5):
        for a, b in zip(first, balance(ops, l, ids, None, 200, 4, 1)):
            assert torch.equal(a, b)


def test_router_offsets_past_32_bits(ops):
    T, E, K = 2200000, 1024, 2  # 2.25e9 logits
    l = torch.full((T, E), -20.0, device="cuda")
    rows = [0, 2097151, 2097152, T - 1]
    sub = torch.randn(len(rows), E, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    l[rows] = sub
    m = torch.zeros(T, dtype=torch.uint8, device="cuda")
    m[rows] = 1
    ids = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    ids[rows] = sub.topk(K, dim=1).indices.to(torch.int32)
    c, p, v, lo = balance(ops, l, ids, m, E, 1, 0)
    ref = bo.balance(sub.cpu().numpy(), ids[rows].cpu().numpy(), None, E, 1, 0)
    assert np.array_equal(c.cpu().numpy(), ref["counts"]) and int(v[1]) == len(rows)
    within(f64(p), ref["mean_prob"], 400 * U * ref["mean_prob"] + 2.0 ** -30, "mean_prob")
    gl = f32([1.0, 1.0])
    out = torch.full((T, E), 3.0, device="cuda")
    ops.route_backward(l, ids, E, out, token_mask=m, counts=c, valid=v, grad_losses=gl)
    small = torch.empty(len(rows), E, device="cuda")
    ops.route_backward(sub, ids[rows].contiguous(), E, small, counts=c, valid=v, grad_losses=gl)
    assert torch.equal(out[rows], small)
    out[rows] = 0
    assert not out.any()


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 8, 2048), (3, 2, 256), (5, 32, 520), (17, 4, 2880), (9, 10, 1032),
                                   (2, 3, 7168), (2, 5, 8200), (1, 2, 32768), (300, 6, 64)])
@pytest.mark.parametrize("shared", [False, True])
def test_unpermute_backward_matches_oracle(ops, T, K, H, shared):
    g = np.random.default_rng(T * K + H)
    dout, y = bf(g.normal(size=(T, H))), bf(g.normal(size=(T * K, H)))
    w = f32(g.normal(size=(T, K)))
    f2r = g.permutation(T * K).astype(np.int32)
    if T * K > 4:  # dropped replicas, and a row that does not exist
        f2r[[1, T * K - 1]] = [-1, T * K]
    sy, sg = (bf(g.normal(size=(T, H))), f32(g.normal(size=T))) if shared else (None, None)
    dy = torch.full_like(y, 3.0)
    dw = torch.full_like(w, 3.0)
    dsy, dsg = (torch.empty_like(sy), torch.empty_like(sg)) if shared else (None, None)
    ops.unpermute_backward(dout, i32(f2r), w, T, K, H, y=y, dy=dy, d_weights=dw, shared_y=sy, shared_gate=sg,
                           d_shared_y=dsy, d_shared_gate=dsg)
    torch.cuda.synchronize()
    ref = bo.unpermute_backward(f64(dout), f64(y), f2r, w.cpu().numpy(), None if sy is None else f64(sy),
                                None if sg is None else f64(sg))
    untouched = np.isnan(ref["dy"])
    want = np.where(untouched, 3.0, ref["dy"])
    within(f64(dy), want, (B + 2 * U) * np.abs(want) * ~untouched, "dy")
    abs_dot = np.zeros((T, K))
    for i, r in enumerate(f2r):
        if 0 <= r < T * K:
            abs_dot[i // K, i % K] = np.abs(f64(dout)[i // K] * f64(y)[r]).sum()
    within(f64(dw), ref["d_weights"], 96 * U * abs_dot, "d_weights")
    if shared:
        within(f64(dsy), ref["d_shared_y"], (B + 2 * U) * np.abs(ref["d_shared_y"]), "d_shared_y")
        within(f64(dsg), ref["d_shared_gate"], 96 * U * np.abs(f64(dout) * f64(sy)).sum(1), "d_shared_gate")
    # each output alone, and in place
    one = torch.empty_like(w)
    ops.unpermute_backward(dout, i32(f2r), None, T, K, H, y=y, d_weights=one)
    assert torch.equal(one, dw)
    alone = torch.full_like(y, 3.0)
    ops.unpermute_backward(dout, i32(f2r), w, T, K, H, dy=alone)
    assert torch.equal(alone, dy)
    over = y.clone()
    ops.unpermute_backward(dout, i32(f2r), w, T, K, H, y=over, dy=over, d_weights=one)
    assert torch.equal(one, dw) and np.array_equal(f64(over)[~untouched], f64(dy)[~untouched])
    if shared:
        a, b = torch.empty_like(sg), torch.empty_like(sy)
        ops.unpermute_backward(dout, i32(f2r), None, T, K, H, shared_y=sy, d_shared_gate=a)
        ops.unpermute_backward(dout, i32(f2r), None, T, K, H, shared_gate=sg, d_shared_y=b)
        assert torch.equal(a, dsg) and torch.equal(b, dsy)


def test_unpermute_backward_is_the_gradient_of_unpermute(ops):
    # the combine is linear in y and in the weights: out(y + e) - out(y) = <d, e>
    T, K, H = 6, 4, 256
    g = np.random.default_rng(3)
    y, dout = bf(g.normal(size=(T * K, H))), bf(g.normal(size=(T, H)))
    w = f32(g.normal(size=(T, K)))
    f2r = i32(g.permutation(T * K))
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    ops.unpermute_backward(dout, f2r, w, T, K, H, y=y, dy=dy, d_weights=dw)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ops.unpermute(y, f2r, w, T, K, H, out)
    lhs = (f64(dout) * f64(out)).sum()
    size = (np.abs(f64(dout)) * np.abs(f64(out))).sum()
    within((f64(w) * f64(dw)).sum(), lhs, B * size + 1e-4 * np.abs(f64(w) * f64(dw)).sum(), "<w, dw> = <dout, out>")
    within((f64(y) * f64(dy)).sum(), lhs, B * (size + np.abs(f64(y) * f64(dy)).sum()), "<y, dy> = <dout, out>")


# ------------------------------------------------------------------ streams and graphs
def test_operators_on_another_stream_and_in_a_graph(ops):
    T, H, E, K = 200, 2048, 64, 4
    x, r, w = norm_inputs(T, H, True, 12)
    l, ids, m = router_case(4, 50, E, K, 0, 0, "tail", 13)
    dl, di, dm = f32(np.nan_to_num(l)), i32(np.abs(ids) % E), torch.from_numpy(m).cuda()
    wt, gw, gl = torch.rand(T, K, device="cuda"), torch.randn(T, K, device="cuda"), f32([1.0, 0.1])
    y = torch.randn(T * K, H, device="cuda").to(torch.bfloat16)
    f2r = torch.randperm(T * K, device="cuda").to(torch.int32)
    bal = torch.zeros(ops.balance_loss_scratch_bytes(T, E, 4), dtype=torch.uint8, device="cuda")
    bwd = torch.empty(ops.add_rmsnorm_backward_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")

    def buffers():
        e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        b = torch.bfloat16
        return {"h": e(T, H, dt=b), "y": e(T, H, dt=b), "rstd": e(T), "yq": e(T, H, dt=torch.uint8), "ys": e(T, 16),
                "dx": e(T, H, dt=b), "dw": e(H), "c": e(4, E, dt=torch.int32), "p": e(4, E),
                "v": e(6, dt=torch.int32), "lo": e(2), "dl": e(T, E), "dy": e(T * K, H, dt=b), "dwt": e(T, K)}

    def step(o):
        ops.add_rmsnorm(x, w, EPS, o["y"], residual=r, h=o["h"], rstd=o["rstd"], yq=o["yq"], yq_scale=o["ys"])
        ops.balance_loss(dl, di, E, o["c"], o["p"], o["v"], o["lo"], bal, n_seq=4, token_mask=dm)
        ops.unpermute_backward(o["y"], f2r, wt, T, K, H, y=y, dy=o["dy"], d_weights=o["dwt"])
        ops.route_backward(dl, di, E, o["dl"], weights=wt, d_weights=gw, token_mask=dm, n_seq=4, counts=o["c"],
                           valid=o["v"], grad_losses=gl)
        ops.add_rmsnorm_backward(o["y"], o["h"], o["rstd"], w, o["dx"], o["dw"], bwd)

    ref, side, graphed = buffers(), buffers(), buffers()
    step(ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for _ in range(3):
        for t in graphed.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], side[k]), k
        assert torch.equal(ref[k], graphed[k]), k
