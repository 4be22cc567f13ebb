"""GPU: activations kept in 8 bits, and the norm's gradient from them, against the float64 oracle.

The scale is one correctly rounded division (2^-24 relative) and a code half a step from its
quotient (2^-4 relative, 2^-10 below the normal codes), which the scale's error moves by 2^-22
at most.  What the norm's gradient may be off is derived as for its bf16 form: the codes'
values are exact products in fp32 up to 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixture_experts_layer_07_gb300 import build
    build.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()}/{bad.size} out of tolerance, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g}x")


def rows(T, H, seed=0):
    g = np.random.default_rng(seed)
    x = g.normal(size=(T, H)) * np.exp(2 * g.normal(size=(T, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(BF16).cuda()


def pack(ops, x):
    T, H = x.shape
    xq = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    xs = torch.full((T, -(-H // 128)), -1.0, device="cuda")
    ops.pack_q8(x, xq, xs)
    return xq, xs


SIZES = [(1, 16), (1, 2048), (3, 128), (2, 144), (7, 272), (9, 1040), (257, 2880), (100, 96), (4, 7168), (2, 32784)]


@pytest.mark.parametrize("T,H", SIZES)
def test_pack_and_unpack_match_oracle(ops, T, H):
    x = rows(T, H, T + H)
    xq, xs = pack(ops, x)
    want, s = bo.pack_q8(f64(x))
    within(f64(xs), s, U * s, "scale")
    within(f64(xq.float()), want, (2.0 ** -4 + 2.0 ** -20) * np.abs(want) + 2.0 ** -10, "codes")
    back = torch.full_like(x, 7.0)
    ops.unpack_q8(xq, xs, back)
    wide = np.repeat(f64(xs), 128, axis=1)[:, :H]
    v = f64(xq.float()) * wide
    within(f64(back), v, (B + 2 * U) * np.abs(v), "unpacked")
    # packing what was unpacked keeps the largest value of a group, so its scale to bf16's rounding
    within(f64(pack(ops, back)[1]), s, (B + 4 * U) * s, "scale again")


@pytest.mark.parametrize("T,H", [(1, 256), (33, 528), (2, 8208), (65, 2880), (300, 1024), (2, 16400)])
@pytest.mark.parametrize("dh", [False, True])
def test_norm_backward_matches_oracle(ops, T, H, dh):
    g = np.random.default_rng(T)
    h = rows(T, H, H)
    hq, hs = pack(ops, h)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    w = torch.from_numpy((1 + 0.2 * g.normal(size=H)).astype(np.float32)).cuda().to(F32 if dh else BF16)
    dy = torch.from_numpy(g.normal(size=(T, H)).astype(np.float32)).to(BF16).cuda()
    e = torch.from_numpy(g.normal(size=(T, H)).astype(np.float32)).to(BF16).cuda() if dh else None
    dx, dw = torch.full_like(dy, 7.0), torch.full((H,), 7.0, device="cuda")
    scratch = torch.full((ops.add_rmsnorm_backward_scratch_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.add_rmsnorm_backward_q8(dy, hq, hs, rstd, w, dx, dw, scratch, dh=e)
    torch.cuda.synchronize()
    v = f64(hq.float()) * np.repeat(f64(hs), 128, axis=1)[:, :H]
    r = f64(rstd)[:, None]
    n, gw = v * r, f64(dy) * f64(w)
    want = r * (gw - n * (gw * n).mean(axis=1, keepdims=True)) + (f64(e) if dh else 0.0)
    # the dot product: chains of 64 columns at most and a tree, (64 + 16) u of the terms' sum
    dot = 96 * U * np.abs(gw * n).mean(axis=1, keepdims=True)
    off = r * (np.abs(n) * dot + 8 * U * (np.abs(gw) + np.abs(n) * np.abs(gw * n).mean(axis=1, keepdims=True)))
    within(f64(dx), want, off + B * (np.abs(want) + off) + 4 * U * np.abs(want), "dx")
    terms = np.abs(f64(dy) * n).sum(axis=0)
    within(f64(dw), (f64(dy) * n).sum(axis=0), (T / 152 + 96) * U * terms, "dweight")


def test_codes_are_those_of_the_division(ops):
    # scales far outside the fast range, subnormal ones and all-zero groups among them
    g = np.random.default_rng(1)
    x = torch.from_numpy(g.normal(size=(200, 656)).astype(np.float32)).cuda()
    x = (x * torch.from_numpy(2.0 ** g.integers(-130, 120, size=(200, 1))).float().cuda()).to(BF16)
    x[3] = 0
    x[7, 128:256] = 0
    xq, xs = pack(ops, x)
    p = torch.zeros(200, 768, device="cuda")
    p[:, :656] = x.float()
    p = p.view(200, 6, 128)
    m = p.abs().amax(2)
    s = m / torch.full_like(m, 448.0)
    q = torch.where(s[..., None] > 0, p / s[..., None], 0.0).clamp(-448, 448).view(200, 768)[:, :656]
    assert torch.equal(xs, s)
    assert torch.equal(xq.view(torch.uint8), q.to(torch.float8_e4m3fn).contiguous().view(torch.uint8))


def test_what_is_not_finite_stays_in_its_group(ops):
    x = rows(6, 400)
    clean = [t.clone() for t in pack(ops, x)]
    x[1, 130], x[2, 399], x[3, 0] = float("nan"), float("inf"), -float("inf")
    xq, xs = pack(ops, x)
    back = torch.empty_like(x)
    ops.unpack_q8(xq, xs, back)
    torch.cuda.synchronize()
    hit = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[2, 3] = hit[3, 0] = True
    wide = hit.repeat_interleave(128, 1)[:, :400]
    assert torch.equal(xs[~hit], clean[1][~hit]) and not xs[hit].isfinite().any()
    assert torch.equal(xq.view(torch.uint8)[~wide], clean[0].view(torch.uint8)[~wide])
    assert not back[wide].isfinite().any() and back[~wide].isfinite().all()


def test_the_layer_reads_packed_codes(ops):
    from mixture_experts_layer_07_gb300 import synth
    from tests import gpu_util as gu
    spec = synth.SPECS["tiny"].with_(H=272, E=8, K=2, I=160, wdtype="fp8", act="fp8")
    t = gu.layer_tensors(synth.host_inputs(spec, 100, seed=3))
    cfg = gu.config_for(ops, spec, 100)
    layer = ops.MoELayer(cfg, t)
    want = layer(t["x"]).clone()
    xq, xs = pack(ops, t["x"])
    got = torch.empty_like(want)
    ops.layer_q8(cfg, t["x"], xq, xs, layer.weights, got, layer.workspace, layer.dev_status)
    assert torch.equal(got, want)


def test_rows_past_32_bits(ops):
    T, H = 262200, 8208  # 2^31 + 4 x 10^6 codes
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    x[-3:] = rows(3, H, 2)
    xq, xs = pack(ops, x)
    small = pack(ops, x[-3:].contiguous())
    assert torch.equal(xq[-3:].view(torch.uint8), small[0].view(torch.uint8)) and torch.equal(xs[-3:], small[1])
    assert not xs[:-3].any()
    x.fill_(7.0)
    ops.unpack_q8(xq, xs, x)
    want = torch.empty(3, H, dtype=BF16, device="cuda")
    ops.unpack_q8(*small, want)
    assert torch.equal(x[-3:], want) and not x[:-3].any()


def test_norm_backward_over_its_inputs_without_tokens_and_captured(ops):
    T, H = 77, 384
    h = rows(T, H, 5)
    hq, hs = pack(ops, h)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    w = torch.ones(H, device="cuda")
    dy, dh = rows(T, H, 6), rows(T, H, 7)
    n = ops.add_rmsnorm_backward_scratch_bytes(T, H)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    run = lambda a, b, o, s=None: ops.add_rmsnorm_backward_q8(a, hq, hs, rstd, w, o, dw, scratch, dh=b, stream=s)  # noqa: E731
    run(dy, dh, dx)
    want = dw.clone()
    for over in (0, 1):
        a, b = dy.clone(), dh.clone()
        run(a, b, (a, b)[over])
        assert torch.equal((a, b)[over], dx) and torch.equal(dw, want)
    out = torch.zeros_like(dx)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(dy, dh, out, s)
    s.synchronize()
    assert torch.equal(out, dx)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(dy, dh, out)
        ops.pack_q8(out, hq, hs)
        ops.unpack_q8(hq, hs, out)
    keep = hq.clone(), hs.clone()
    g.replay()
    torch.cuda.synchronize()
    q, sc = pack(ops, dx)
    back = torch.empty_like(dx)
    ops.unpack_q8(q, sc, back)
    assert torch.equal(out, back) and not torch.equal(keep[1], hs)
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    empty = e(0, H, dt=BF16)
    ops.add_rmsnorm_backward_q8(empty, e(0, H, dt=torch.uint8), e(0, 3), e(0), w, empty, dw, scratch)
    ops.pack_q8(empty, e(0, H, dt=torch.uint8), e(0, 3))
    ops.unpack_q8(e(0, H, dt=torch.uint8), e(0, 3), empty)
    torch.cuda.synchronize()
    assert not dw.any()


@pytest.mark.parametrize("H", [64, 256, 1040])
def test_norm_backward_repeats_its_bits(ops, H):
    # rows of one warp and of several; lanes share their copies of the codes
    T = 5000
    h = rows(T, H, 1)
    hq, hs = pack(ops, h)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    w, dy = torch.ones(H, device="cuda"), rows(T, H, 2)
    scratch = torch.empty(ops.add_rmsnorm_backward_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(5):
        dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
        ops.add_rmsnorm_backward_q8(dy, hq, hs, rstd, w, dx, dw, scratch)
        got.append((dx, dw))
    for dx, dw in got[1:]:
        assert torch.equal(dx, got[0][0]) and torch.equal(dw, got[0][1])
    n = f64(hq.float()) * np.repeat(f64(hs), 128, axis=1)[:, :H] * f64(rstd)[:, None]
    want = f64(rstd)[:, None] * (f64(dy) - n * (f64(dy) * n).mean(axis=1, keepdims=True))
    within(f64(got[0][0]), want, B * np.abs(want) + 2.0 ** -16 * np.abs(f64(dy)).max(), "dx")
