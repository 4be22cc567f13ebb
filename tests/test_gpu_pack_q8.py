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
