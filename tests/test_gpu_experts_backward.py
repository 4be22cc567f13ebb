"""GPU: the experts' gradient against the float64 oracle.

Tolerances are the oracle's own bound (``block_oracle.experts_backward`` with errors): fp32
sums of bf16 products, three roundings to bf16 between the products (half a step, 2^-8
relative), and the output's rounding on top (bf16 2^-8, fp32 2^-24).
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


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
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g}x, first at "
                           f"{np.argwhere(bad)[0].tolist()}")


class Case:
    """Inputs of one call, its routing as a stable sort gives it, and output buffers full of 7."""

    def __init__(self, T, H, E, K, I, seed=0, skew=0.0, drop=0.0, q8=False, dw=BF16):
        g = np.random.default_rng(seed)
        self.T, self.H, self.E, self.K, self.I, self.dw_type = T, H, E, K, I, dw
        bf = lambda a: torch.from_numpy(np.asarray(a, np.float32)).to(BF16).cuda()  # noqa: E731
        self.x = bf(g.normal(size=(T, H)) * np.exp(0.3 * g.normal(size=(T, 1))))
        self.dout, self.dx_add = bf(g.normal(size=(T, H)) * 0.01), bf(g.normal(size=(T, H)) * 0.01)
        self.w1, self.w3 = (bf(g.normal(size=(E, I, H)) * H ** -0.5) for _ in range(2))
        self.w2 = bf(g.normal(size=(E, H, I)) * I ** -0.5)
        self.weights = torch.from_numpy(g.random((T, K)).astype(np.float32)).cuda()
        key = g.random((T, E)) + skew * (np.arange(E) == E // 2)
        self.ids = np.argsort(-key, axis=1, kind="stable")[:, :K].astype(np.int64)
        if drop:
            self.ids[g.random((T, K)) < drop] = -1
        self.set_routing()
        self.xq = self.xs = None
        if q8:
            from mixture_experts_layer_07_gb300 import ops as o
            self.xq = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
            self.xs = torch.empty(T, -(-H // 128), device="cuda")
            o.pack_q8(self.x, self.xq, self.xs)
            o.unpack_q8(self.xq, self.xs, self.x)  # what the codes stand for
        self.new_outputs()

    def set_routing(self):
        flat = self.ids.reshape(-1)
        keep = np.flatnonzero(flat >= 0)
        order = keep[np.argsort(flat[keep], kind="stable")]
        r2f = np.full(flat.size, -1, np.int32)
        r2f[:order.size] = order
        f2r = np.full(flat.size, -1, np.int32)
        f2r[order] = np.arange(order.size)
        off = np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=self.E))])
        dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        self.r2f, self.f2r, self.off = dev(r2f), dev(f2r), dev(off)

    def new_outputs(self):
        full = lambda shape, t: torch.full(shape, 7.0, dtype=t, device="cuda")  # noqa: E731
        self.dx, self.d_weights = full((self.T, self.H), BF16), full((self.T, self.K), F32)
        self.dw1, self.dw3 = (full(tuple(self.w1.shape), self.dw_type) for _ in range(2))
        self.dw2 = full(tuple(self.w2.shape), self.dw_type)
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def scratch(self, ops, fill=0xFF):
        n = ops.experts_backward_scratch_bytes(self.T, self.H, self.E, self.K, self.I)
        return torch.full((n,), fill, dtype=torch.uint8, device="cuda")

    def run(self, ops, scratch=None, **kw):
        q8 = self.xq is not None
        args = dict(x=None if q8 else self.x, xq=self.xq, xq_scale=self.xs, dx_add=self.dx_add, dx=self.dx,
                    d_weights=self.d_weights, dw1=self.dw1, dw3=self.dw3, dw2=self.dw2, dev_status=self.status)
        ops.experts_backward(self.dout, self.off, self.r2f, self.f2r, self.weights, self.w1, self.w3, self.w2,
                             self.scratch(ops) if scratch is None else scratch, **{**args, **kw})
        return self

    def outputs(self):
        return [t.clone() for t in (self.dx, self.d_weights, self.dw1, self.dw3, self.dw2)]

    def check(self, base=0.0, add=True):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        ref = bo.experts_backward(*(f64(t) for t in (self.x, self.dout)), self.ids,
                                  *(f64(t) for t in (self.weights, self.w1, self.w3, self.w2)), errors=(U, B))
        dx = ref["dx"] + (f64(self.dx_add) if add else 0.0)
        tiny = 1e-30
        within(f64(self.d_weights), ref["d_weights"], ref["e_d_weights"] + U * np.abs(ref["d_weights"]) + tiny,
               "d_weights")
        e = ref["e_dx"] + (self.K + 1) * U * (np.abs(dx) + ref["e_dx"]) + tiny
        within(f64(self.dx), dx, e + B * (np.abs(dx) + e), "dx")
        for n in ("dw1", "dw3", "dw2"):
            want, e, b = ref[n] + base, ref["e_" + n] + tiny, B if self.dw_type == BF16 else U
            within(f64(getattr(self, n)), want, e + b * (np.abs(want) + e), n)
        return self


# one token; sizes below a tile, between tiles and at their edges; rows of one, 64, 65, 128, 129 and more
SIZES = [(1, 16, 1, 1, 16), (1, 256, 8, 2, 128), (5, 64, 4, 3, 48), (64, 128, 1, 1, 64), (65, 144, 1, 1, 80),
         (37, 272, 3, 3, 144), (128, 192, 2, 2, 256), (129, 528, 1, 1, 272), (100, 256, 8, 2, 128),
         (300, 320, 6, 2, 400), (50, 1040, 40, 4, 96), (700, 96, 5, 2, 1040)]


@pytest.mark.parametrize("T,H,E,K,I", SIZES)
@pytest.mark.parametrize("q8", [False, True])
def test_matches_oracle(ops, T, H, E, K, I, q8):
    Case(T, H, E, K, I, seed=T + H, q8=q8, dw=F32 if q8 else BF16).run(ops).check()
