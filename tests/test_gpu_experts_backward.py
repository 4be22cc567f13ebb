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


@pytest.mark.parametrize("q8", [False, True])
def test_many_wide_rows(ops, q8):
    # several tiles per expert and several blocks of both sizes, none of them whole
    Case(512, 2880, 4, 2, 2896, seed=3, skew=0.3, q8=q8).run(ops).check()


def test_the_most_experts_and_replicas(ops):
    c = Case(50, 32, 1024, 32, 48, seed=7).run(ops).check()
    # and in a scratch that is aligned to no more than it has to be
    n = ops.experts_backward_scratch_bytes(50, 32, 1024, 32, 48)
    wide = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    want = c.outputs()
    c.new_outputs()
    start = (256 - wide.data_ptr()) % 512
    assert (wide.data_ptr() + start) % 512 == 256
    for a, b in zip(want, c.run(ops, wide[start:start + n]).outputs()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H,E,K,I", [(60, 128, 9, 2, 64), (1, 64, 3, 3, 32), (400, 144, 16, 4, 208)])
def test_dropped_replicas(ops, T, H, E, K, I):
    c = Case(T, H, E, K, I, seed=5, drop=0.4).run(ops).check()
    assert (f64(c.d_weights)[c.ids < 0] == 0).all()
    # maps that point past the rows are dropped replicas too
    d = Case(T, H, E, K, I, seed=5, drop=0.4)
    d.f2r[d.f2r < 0] = 2 ** 31 - 1
    for a, b in zip(c.outputs(), d.run(ops).outputs()):
        assert torch.equal(a, b)


def test_nothing_routed(ops):
    c = Case(33, 64, 4, 2, 48, drop=1.0).run(ops)
    torch.cuda.synchronize()
    assert torch.equal(c.dx, c.dx_add) and not c.d_weights.any()
    assert not (c.dw1.any() or c.dw3.any() or c.dw2.any())


def test_one_expert_takes_all(ops):
    c = Case(300, 128, 12, 1, 96, skew=10.0).run(ops).check()
    rest = torch.arange(12, device="cuda") != 6
    assert not (c.dw1[rest].any() or c.dw3[rest].any() or c.dw2[rest].any())


def test_a_shared_expert_with_its_gate(ops):
    c = Case(200, 256, 1, 1, 128, seed=9)
    assert c.r2f.tolist() == list(range(200)) and c.off.tolist() == [0, 200]
    c.run(ops).check()


def test_gradients_are_added_to_what_is_there(ops):
    c = Case(40, 144, 16, 1, 80, dw=F32)
    empty = np.bincount(c.ids.reshape(-1), minlength=16) == 0
    assert empty.any()
    c.run(ops, accumulate=True).check(base=7.0)
    for t in (c.dw1, c.dw3, c.dw2):
        assert (f64(t)[empty] == 7.0).all()
    twice = Case(40, 144, 16, 1, 80, dw=F32)
    twice.run(ops)
    once = [t.clone() for t in (twice.dw1, twice.dw3, twice.dw2)]
    twice.run(ops, accumulate=True)
    for a, b in zip(once, (twice.dw1, twice.dw3, twice.dw2)):
        assert torch.equal(2 * a, b)  # exact in fp32


def test_each_output_alone(ops):
    full = Case(90, 160, 5, 2, 112).run(ops)
    torch.cuda.synchronize()
    none = dict(dx=None, d_weights=None, dw1=None, dw3=None, dw2=None)
    for keep in (("dx",), ("d_weights",), ("dw1", "dw3", "dw2")):
        c = Case(90, 160, 5, 2, 112)
        c.run(ops, **{k: v for k, v in none.items() if k not in keep})
        for name in none:
            got = getattr(c, name)
            assert torch.equal(got, getattr(full, name)) if name in keep else bool((got == 7.0).all()), name


def test_without_an_addend(ops):
    Case(50, 64, 4, 2, 64).run(ops, dx_add=None).check(add=False)


@pytest.mark.parametrize("over", ["dx_add", "dout", "x"])
def test_dx_over_an_input(ops, over):
    want = Case(150, 128, 6, 3, 64).run(ops).outputs()
    c = Case(150, 128, 6, 3, 64)
    c.run(ops, dx=getattr(c, over))
    c.dx = getattr(c, over)
    for a, b in zip(want, c.outputs()):
        assert torch.equal(a, b)


def test_same_bits_whatever_the_scratch_holds(ops):
    c = Case(333, 272, 7, 3, 144)
    want = c.run(ops, c.scratch(ops, 0)).outputs()
    shared = c.scratch(ops, 0xFF)
    for other in (None, (700, 96, 5, 2, 48)):  # again, and after a call of another size in the same scratch
        if other:
            o = Case(*other, seed=8)
            o.run(ops, shared if shared.numel() >= o.scratch(ops).numel() else None)
        c.new_outputs()
        for a, b in zip(want, c.run(ops, shared).outputs()):
            assert torch.equal(a, b)


def test_a_nan_stays_with_its_token_and_experts(ops):
    clean = Case(200, 128, 8, 2, 96, seed=4).run(ops)
    torch.cuda.synchronize()
    for where in ("x", "dout"):
        c = Case(200, 128, 8, 2, 96, seed=4)
        getattr(c, where)[77, 5] = float("nan")
        c.run(ops)
        torch.cuda.synchronize()
        assert int(c.status) == 0
        others = torch.arange(200, device="cuda") != 77
        assert torch.equal(c.dx[others], clean.dx[others]) and torch.equal(c.d_weights[others], clean.d_weights[others])
        assert c.dx[77].isnan().any() and c.d_weights[77].isnan().all()
        hit = torch.zeros(8, dtype=torch.bool, device="cuda")
        hit[torch.from_numpy(c.ids[77]).cuda()] = True
        for n in ("dw1", "dw3", "dw2"):
            got = getattr(c, n)
            assert torch.equal(got[~hit], getattr(clean, n)[~hit]) and got[hit].isnan().flatten(1).any(1).all()


def test_weights_that_are_infinite_stay_in_their_columns(ops):
    # rows behind an expert's last one must not bring 0 x inf into its sums
    c, d = (Case(70, 64, 3, 1, 48, seed=6) for _ in range(2))
    d.w1[1, 5, 3] = float("inf")
    c.run(ops), d.run(ops)
    torch.cuda.synchronize()
    keep = torch.arange(48, device="cuda") != 5
    for n in ("dw1", "dw3"):
        assert torch.equal(getattr(c, n)[:, keep], getattr(d, n)[:, keep])
    assert torch.equal(c.dw2[:, :, keep], d.dw2[:, :, keep])


def test_no_tokens(ops):
    c = Case(0, 64, 4, 2, 32, dw=F32).run(ops)
    torch.cuda.synchronize()
    assert not (c.dw1.any() or c.dw3.any() or c.dw2.any())
    c = Case(0, 64, 4, 2, 32, dw=F32).run(ops, accumulate=True)
    torch.cuda.synchronize()
    assert bool((c.dw1 == 7.0).all() and (c.dw2 == 7.0).all())


def test_another_stream_and_a_captured_call(ops):
    a, b = Case(120, 128, 6, 2, 64, seed=1), Case(120, 128, 6, 2, 64, seed=2)
    want = [c.run(ops).outputs() for c in (a, b)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c = Case(120, 128, 6, 2, 64, seed=1)
    scratch = c.scratch(ops)
    s.wait_stream(torch.cuda.current_stream())
    c.run(ops, scratch, stream=s)
    s.synchronize()
    for x, y in zip(want[0], c.outputs()):
        assert torch.equal(x, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(ops, scratch)
    for case, expected in ((b, want[1]), (a, want[0])):
        for n in ("x", "dout", "dx_add", "weights", "w1", "w3", "w2", "off", "r2f", "f2r"):
            getattr(c, n).copy_(getattr(case, n))
        scratch.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(expected, c.outputs()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("T", [1, 4, 24, 200])
def test_routing_of_a_layer_as_it_left_it(ops, T):
    # every path of the layer leaves its routing in the workspace
    from mixture_experts_layer_07_gb300 import synth
    from tests import gpu_util as gu
    spec = synth.SPECS["tiny"]
    t = gu.layer_tensors(synth.host_inputs(spec, T, seed=11))
    layer = ops.MoELayer(gu.config_for(ops, spec, 256), t)
    layer(t["x"])
    c = Case(T, spec.H, spec.E, spec.K, spec.I, seed=T)
    c.x, c.w1, c.w3, c.w2 = t["x"], t["w1"], t["w3"], t["w2"]
    view = lambda n, dt, *s: layer.view(n, dt, s).clone()  # noqa: E731
    c.off, c.weights = view("offsets", I32, spec.E + 1), view("weights", F32, T, spec.K)
    c.r2f, c.f2r = view("row_to_flat", I32, T * spec.K), view("flat_to_row", I32, T * spec.K)
    c.ids = view("ids", I32, T, spec.K).cpu().numpy().astype(np.int64)
    want = c.run(ops).check().outputs()
    # and through the layer itself
    c.new_outputs()
    layer.experts_backward(c.dout, c.scratch(ops), x=c.x, dx_add=c.dx_add, dx=c.dx, d_weights=c.d_weights, dw1=c.dw1,
                           dw3=c.dw3, dw2=c.dw2)
    assert int(layer.dev_status) == 0
    for a, b in zip(want, c.outputs()):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="^dout: 257 tokens"):
        layer.experts_backward(torch.empty(257, spec.H, dtype=BF16, device="cuda"), c.scratch(ops), x=c.x, dx=c.dx)


def test_rows_past_32_bits(ops):
    # 262400 rows of 8192: the last ones lie beyond 2^31 values, and 2^32 bytes in every row buffer
    T, H, E, K, I = 32800, 8192, 8, 8, 16
    g = torch.Generator("cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dout = rand(T, H).to(BF16), (rand(T, H) * 0.01).to(BF16)
    w1, w3 = ((rand(E, I, H) * H ** -0.5).to(BF16) for _ in range(2))
    w2 = (rand(E, H, I) * I ** -0.5).to(BF16)
    w = torch.rand(T, K, device="cuda", generator=g)
    # every token on every expert: row e T + t
    t, e = torch.arange(T, device="cuda"), torch.arange(E, device="cuda")
    r2f = (t[None, :] * K + e[:, None]).reshape(-1).to(I32)
    f2r = (e[None, :] * T + t[:, None]).reshape(-1).to(I32)
    off = (torch.arange(E + 1, device="cuda") * T).to(I32)
    dx, dw = torch.empty_like(x), torch.empty(T, K, device="cuda")
    d1, d3, d2 = (torch.empty_like(m) for m in (w1, w3, w2))
    scratch = torch.empty(ops.experts_backward_scratch_bytes(T, H, E, K, I), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    ops.experts_backward(dout, off, r2f, f2r, w, w1, w3, w2, scratch, x=x, dx=dx, d_weights=dw, dw1=d1, dw3=d3,
                         dw2=d2, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    # tokens of the last tile, in 64 bits by the oracle
    last = slice(T - 40, T)
    ids = np.tile(np.arange(E), (40, 1))
    ref = bo.experts_backward(f64(x[last]), f64(dout[last]), ids, f64(w[last]), f64(w1), f64(w3), f64(w2), (U, B))
    within(f64(dx[last]), ref["dx"], ref["e_dx"] + B * (np.abs(ref["dx"]) + ref["e_dx"]) + 1e-30, "dx")
    within(f64(dw[last]), ref["d_weights"], ref["e_d_weights"] + U * np.abs(ref["d_weights"]), "d_weights")
    # the last expert's matrices over all rows: the roundings' errors have no common sign, so that the
    # sums' relative error stays near one rounding's; half a step of two roundings bounds it amply
    D = torch.float64
    xe, de = x.to(D), dout.to(D)
    gate, up, a = xe @ w1[7].to(D).t(), xe @ w3[7].to(D).t(), de @ w2[7].to(D)
    s = torch.sigmoid(gate)
    wt = w[:, 7:8].to(D)
    for got, ref in ((d1[7], (wt * a * up * s * (1 + gate * (1 - s))).t() @ xe), (d3[7], (wt * a * gate * s).t() @ xe),
                     (d2[7], de.t() @ (wt * gate * s * up))):
        rel = float((got.to(D) - ref).norm() / ref.norm())
        assert rel < 2 * B, rel


def test_two_calls_at_once(ops):
    # on two streams, with a scratch each
    cases = [Case(500, 512, 9, 3, 320, seed=s) for s in (1, 2)]
    want = [c.run(ops).outputs() for c in cases]
    scratch = [c.scratch(ops) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, s in zip(cases, scratch, streams):
            c.run(ops, w, stream=s)
    torch.cuda.synchronize()
    for c, expected in zip(cases, want):
        assert int(c.status) == 0
        for a, b in zip(expected, c.outputs()):
            assert torch.equal(a, b)
