"""GPU: the layer on quantised activations reads the codes that it is given --
all of them, each row's own, on a workspace that has never held them."""
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_block import ops, quantise, w8a8_case  # noqa: F401

pytestmark = pytest.mark.gpu

# H = 4368: past the 4096 columns of the copy's first pass and the 32 scales of
# its first pass, the last group 16 columns wide; 272 and 128: one pass, ragged and whole
SHAPES = [(1, 272), (33, 272), (9, 128), (1, 4368), (7, 4368), (300, 4368)]


def poisoned(ops, cfg, t):  # noqa: F811
    """A layer whose workspace holds 0xFF wherever it need not start at zero."""
    layer = ops.MoELayer(cfg, t)
    layer.workspace[layer.layout.logits:].fill_(0xFF)
    return layer


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("shared", [False, True])
def test_layer_q8_on_a_workspace_of_its_own(ops, T, H, shared):  # noqa: F811
    spec, t = w8a8_case(H=H, T=T, has_shared=shared)
    cfg = gu.config_for(ops, spec, T)
    want = ops.MoELayer(cfg, t)(t["x"])
    xq, xs = quantise(t["x"])
    layer, got = poisoned(ops, cfg, t), torch.empty_like(want)
    ops.layer_q8(cfg, t["x"], xq, xs, layer.weights, got, layer.workspace, layer.dev_status)
    torch.cuda.synchronize()
    assert int(layer.dev_status) == 0 and want.isfinite().all() and torch.equal(got, want)


@pytest.mark.parametrize("T,H", SHAPES)
def test_layer_q8_takes_the_experts_rows_from_the_codes(ops, T, H):  # noqa: F811
    """Codes of another batch: the routing stays x's, the experts' part is the other batch's."""
    spec, t = w8a8_case(H=H, T=T)
    K, E, I = spec.K, spec.E, spec.I
    cfg = gu.config_for(ops, spec, T)
    g = torch.Generator("cuda").manual_seed(T + H)
    other = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    layer, got = poisoned(ops, cfg, t), torch.empty_like(other)
    ops.layer_q8(cfg, t["x"], *quantise(other), layer.weights, got, layer.workspace, layer.dev_status)
    i32 = torch.int32
    f2r, offsets = layer.view("flat_to_row", i32, (T * K,)), layer.view("offsets", i32, (E + 1,))
    weights = layer.view("weights", torch.float32, (T, K))
    # the same from the operators, quantising the permuted rows themselves
    xp = torch.empty(T * K, H, dtype=torch.bfloat16, device="cuda")
    xp[f2r.long()] = other.repeat_interleave(K, 0)
    hact = torch.empty(T * K, I, dtype=torch.bfloat16, device="cuda")
    y, want = torch.empty_like(xp), torch.empty_like(other)
    scratch = torch.zeros(ops.grouped_gemm_scratch_bytes(T * K, E, H, I, ops.W8A8_FP8), dtype=torch.uint8, device="cuda")
    ops.grouped_gemm(xp, offsets, E, H, I, t["w1"], t["w3"], t["w2"], hact, y, scratch, wdtype=ops.W8A8_FP8,
                     s1=t["s1"], s3=t["s3"], s2=t["s2"])
    ops.unpermute(y, f2r, weights, T, K, H, want)
    ref = ops.MoELayer(cfg, t)(t["x"])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not torch.equal(got, ref)


@pytest.mark.parametrize("what", ["layer", "block"])
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("T", [1, 300])
def test_outputs_belong_to_the_stream_that_fills_them(ops, what, handle, T):  # noqa: F811
    """Memory goes back to the stream that it came from, so an output must come from the stream
    that writes it: neither may it be memory that the current stream has just given up, nor may
    the current stream get it back while the other one still works on it."""
    spec, t = w8a8_case(H=272, T=T)
    cfg = gu.config_for(ops, spec, T)
    x, r = t["x"], torch.ones_like(t["x"])
    norm = torch.ones(272, dtype=torch.bfloat16, device="cuda")
    call = (lambda **k: (ops.MoELayer(cfg, t)(x, **k),)) if what == "layer" else \
        (lambda **k: ops.MoEBlock(cfg, t, norm)(x, r, **k))
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    gone = [torch.empty_like(x) for _ in range(8)]
    given_up = {g.data_ptr() for g in gone}
    del gone
    got = call(stream=s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    filled = {g.data_ptr() for g in got}
    assert not filled & given_up
    del got, a
    now = [torch.empty_like(x) for _ in range(64)]
    assert not filled & {n.data_ptr() for n in now}


def test_block_on_another_stream_in_a_graph(ops):  # noqa: F811
    spec, t = w8a8_case(H=272, T=40)
    cfg = gu.config_for(ops, spec, 40)
    norm = torch.ones(272, dtype=torch.bfloat16, device="cuda")
    block, r = ops.MoEBlock(cfg, t, norm), torch.ones_like(t["x"])
    want = block(t["x"], r)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = block(t["x"], r, stream=s)
    for g in got:
        g.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("inside", [False, True])
@pytest.mark.parametrize("given", ["default", "zero", "current", "side"])
def test_outputs_on_the_default_stream_are_its_memory(ops, inside, given):  # noqa: F811
    """The default stream's handle is 0; the allocator says whose memory an output is."""
    spec, t = w8a8_case(H=272, T=300)
    block = ops.MoEBlock(gu.config_for(ops, spec, 300), t, torch.ones(272, dtype=torch.bfloat16, device="cuda"))
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side if inside else torch.cuda.default_stream()):
        stream = {"default": torch.cuda.default_stream(), "zero": 0, "current": torch.cuda.current_stream(),
                  "side": other}[given]
        handle = stream if given == "zero" else stream.cuda_stream
        got = block(t["x"], torch.ones_like(t["x"]), stream=stream)
    torch.cuda.synchronize()
    for g in got:
        owner, = [s["stream"] for s in torch.cuda.memory_snapshot()
                  if s["address"] <= g.data_ptr() < s["address"] + s["total_size"]]
        assert owner == handle
