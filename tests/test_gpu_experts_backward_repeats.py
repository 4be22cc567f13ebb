"""GPU: calls of the experts' gradient one behind the other, as a training step makes them for its
layers: the pairs of one launch end while those of the next begin on the same SMs."""
import pytest
import torch

from tests.test_gpu_experts_backward import Case, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def test_calls_one_behind_the_other(ops):  # noqa: F811
    # units for a part of the pairs, for one wave and for several; all three parts' ends follow closely
    cases = [Case(*s, seed=i) for i, s in enumerate([(100, 256, 8, 2, 128), (1, 64, 1, 1, 48), (500, 512, 9, 3, 320),
                                                     (64, 1040, 40, 4, 96)])]
    scratch = torch.full((max(c.scratch(ops).numel() for c in cases),), 0xFF, dtype=torch.uint8, device="cuda")
    want = [c.run(ops, scratch).outputs() for c in cases]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(25):
            for c in cases:
                c.run(ops, scratch)
    for _ in range(20):
        for c in cases:
            for t in (c.dx, c.d_weights, c.dw1, c.dw3, c.dw2):
                t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        for c, expected in zip(cases, want):
            assert int(c.status) == 0
            for a, b in zip(expected, c.outputs()):
                assert torch.equal(a, b)
