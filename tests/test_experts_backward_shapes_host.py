"""Shapes of the experts' matrices in the experts' gradient.  w1, w3 [E, I, H] and w2 [E, H, I] hold
as many values as their transposes.  (No GPU: the tensors only say that they are on one, and no call
gets as far as a launch.)"""
import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, H, E, K, I = 4, 256, 3, 2, 32


class Placed:
    """A tensor's type and shape, at an aligned address of a GPU that nothing reads."""

    is_cuda = True

    def __init__(self, *shape, dtype=F32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


@pytest.fixture(scope="module")
def ops():
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    return o


def call(ops, dw=BF16, **change):
    m = lambda dt: (Placed(E, I, H, dtype=dt), Placed(E, I, H, dtype=dt), Placed(E, H, I, dtype=dt))  # noqa: E731
    (w1, w3, w2), (dw1, dw3, dw2) = m(BF16), m(dw)
    x = Placed(T, H, dtype=BF16)
    args = dict(dout=x, offsets=Placed(E + 1, dtype=I32), row_to_flat=Placed(T * K, dtype=I32),
                flat_to_row=Placed(T * K, dtype=I32), weights=Placed(T, K), w1=w1, w3=w3, w2=w2,
                scratch=Placed(256, dtype=torch.uint8),  # less than any call needs
                x=x, dx=x, dw1=dw1, dw3=dw3, dw2=dw2, stream=0)
    assert ops.experts_backward_scratch_bytes(T, H, E, K, I) > 256
    ops.experts_backward(**{**args, **change})


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("name", ["w1", "w3", "w2", "dw1", "dw3", "dw2"])
def test_matrices_of_other_shapes_are_refused(ops, name, dw):
    for other in ((E, I, H) if name.endswith("w2") else (E, H, I), (E * I, H), (E * H * I,), (1, E * H, I), (I, E, H)):
        t = Placed(*other, dtype=dw if name[0] == "d" else BF16)
        # E and I are w1's: the offsets or w3 may be the first that do not fit them
        with pytest.raises(ValueError, match=f"^({name}{'|offsets|w3' if name == 'w1' else ''}): .*expected"):
            call(ops, dw, **{name: t})


@pytest.mark.parametrize("dw", [BF16, F32])
def test_the_documented_shapes_reach_the_library(ops, dw):
    for some in ({}, dict(dw1=None, dw3=None, dw2=None)):
        with pytest.raises(ops.MoEError) as e:
            call(ops, dw, **some)
        assert e.value.code == 3  # its own check of the scratch
    with pytest.raises(ops.MoEError) as e:
        call(ops, dw, dw3=None)
    assert e.value.code == 1
