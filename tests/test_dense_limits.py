"""Sizes at the limits of the operators around the MoE layer, checked without a GPU."""
import pytest

import routed_expert_ffn_04_amd as moe


class Shape:
    """Stands for a tensor on a GPU; only its sizes are looked at."""
    device = "cuda:0"

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 4])
def test_sizes_that_an_int32_does_not_hold_are_refused(size):
    """They would reach the library as their low 32 bits: 2^32 + 4 rows as 4."""
    t = Shape(size, 16)
    for call in (lambda: moe.quant_i8(t), lambda: moe.norm(t), lambda: moe.norm_backward(t, None, t, t),
                 lambda: moe.linear_i8(t, None, t, None), lambda: moe.ffn(t, None), lambda: moe.ffn_backward(t, t, None),
                 lambda: moe.quant_i8(Shape(4, size))):
        with pytest.raises(ValueError, match=str(2 ** 31 - 1)):
            call()
    w = Shape(1, size, 16)
    with pytest.raises(ValueError, match=str(2 ** 31 - 1)):
        moe._dense_bank(moe.Experts(w, w, w), 16, 0)
