"""Refusals of the paged calls' Python wrappers: arguments that are no tensors, and
shapes without heads.  On the host, with tensors that only say they are on a GPU."""
import pytest
import torch

import product_vq_kv_gb300 as vq
from test_streams import fake, half, i32, u8


def test_attention_without_heads_is_refused():
    with pytest.raises(ValueError, match="does not match"):
        vq.vq_paged_attention(half(4, 4, 64), i32(3), i32(2), i32(2, 5), u8(9, 0, 16, 8), u8(9, 0, 16, 8), half(0, 256, 8),
                              half(0, 256, 8))


@pytest.mark.parametrize("smooth", [1.0, [1.0], "factors"])
def test_append_factors_that_are_no_tensor_are_refused(smooth):
    with pytest.raises(TypeError, match="k_smooth"):
        vq.vq_paged_append(half(4, 2, 64), half(4, 2, 64), fake((4,), torch.int64), half(2, 256, 8), half(2, 256, 8),
                           u8(9, 2, 16, 8), u8(9, 2, 16, 8), k_smooth=smooth)
