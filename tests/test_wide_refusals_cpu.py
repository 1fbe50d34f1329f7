"""Widths past 32 bits are refused, not cut off: tensors without memory stand for
those that a GPU could hold.
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr

WIDE = 2 ** 32 + 64


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda: qkr.rms_norm(meta(1, WIDE)), lambda: qkr.rms_norm_fp8(meta(1, WIDE)),
    lambda: qkr.rms_norm_backward(meta(1, WIDE), meta(1, WIDE)),
    lambda: qkr.gated_feed_forward(meta(1, WIDE), meta(8, WIDE), meta(8, WIDE)),
    lambda: qkr.gated_feed_forward(meta(1, 64), meta(WIDE, 64), meta(WIDE, 64)),
    lambda: qkr.attention_packed(*[meta(1, 1, WIDE)] * 3, meta(2, dtype=torch.int32)),
    lambda: qkr.attention_packed(meta(1, WIDE, 64), meta(1, 1, 64), meta(1, 1, 64), meta(2, dtype=torch.int32))])
def test_refused(call):
    with pytest.raises(ValueError, match="below 2\\^31"):
        call()
