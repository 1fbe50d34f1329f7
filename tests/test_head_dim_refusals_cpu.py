"""Heads of no numbers are refused as other calls that do not fit are: without a
GPU by the check for one, with one by the library.
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from diffusion_transformer_qk_amd import binding as b


def test_heads_of_no_numbers():
    q = torch.zeros((1, 4, 2, 0), dtype=torch.bfloat16)
    lse = torch.zeros((1, 2, 4))
    offsets = torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda: qkr.attention(q, q, q), lambda: qkr.attention_backward(q, q, q, q, q, lse),
                 lambda: qkr.attention_packed(q[0], q[0], q[0], offsets),
                 lambda: qkr.attention_packed_backward(q[0], q[0], q[0], q[0], q[0], lse[0], offsets)):
        with pytest.raises((ValueError, qkr.QkrError)):
            call()
    lib = b.load_library()
    args = b.AttnPackedArgs(1, 4, 4, 2, 2, 0, 0, b.QKR_BF16, 1.0, 0, None, None)
    assert lib.dit_attention_packed_workspace_size(args) == b.QKR_ERR_UNSUPPORTED
    assert lib.dit_attention_workspace_size(b.AttnArgs(1, 4, 4, 2, 2, 0, 0, b.QKR_BF16, 1.0, None)) == b.QKR_ERR_UNSUPPORTED
