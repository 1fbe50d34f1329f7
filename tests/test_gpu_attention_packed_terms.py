"""How p and ds are rounded in attention of packed sequences: in two 16-bit terms
where a sequence has up to 32 query rows a key head, in one above, whatever the
other sequences of the call are.  Each sequence is held to the bounds of
attention_reference.py for a sample of its own size, whose terms go by those rows.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests import attention_reference as ref
from tests.test_gpu_attention_packed import DEV, inputs, offsets_of, slices

pytestmark = pytest.mark.gpu

# Short sequences beside long ones, on both sides of 32 rows with the groups below,
# and, last, one long sequence among so many short ones that the mean is below 32.
LENGTHS = [
    ([1, 700], None), ([13, 1100, 32, 33], None), ([16, 17, 900, 8, 0, 11], None), ([400, 1, 7], [90, 2500, 130]),
    ([2, 600], [3000, 64]), ([300, *[1] * 40, 5, *[2] * 40], None),
]
KINDS = [(64, 3, 3, "bfloat16"), (64, 4, 2, "float16"), (128, 2, 2, "float16"), (128, 4, 1, "bfloat16"),
         (256, 2, 2, "bfloat16"), (256, 6, 2, "float16")]


def call(lengths, kv, causal, d, heads, kv_heads, dtype):
    t = inputs(31, lengths, kv or lengths, heads, kv_heads, d, getattr(torch, dtype), 2, 3)
    kw = dict(kv_offsets=offsets_of(kv, 2) if kv else None, causal=causal)
    out, lse = qkr.attention_packed(t["q"], t["k"], t["v"], offsets_of(lengths, 2), **kw)
    return t, kw, out, lse


def each(t, lengths, kv, causal):
    """Rows and keys of the sequences that have rows, and the reference of each."""
    for rows, keys in zip(slices(lengths, 2), slices(kv or lengths, 2)):
        if rows.stop > rows.start:
            yield rows, keys, ref.forward(*(t[n][s][None] for n, s in (("q", rows), ("k", keys), ("v", keys))),
                                          causal=causal)


@pytest.mark.parametrize("lengths,kv", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,dtype", KINDS)
def test_forward(lengths, kv, causal, d, heads, kv_heads, dtype):
    t, _, out, lse = call(lengths, kv, causal, d, heads, kv_heads, dtype)
    for rows, keys, r in each(t, lengths, kv, causal):
        got = out[rows].double().permute(1, 0, 2)
        assert bool(((got - r["out"][0]).abs() <= r["bound"][0]).all()), (rows, keys)
        s, some = lse[:, rows].double(), r["some"][0]
        assert bool((s[~some] == -math.inf).all())
        assert bool(((s - r["lse"][0]).abs()[some] <= r["lse_bound"][0][some]).all()), (rows, keys)


@pytest.mark.parametrize("lengths,kv", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,dtype", KINDS)
def test_backward(lengths, kv, causal, d, heads, kv_heads, dtype):
    t, kw, out, lse = call(lengths, kv, causal, d, heads, kv_heads, dtype)
    grads = dict(zip(("dq", "dk", "dv"), qkr.attention_packed_backward(
        t["dout"], t["q"], t["k"], t["v"], out, lse, offsets_of(lengths, 2), **kw)))
    for rows, keys, r in each(t, lengths, kv, causal):
        for n, (want, bound) in ref.backward(r, t["dout"][rows][None], out[rows][None], out.dtype).items():
            got = grads[n][rows if n == "dq" else keys].double().permute(1, 0, 2)
            assert bool(((got - want[0]).abs() <= bound[0]).all()), (n, rows, keys)


def test_the_bounds_tell_the_terms_apart():
    """One term of p does not meet the bound of a short sequence (by the oracle, on the CPU)."""
    g = torch.Generator().manual_seed(32)
    q, k, v = (torch.randn((1, n, 2, 64), generator=g).to(torch.bfloat16) for n in (16, 500, 500))
    r = ref.forward(q, k, v)
    p = r["p"].to(torch.bfloat16).double()
    off = (p @ r["v"] - r["out"]).abs()
    assert not bool((off <= r["bound"]).all())
    rest = (r["p"] - p).to(torch.bfloat16).double()
    assert bool((((p + rest) @ r["v"] - r["out"]).abs() <= r["bound"]).all())
