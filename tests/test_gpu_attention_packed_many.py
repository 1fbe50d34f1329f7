"""Attention of more packed sequences than a wave has lanes, which the search of a
block's sequence takes in several steps: every sequence's out, lse and gradients
against 64 bits, with the bounds of attention_reference.py for a sample of its size.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests import attention_reference as ref
from tests.test_gpu_attention_packed import DEV, inputs, offsets_of

pytestmark = pytest.mark.gpu


def run(seed, lengths, kv, heads, kv_heads, d, dtype, causal):
    t = inputs(seed, lengths, kv, heads, kv_heads, d, dtype, 1, 2)
    offsets, kv_offsets = offsets_of(lengths, 1), offsets_of(kv, 1)
    kw = dict(kv_offsets=kv_offsets, causal=causal)
    out, lse = qkr.attention_packed(t["q"], t["k"], t["v"], offsets, **kw)
    grads = qkr.attention_packed_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, offsets, **kw)
    return t, out, lse, dict(zip(("dq", "dk", "dv"), grads)), offsets.tolist(), kv_offsets.tolist()


def close(got, want, bound, what):
    assert bool(((got.double().permute(0, 2, 1, 3) - want).abs() <= bound).all()), what


def check(seed, lengths, kv, heads, kv_heads, d, dtype, causal):
    """Sequences of the same numbers of queries and keys are the samples of one reference."""
    t, out, lse, grads, q_at, k_at = run(seed, lengths, kv, heads, kv_heads, d, dtype, causal)
    alike = {}
    for i, size in enumerate(zip(lengths, kv)):
        alike.setdefault(size, []).append(i)
    for (nq, nk), which in alike.items():
        rows = torch.tensor([[q_at[i] + j for j in range(nq)] for i in which], dtype=torch.long, device=DEV)
        keys = torch.tensor([[k_at[i] + j for j in range(nk)] for i in which], dtype=torch.long, device=DEV)
        if nq == 0:
            assert all(bool((grads[n][keys] == 0).all()) for n in ("dk", "dv")), which
            continue
        r = ref.forward(t["q"][rows], t["k"][keys], t["v"][keys], causal=causal)
        close(out[rows], r["out"], r["bound"], ("out", nq, nk))
        s, some = lse[:, rows].permute(1, 0, 2).double(), r["some"]
        assert bool((s[~some] == -math.inf).all())
        assert bool(((s - r["lse"]).abs()[some] <= r["lse_bound"][some]).all()), ("lse", nq, nk)
        for n, (want, bound) in ref.backward(r, t["dout"][rows], out[rows], dtype).items():
            close(grads[n][rows if n == "dq" else keys], want, bound, (n, nq, nk))


@pytest.mark.parametrize("count", [63, 64, 65, 300, 4097, 5000])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,dtype", [(64, 2, 1, torch.bfloat16), (64, 2, 2, torch.float16),
                                                    (128, 3, 1, torch.float16)])
def test_short_sequences(count, causal, d, heads, kv_heads, dtype):
    g = torch.Generator().manual_seed(count)
    lengths = torch.randint(0, 4, (count,), generator=g).tolist()
    kv = torch.randint(0, 9, (count,), generator=g).tolist()
    check(51, lengths, kv, heads, kv_heads, d, dtype, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,dtype", [(64, 2, 1, torch.float16), (128, 2, 2, torch.bfloat16),
                                                    (256, 1, 1, torch.float16)])
def test_sequences_of_several_blocks(causal, d, heads, kv_heads, dtype):
    """Blocks of keys and of rows that begin in one step of the search and end in another."""
    g = torch.Generator().manual_seed(d)
    lengths = [n if n > 40 else 0 for n in torch.randint(0, 300, (140,), generator=g).tolist()]
    kv = [n if n > 30 else 0 for n in torch.randint(0, 300, (140,), generator=g).tolist()]
    check(52, lengths, kv, heads, kv_heads, d, dtype, causal)


def test_the_neighbour_is_told_apart():
    """The oracle's gradients of the sequence beside are not within the bounds."""
    t = inputs(53, [2, 2], [8, 8], 2, 1, 64, torch.bfloat16)
    a, b = (ref.forward(*(t[n][None, s] for n, s in (("q", q), ("k", k), ("v", k)))) for q, k in (
        (slice(0, 2), slice(0, 8)), (slice(2, 4), slice(8, 16))))
    ga, gb = (ref.backward(r, t["dout"][None, s], r["out"].permute(0, 2, 1, 3).to(torch.bfloat16), torch.bfloat16)
              for r, s in ((a, slice(0, 2)), (b, slice(2, 4))))
    for n in ("dq", "dk", "dv"):
        assert not bool(((gb[n][0] - ga[n][0]).abs() <= ga[n][1]).all())
