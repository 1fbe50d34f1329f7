"""Instruction checks on the feed-forward kernels' gfx950 code (CPU, no GPU).

Large tiles' products are written in assembly, whose distances the compiler does
not keep: each has two wait states in front of it, and where the sums are first
read the longest wait of a matrix instruction's result has passed.  No kernel adds
atomically, and none touches scratch memory.
"""
import re

from tests.test_attention_cpu import objects as attention_objects  # noqa: F401 (a fixture)
from tests.test_attention_isa_cpu import attention, pytestmark  # noqa: F401

KEPT = re.compile(r"v_mfma_f32_16x16x32_(bf16|f16) a\[")
READ = re.compile(r"v_accvgpr_read_b32 ")


def feed_forward(kernels):
    return {n: [text for text, _ in code] for n, code in kernels.items() if "feed_forward" in n}


def test_products_in_assembly_keep_their_distances(attention):  # noqa: F811
    seen = 0
    for name, code in feed_forward(attention).items():
        kept = [i for i, t in enumerate(code) if KEPT.match(t)]
        if "Li4E" not in name or not kept:       # tiles of 256 x 256, four blocks of 32 a wave
            continue
        seen += 1
        assert all(code[i - 1] == "s_nop 1" for i in kept), name
        reads = [i for i, t in enumerate(code) if READ.match(t)]
        for i in reads:
            before = [k for k in kept if k < i]
            if not before:
                continue
            between = code[before[-1]:i]
            waits = [k for k, t in enumerate(between) if t == "s_nop 15"]
            assert waits and between[waits[0] + 1] == "s_nop 7", (name, i)
    assert seen >= 6          # forward of two types and activations, dx and dw of two types


def test_no_atomics_and_no_scratch(attention):  # noqa: F811
    found = feed_forward(attention)
    assert found
    for name, code in found.items():
        assert not [t for t in code if re.match(r"(global|buffer|flat|ds)_\w*(atomic|add|max|min)\w*", t)], name
        assert not [t for t in code if t.startswith("scratch_")], name
