"""Instruction checks on the attention library's gfx950 code, and on both
libraries' scalar memory instructions (CPU, no GPU).

  * A load straight into LDS reads its buffer resource from scalar registers.
    A vector instruction (the compiler keeps scalars it has no room for in
    lanes of vector registers) must not have written one of those in the five
    wait states before, and inside inline assembly the compiler inserts no
    waits of its own.  So those wait states may hold nothing but the assembly's
    own instructions, whatever the compiler puts in front of it.
  * Scalar memory instructions are told by their encoding; all are loads.
"""
import os
import re
import subprocess

import pytest

from diffusion_transformer_qk_amd import build
from tests.test_attention_cpu import objects as attention_objects  # noqa: F401 (a fixture)
from tests.test_code_object import LLVM, TOOLS, _code_objects

OBJDUMP = os.path.join(LLVM, "llvm-objdump")

pytestmark = pytest.mark.skipif(
    not all(os.path.exists(os.path.join(LLVM, t)) for t in TOOLS) or not os.path.exists(OBJDUMP),
    reason="ROCm LLVM tools not available")

LDS_LOAD = re.compile(r"buffer_load_dword(x4)? v\d+, s\[\d+:\d+\], 0 offen( offset:\d+)? lds$")
OWN = re.compile(r"s_nop \d+$|s_mov_b32 m0, s\d+$|s_add_u32 m0, m0, ")
SCALAR_MEMORY = {"s_load_dword", "s_load_dwordx2", "s_load_dwordx4", "s_load_dwordx8", "s_load_dwordx16"}


def kernels(paths):
    """{kernel symbol: [(instruction, first word of its encoding)]}."""
    out = {}
    for co in paths:
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", co], check=True, capture_output=True,
                              text=True).stdout
        current = None
        for line in text.splitlines():
            m = re.match(r"^[0-9a-f]+ <(\w+)>:", line)
            if m:
                current = out.setdefault(m.group(1), [])
                continue
            m = re.match(r"^\t(.*?)\s*// [0-9A-F]+: ([0-9A-F]{8})", line)
            if m and current is not None:
                current.append((" ".join(m.group(1).split()), int(m.group(2), 16)))
    return out


@pytest.fixture(scope="module")
def attention(attention_objects):  # noqa: F811
    return kernels(attention_objects)


def test_loads_into_lds_have_their_wait_states(attention):
    assert os.path.exists(build.ATTN_LIB)
    seen = 0
    for name, code in attention.items():
        for i, (text, _) in enumerate(code):
            if not re.search(r"\slds$", text):
                continue
            assert LDS_LOAD.match(text), (name, text)
            seen += 1
            states, j = 0, i
            while states < 5:
                j -= 1
                before = code[j][0]
                assert OWN.match(before) or LDS_LOAD.match(before), (name, [c[0] for c in code[j:i + 1]])
                states += int(before.split()[1]) + 1 if before.startswith("s_nop") else 1
    assert seen >= 48 * 8


@pytest.mark.parametrize("library", ["attention", "main"])
def test_scalar_memory_instructions_are_loads(library, request, tmp_path):
    code = request.getfixturevalue("attention") if library == "attention" else kernels(_code_objects(str(tmp_path)))
    assert len(code) > 50
    # the encoding's upper six bits are 110000
    used = {text.split()[0] for body in code.values() for text, word in body if word >> 26 == 0x30}
    assert used and used <= SCALAR_MEMORY, used - SCALAR_MEMORY
