"""Attention's entry points without a GPU: refusals, sizes, and what its code
objects hold.  Every call here is rejected (or has nothing to do) before any
HIP call; pointers are fake and never dereferenced.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch
import yaml

import diffusion_transformer_qk_amd as qkr
from diffusion_transformer_qk_amd import binding as b
from diffusion_transformer_qk_amd import build
from tests.test_code_object import LLVM, MAGIC, TARGET, TOOLS

A = 1 << 20
FAR = 1 << 30          # steps between the fake tensors of a call


def args(**over):
    v = dict(batch=2, q_tokens=100, kv_tokens=200, heads=8, kv_heads=4, head_dim=64, causal=0,
             dtype=b.QKR_BF16, scale=0.125, kv_lengths=None)
    v.update(over)
    return b.AttnArgs(**v)


def tensor(at, tokens, heads, d=64, **over):
    v = dict(data=at, batch_stride=tokens * heads * d, token_stride=heads * d, head_stride=d)
    v.update(over)
    return b.AttnTensor(**v)


def forward(a=None, **over):
    a = args() if a is None else a
    d = a.head_dim
    t = dict(q=tensor(A, a.q_tokens, a.heads, d), k=tensor(A + FAR, a.kv_tokens, a.kv_heads, d),
             v=tensor(A + 2 * FAR, a.kv_tokens, a.kv_heads, d), out=tensor(A + 3 * FAR, a.q_tokens, a.heads, d),
             lse=A + 4 * FAR, ws=A + 5 * FAR, ws_bytes=1 << 40)
    t.update(over)
    return b.load_library().dit_attention(a, t["q"], t["k"], t["v"], t["out"], t["lse"], t["ws"], t["ws_bytes"], 0)


def backward(a=None, **over):
    a = args() if a is None else a
    d = a.head_dim
    names = ("dout", "q", "k", "v", "out", "dq", "dk", "dv")
    t = {n: tensor(A + i * FAR, *((a.kv_tokens, a.kv_heads) if n[-1] in "kv" else (a.q_tokens, a.heads)), d)
         for i, n in enumerate(names)}
    t.update(lse=A + 8 * FAR, ws=A + 9 * FAR, ws_bytes=1 << 40)
    t.update(over)
    return b.load_library().dit_attention_backward(
        a, *(t[n] for n in names[:5]), t["lse"], *(t[n] for n in names[5:]), t["ws"], t["ws_bytes"], 0)


BAD_ARGS = [
    (dict(head_dim=96), b.QKR_ERR_UNSUPPORTED), (dict(head_dim=0), b.QKR_ERR_UNSUPPORTED),
    (dict(head_dim=512), b.QKR_ERR_UNSUPPORTED), (dict(dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED),
    (dict(dtype=3), b.QKR_ERR_ARG), (dict(dtype=-1), b.QKR_ERR_ARG),
    (dict(causal=2), b.QKR_ERR_ARG), (dict(scale=0.0), b.QKR_ERR_ARG), (dict(scale=-1.0), b.QKR_ERR_ARG),
    (dict(scale=float("nan")), b.QKR_ERR_ARG), (dict(scale=float("inf")), b.QKR_ERR_ARG),
    (dict(scale=3e38), b.QKR_ERR_ARG),
    (dict(batch=-1), b.QKR_ERR_SHAPE), (dict(q_tokens=-1), b.QKR_ERR_SHAPE), (dict(kv_tokens=-1), b.QKR_ERR_SHAPE),
    (dict(q_tokens=1 << 24), b.QKR_ERR_SHAPE), (dict(kv_tokens=1 << 24), b.QKR_ERR_SHAPE),
    (dict(kv_heads=0), b.QKR_ERR_SHAPE), (dict(heads=7), b.QKR_ERR_SHAPE), (dict(heads=2), b.QKR_ERR_SHAPE),
    (dict(heads=65537, kv_heads=65537), b.QKR_ERR_SHAPE), (dict(batch=1 << 21), b.QKR_ERR_SHAPE),
    (dict(q_tokens=(1 << 24) - 1, heads=64, kv_heads=1), b.QKR_ERR_SHAPE),
    (dict(batch=200, heads=65536, kv_heads=1, q_tokens=1), b.QKR_ERR_SHAPE),
]


@pytest.mark.parametrize("over,code", BAD_ARGS)
def test_bad_arguments(over, code):
    a = args(**over)
    lib = b.load_library()
    assert lib.dit_attention_workspace_size(a) == code
    assert lib.dit_attention_backward_workspace_size(a) == code
    assert forward(a) == code and backward(a) == code


def test_missing_arguments():
    lib = b.load_library()
    assert lib.dit_attention_workspace_size(None) == b.QKR_ERR_NULL
    assert forward(lse=0) == b.QKR_ERR_NULL and backward(lse=0) == b.QKR_ERR_NULL
    for name in ("q", "k", "v", "out"):
        assert forward(**{name: None}) == b.QKR_ERR_NULL
    for name in ("dout", "q", "k", "v", "out", "dq", "dk", "dv"):
        assert backward(**{name: None}) == b.QKR_ERR_NULL
        assert backward(**{name: tensor(0, 100, 8)}) == b.QKR_ERR_NULL


@pytest.mark.parametrize("over,code", [
    (dict(data=A + 8), b.QKR_ERR_ALIGN), (dict(token_stride=516), b.QKR_ERR_ALIGN),
    (dict(batch_stride=100 * 512 + 4), b.QKR_ERR_ALIGN), (dict(head_stride=65), b.QKR_ERR_ALIGN),
    (dict(token_stride=-512), b.QKR_ERR_SHAPE), (dict(head_stride=-64), b.QKR_ERR_SHAPE),
    (dict(batch_stride=-8), b.QKR_ERR_SHAPE), (dict(token_stride=(1 << 22) + 8), b.QKR_ERR_SHAPE),
    (dict(batch_stride=(1 << 44) + 8), b.QKR_ERR_SHAPE),
    (dict(token_stride=56), b.QKR_ERR_SHAPE), (dict(token_stride=0), b.QKR_ERR_SHAPE),
])
def test_bad_layouts(over, code):
    assert forward(q=tensor(A, 100, 8, **over)) == code
    assert forward(out=tensor(A + 3 * FAR if over.get("data") is None else over["data"], 100, 8,
                              **{k: v for k, v in over.items() if k != "data"})) == code
    t = {k: v for k, v in over.items() if k != "data"}
    assert backward(dq=tensor(over.get("data", A + 5 * FAR), 100, 8, **t)) == code


def test_strides_whose_spans_would_wrap():
    """A span of 2^64 bytes would count as none, and its overlaps as none."""
    a = args(batch=1 << 20, q_tokens=1, kv_tokens=1, heads=1, kv_heads=1)
    for stride in (1 << 43, (1 << 38) + 8):
        assert forward(a, out=tensor(A + FAR, 1, 1, batch_stride=stride)) == b.QKR_ERR_SHAPE
        assert backward(a, dq=tensor(A + FAR, 1, 1, batch_stride=stride)) == b.QKR_ERR_SHAPE
    assert forward(a, out=tensor(A + FAR, 1, 1, batch_stride=1 << 38)) == b.QKR_ERR_ARG


def test_outputs_must_not_share_memory():
    # with themselves
    assert forward(out=tensor(A + 3 * FAR, 100, 8, head_stride=0)) == b.QKR_ERR_ARG
    assert forward(out=tensor(A + 3 * FAR, 100, 8, batch_stride=0)) == b.QKR_ERR_ARG
    assert forward(out=tensor(A + 3 * FAR, 100, 8, token_stride=504)) == b.QKR_ERR_ARG
    assert backward(dk=tensor(A + 6 * FAR, 200, 4, head_stride=56)) == b.QKR_ERR_ARG
    # with other tensors
    for name in ("q", "k", "v"):
        at = {"q": A, "k": A + FAR, "v": A + 2 * FAR}[name]
        assert forward(out=tensor(at + 16, 100, 8)) == b.QKR_ERR_ARG
    assert forward(lse=A + 64) == b.QKR_ERR_ARG and forward(lse=A + 3 * FAR) == b.QKR_ERR_ARG
    a = args(kv_lengths=A + 3 * FAR + 16)
    assert forward(a) == b.QKR_ERR_ARG
    names = ("dout", "q", "k", "v", "out", "dq", "dk", "dv")
    for i, name in enumerate(names[:7]):
        n = (200, 4) if name[-1] in "kv" else (100, 8)
        assert backward(**{name: tensor(A + 7 * FAR, *n)}) == b.QKR_ERR_ARG, name
    assert backward(lse=A + 7 * FAR) == b.QKR_ERR_ARG
    for i in range(9):
        assert backward(ws=A + i * FAR) == b.QKR_ERR_ARG


def test_slices_of_one_buffer_are_told_apart():
    """Slices of a fused buffer interleave without sharing; an out that reaches
    into one of them, or that cannot be told apart, is refused.  (That slices
    which only interleave are taken needs a launch: the GPU tests have it.)"""
    a = args(batch=2, q_tokens=100, kv_tokens=100, heads=4, kv_heads=4)
    row = 4 * 4 * 64
    f = {n: dict(batch_stride=100 * row, token_stride=row) for n in "qkvo"}
    t = {n: tensor(A + 2 * 256 * i, 100, 4, **f[n]) for i, n in enumerate("qkvo")}
    shifted = tensor(A + 2 * 256 * 3 - 16, 100, 4, **f["o"])
    assert forward(a, q=t["q"], k=t["k"], v=t["v"], out=shifted) == b.QKR_ERR_ARG
    other = tensor(A + 2 * 256 * 3, 100, 4, batch_stride=100 * row + 8, token_stride=row)
    assert forward(a, q=t["q"], k=t["k"], v=t["v"], out=other) == b.QKR_ERR_ARG


def test_workspaces():
    lib = b.load_library()
    a = args()
    need = lib.dit_attention_backward_workspace_size(a)
    assert need >= 2 * 8 * 100 * 8
    assert backward(a, ws=0) == b.QKR_ERR_WORKSPACE and backward(a, ws_bytes=need - 1) == b.QKR_ERR_WORKSPACE
    assert backward(a, ws=A + 9 * FAR + 8) == b.QKR_ERR_ALIGN
    one = args(q_tokens=1, kv_tokens=32760, heads=40, kv_heads=8, head_dim=128, batch=1)
    need = lib.dit_attention_workspace_size(one)
    assert need > 0 and need % (40 * 129 * 4) == 0      # one partial row and its lse a split
    assert forward(one, ws=0) == b.QKR_ERR_WORKSPACE and forward(one, ws_bytes=need - 1) == b.QKR_ERR_WORKSPACE
    assert forward(one, ws=A + 5 * FAR + 4) == b.QKR_ERR_ALIGN
    # a call that fills the chip by itself needs none
    assert qkr.attention_workspace_size(1, 4608, 4608, 48, 48, 128) == 0
    assert qkr.attention_workspace_size(1, 10, 10, 3, 2, 128) == b.QKR_ERR_SHAPE


def test_tensors_without_tokens_may_be_missing():
    """They get past the checks of the pointers (to the first other fault)."""
    assert forward(args(kv_tokens=0), k=None, v=None, lse=0) == b.QKR_ERR_NULL
    assert forward(args(kv_tokens=0), k=None, v=None, lse=A) == b.QKR_ERR_ARG
    assert backward(args(kv_tokens=0), k=None, v=None, dk=None, dv=None, ws=A) == b.QKR_ERR_ARG
    assert backward(args(q_tokens=0), dout=None, q=None, out=None, dq=None, lse=0,
                    dk=tensor(A + 3 * FAR, 200, 4)) == b.QKR_ERR_ARG


def test_nothing_to_do():
    assert forward(args(batch=0)) == b.QKR_OK and backward(args(batch=0)) == b.QKR_OK
    assert forward(args(q_tokens=0)) == b.QKR_OK
    assert backward(args(q_tokens=0, kv_tokens=0)) == b.QKR_OK


def test_binding_refuses_what_does_not_fit():
    q = torch.zeros((2, 10, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((2, 20, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        qkr.attention(q, k, k)
    for bad in (dict(k=k[:, :, :, :32]), dict(k=k[:1]), dict(v=k[:, :5]), dict(k=k.half()), dict(q=q[0, 0]),
                dict(q=q.float(), k=k.float(), v=k.float()), dict(k=k[:, :, :0], v=k[:, :, :0]),
                dict(q=q[:, :, :3]), dict(kv_lengths=torch.zeros(2)), dict(kv_lengths=torch.zeros(3, dtype=torch.int32)),
                dict(lse=torch.zeros(2, 10, 4)), dict(out=q[:, :5]), dict(out=q.half())):
        t = dict(dict(q=q, k=k, v=k), **bad)
        with pytest.raises(ValueError):
            qkr.attention(t.pop("q"), t.pop("k"), t.pop("v"), **t)
    lse = torch.zeros((2, 4, 10))
    for bad in (dict(dout=q[:, :9]), dict(out=q.half()), dict(dq=k), dict(dk=q), dict(dv=k[:1]), dict(lse=lse[:1])):
        t = dict(dict(dout=q, out=q, lse=lse), **bad)
        with pytest.raises(ValueError):
            qkr.attention_backward(t.pop("dout"), q, k, k, t.pop("out"), t.pop("lse"), **t)


# ------------------------------------------------------------------ the code objects

needs_tools = pytest.mark.skipif(not all(os.path.exists(os.path.join(LLVM, t)) for t in TOOLS),
                                 reason="ROCm LLVM tools not available")


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    tmp = str(tmp_path_factory.mktemp("attention_objects"))
    fat = os.path.join(tmp, "fat.bin")
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section", ".hip_fatbin=" + fat,
                    build.ATTN_LIB], check=True)
    with open(fat, "rb") as f:
        data = f.read()
    starts = [m.start() for m in re.finditer(re.escape(MAGIC), data)] + [len(data)]
    paths = []
    for n, (i, j) in enumerate(zip(starts, starts[1:])):
        part, co = (os.path.join(tmp, "%s%d" % (s, n)) for s in ("bundle", "co"))
        with open(part, "wb") as f:
            f.write(data[i:j])
        subprocess.run([os.path.join(LLVM, "clang-offload-bundler"), "--unbundle", "--type=o",
                        "--targets=" + TARGET, "--input=" + part, "--output=" + co], check=True)
        paths.append(co)
    return paths


@needs_tools
def test_kernels_do_not_spill_and_keep_their_waves(objects):
    kernels = []
    for co in objects:
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", co], check=True,
                               capture_output=True, text=True).stdout
        doc = notes[notes.index("---"):]
        kernels += yaml.safe_load(doc[:doc.index("\n...")] if "\n..." in doc else doc)["amdhsa.kernels"]
    # 3 head sizes x 2 types x 2 maskings, forward with 1 and 4 waves
    assert sum("attention_forward_kernel" in k[".name"] for k in kernels) == 24
    # and backward with one term of p and ds and with two
    assert sum("attention_backward_kernel" in k[".name"] for k in kernels) == 24
    for k in kernels:
        # (scalar registers may be parked in lanes of a vector register, not in memory)
        assert not (k[".private_segment_fixed_size"] or k[".vgpr_spill_count"]), k[".name"]
        assert k[".group_segment_fixed_size"] <= 160 * 1024
        m = re.search(r"attention_(forward|backward)_kernelILi(\d+)E", k[".name"])
        # the kernels for few rows (forward: one wave; backward: two terms) take what they need
        if m and not k[".name"].count("ELi1EEE") and not ("backward" in k[".name"] and "Lb1EEE" in k[".name"]):
            waves = {("forward", "64"): 4, ("forward", "128"): 3, ("forward", "256"): 2,
                     ("backward", "64"): 3, ("backward", "128"): 2, ("backward", "256"): 1}[m.groups()]
            assert 512 // (-(-k[".vgpr_count"] // 8) * 8) >= waves, (k[".name"], k[".vgpr_count"])
            assert waves * k[".group_segment_fixed_size"] <= 160 * 1024


@needs_tools
def test_products_run_on_the_matrix_cores(objects):
    text = "".join(subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", co], check=True,
                                  capture_output=True, text=True).stdout for co in objects)
    assert "v_mfma_f32_32x32x16_bf16" in text and "v_mfma_f32_32x32x16_f16" in text
    assert not re.search(r"\sv_pk_(add|mul|fma)_f32", text)
    # no atomic additions anywhere: results do not depend on the order of workgroups
    assert not re.search(r"\s(global|buffer|flat|ds)_atomic", text) and not re.search(r"\sds_add", text)


def test_the_main_library_brings_the_attention_library_along():
    out = subprocess.run(["readelf", "-d", qkr.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert "libdit_attention.so" in out and "$ORIGIN" in out
    names = subprocess.run(["nm", "-D", "--undefined-only", build.ATTN_LIB], capture_output=True, text=True,
                           check=True).stdout
    assert "getenv" not in names
    assert ctypes.CDLL(qkr.LIB_PATH).dit_attention


def test_strides_of_a_dimension_of_one_do_not_count():
    """They get past the checks of the layouts (to the overlap of q and out)."""
    a = args(batch=1, q_tokens=1, kv_tokens=1, heads=1, kv_heads=1)
    for stride in (3, -8, 1 << 40, (1 << 22) + 8):
        over = dict(batch_stride=stride, token_stride=stride, head_stride=stride)
        t = [tensor(A + i * FAR, 1, 1, **over) for i in range(9)]
        assert forward(a, q=t[0], k=t[1], v=t[2], out=t[0]) == b.QKR_ERR_ARG
        assert forward(a, q=t[0], k=t[1], v=t[2], out=t[3], lse=A + 3 * FAR) == b.QKR_ERR_ARG
        assert backward(a, dout=t[0], q=t[1], k=t[2], v=t[3], out=t[4], dq=t[5], dk=t[6], dv=t[6]) == b.QKR_ERR_ARG
        assert backward(a, dq=tensor(A, 1, 1, batch_stride=1, token_stride=stride, head_stride=stride,
                                     data=A + 5 * FAR + 8)) == b.QKR_ERR_ALIGN
    # and of more than one they do
    two = args(batch=1, q_tokens=2, kv_tokens=1, heads=1, kv_heads=1)
    assert forward(two, q=tensor(A, 2, 1, token_stride=3)) == b.QKR_ERR_ALIGN
    assert forward(two, q=tensor(A, 2, 1, token_stride=(1 << 22) + 8)) == b.QKR_ERR_SHAPE
