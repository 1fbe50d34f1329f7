"""The packed attention entry points without a GPU: refusals, workspace sizes,
what is rejected by the binding, and what their kernels' code objects hold.
Nothing here reaches a HIP call.
"""
import os
import re
import subprocess

import pytest
import torch
import yaml

import diffusion_transformer_qk_amd as qkr
from diffusion_transformer_qk_amd import binding as b
from tests.test_attention_cpu import A, FAR, LLVM, needs_tools, objects, tensor  # noqa: F401 (a fixture)


def args(**over):
    v = dict(sequences=3, q_tokens=100, kv_tokens=200, heads=8, kv_heads=4, head_dim=64, causal=0, dtype=b.QKR_BF16,
             scale=0.125, fill_rest=0, q_offsets=A + 10 * FAR, kv_offsets=A + 11 * FAR)
    v.update(over)
    return b.AttnPackedArgs(**v)


def forward(a=None, **over):
    a = args() if a is None else a
    d = a.head_dim
    t = dict(q=tensor(A, a.q_tokens, a.heads, d), k=tensor(A + FAR, a.kv_tokens, a.kv_heads, d),
             v=tensor(A + 2 * FAR, a.kv_tokens, a.kv_heads, d), out=tensor(A + 3 * FAR, a.q_tokens, a.heads, d),
             lse=A + 4 * FAR, ws=A + 5 * FAR, ws_bytes=1 << 40)
    t.update(over)
    return b.load_library().dit_attention_packed(a, *t.values(), 0)


def backward(a=None, **over):
    a = args() if a is None else a
    d = a.head_dim
    names = ("dout", "q", "k", "v", "out", "dq", "dk", "dv")
    t = {n: tensor(A + i * FAR, *((a.kv_tokens, a.kv_heads) if n[-1] in "kv" else (a.q_tokens, a.heads)), d)
         for i, n in enumerate(names)}
    t.update(lse=A + 8 * FAR, ws=A + 9 * FAR, ws_bytes=1 << 40)
    t.update(over)
    return b.load_library().dit_attention_packed_backward(
        a, *(t[n] for n in names[:5]), t["lse"], *(t[n] for n in names[5:]), t["ws"], t["ws_bytes"], 0)


@pytest.mark.parametrize("over,code", [
    (dict(head_dim=96), b.QKR_ERR_UNSUPPORTED), (dict(dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED),
    (dict(dtype=3), b.QKR_ERR_ARG), (dict(causal=2), b.QKR_ERR_ARG), (dict(scale=0.0), b.QKR_ERR_ARG),
    (dict(scale=float("nan")), b.QKR_ERR_ARG), (dict(fill_rest=2), b.QKR_ERR_ARG), (dict(fill_rest=-1), b.QKR_ERR_ARG),
    (dict(sequences=-1), b.QKR_ERR_SHAPE), (dict(sequences=1 << 24), b.QKR_ERR_SHAPE),
    (dict(sequences=1 << 21), b.QKR_ERR_SHAPE), (dict(q_tokens=-1), b.QKR_ERR_SHAPE),
    (dict(q_tokens=1 << 24), b.QKR_ERR_SHAPE), (dict(kv_tokens=1 << 24), b.QKR_ERR_SHAPE),
    (dict(kv_heads=0), b.QKR_ERR_SHAPE), (dict(heads=7), b.QKR_ERR_SHAPE),
    (dict(q_tokens=(1 << 24) - 1, heads=64, kv_heads=1), b.QKR_ERR_SHAPE)])
def test_bad_arguments(over, code):
    a = args(**over)
    lib = b.load_library()
    assert lib.dit_attention_packed_workspace_size(a) == code
    assert lib.dit_attention_packed_backward_workspace_size(a) == code
    assert forward(a) == code and backward(a) == code


def test_missing_misaligned_and_shared():
    lib = b.load_library()
    assert lib.dit_attention_packed_workspace_size(None) == b.QKR_ERR_NULL
    for f in (forward, backward):
        assert f(lse=0) == b.QKR_ERR_NULL and f(args(q_offsets=None)) == b.QKR_ERR_NULL
        assert f(lse=A + 8 * FAR + 2) == b.QKR_ERR_ALIGN
        assert f(args(q_offsets=A + 10 * FAR + 2)) == b.QKR_ERR_ALIGN
        assert f(args(kv_offsets=A + 10 * FAR + 1)) == b.QKR_ERR_ALIGN
    for name in ("q", "k", "v", "out"):
        assert forward(**{name: None}) == b.QKR_ERR_NULL
    for name in ("dout", "q", "k", "v", "out", "dq", "dk", "dv"):
        assert backward(**{name: None}) == b.QKR_ERR_NULL
    for offset in ("q_offsets", "kv_offsets"):
        for i in (3, 4):                                   # out, lse
            assert forward(args(**{offset: A + i * FAR})) == b.QKR_ERR_ARG
        for i in (5, 6, 7, 9):                             # dq, dk, dv, the workspace
            assert backward(args(**{offset: A + i * FAR})) == b.QKR_ERR_ARG
    assert forward(out=tensor(A + 16, 100, 8)) == b.QKR_ERR_ARG and forward(lse=A + 64) == b.QKR_ERR_ARG
    assert forward(out=tensor(A + 3 * FAR, 100, 8, token_stride=504)) == b.QKR_ERR_ARG
    assert forward(q=tensor(A + 8, 100, 8)) == b.QKR_ERR_ALIGN
    # one sample: the batch's stride does not count
    assert forward(q=tensor(A, 100, 8, batch_stride=3), out=tensor(A, 100, 8, batch_stride=-5)) == b.QKR_ERR_ARG
    assert backward(dk=tensor(A + 7 * FAR, 200, 4)) == b.QKR_ERR_ARG


def test_workspaces():
    size = qkr.attention_packed_workspace_size
    need = size(3, 100, 200, 8, 4, 64, backward=True)
    assert need >= 2 * 8 * 100 * 4
    assert backward(ws=0) == b.QKR_ERR_WORKSPACE and backward(ws_bytes=need - 1) == b.QKR_ERR_WORKSPACE
    assert backward(ws=A + 9 * FAR + 8) == b.QKR_ERR_ALIGN
    one = args(sequences=2, q_tokens=2, kv_tokens=30000, heads=40, kv_heads=8, head_dim=128)
    need = size(2, 2, 30000, 40, 8, 128)
    assert need > 0 and need % (2 * 40 * 129 * 4) == 0
    assert forward(one, ws=0) == b.QKR_ERR_WORKSPACE and forward(one, ws_bytes=need - 1) == b.QKR_ERR_WORKSPACE
    assert size(6, 8190, 8190, 40, 40, 128) == 0              # a call that fills the chip by itself
    assert size(3, 10, 10, 3, 2, 128) == b.QKR_ERR_SHAPE


def test_nothing_to_do():
    assert forward(args(q_tokens=0), q=None, out=None, lse=0) == b.QKR_OK
    assert backward(args(q_tokens=0, kv_tokens=0)) == b.QKR_OK


def test_binding_refuses_what_does_not_fit():
    q = torch.zeros((10, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((20, 2, 64), dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        qkr.attention_packed(q, k, k, o, kv_offsets=o)
    for bad in (dict(kv_offsets=None), dict(offsets=o.long()), dict(offsets=o[:0]), dict(offsets=o[None]), dict(kv_offsets=o[:2]),
                dict(kv_offsets=o.long()), dict(q=q[None]), dict(k=k[:, :, :32]), dict(v=k[:5]), dict(k=k.half()),
                dict(k=k[:, :0], v=k[:, :0]), dict(q=q[:, :3]), dict(out=q[:5]), dict(out=q.half()), dict(lse=torch.zeros(10, 4))):
        t = dict(dict(q=q, k=k, v=k, offsets=o, kv_offsets=o), **bad)
        with pytest.raises(ValueError):
            qkr.attention_packed(t.pop("q"), t.pop("k"), t.pop("v"), t.pop("offsets"), **t)
    lse = torch.zeros((4, 10))
    for bad in (dict(dout=q[:9]), dict(out=q.half()), dict(dq=k), dict(dk=q), dict(dv=k[:1]), dict(lse=lse[:1])):
        t = dict(dict(dout=q, out=q, lse=lse), **bad)
        with pytest.raises(ValueError):
            qkr.attention_packed_backward(t.pop("dout"), q, k, k, t.pop("out"), t.pop("lse"), o, kv_offsets=o, **t)


@needs_tools
def test_kernels_do_not_spill_and_keep_their_waves(objects):  # noqa: F811
    kernels = []
    for co in objects:
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", co], check=True, capture_output=True,
                               text=True).stdout
        doc = notes[notes.index("---"):]
        kernels += yaml.safe_load(doc[:doc.index("\n...")] if "\n..." in doc else doc)["amdhsa.kernels"]
    # 3 head sizes x 2 types x 2 maskings, forward with 1 and 4 waves
    assert sum("packed_forward_kernel" in k[".name"] for k in kernels) == 24
    assert sum("packed_backward_kernel" in k[".name"] for k in kernels) == 12
    for k in kernels:
        m = re.search(r"packed_(forward|backward)_kernelILi(\d+)E", k[".name"])
        if m and not k[".name"].count("ELi1EEE"):
            assert not (k[".private_segment_fixed_size"] or k[".vgpr_spill_count"]), k[".name"]
            waves = {("forward", "64"): 4, ("forward", "128"): 3, ("forward", "256"): 2,
                     ("backward", "64"): 3, ("backward", "128"): 2, ("backward", "256"): 1}[m.groups()]
            assert 512 // (-(-k[".vgpr_count"] // 8) * 8) >= waves, (k[".name"], k[".vgpr_count"])
            assert waves * k[".group_segment_fixed_size"] <= 160 * 1024
