"""The gated feed-forward entry points without a GPU: refusals, workspace sizes
and what is rejected by the binding.  Nothing here reaches a HIP call.
"""
import os
import shutil
import subprocess

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from diffusion_transformer_qk_amd import binding as b

A = 1 << 20
FAR = 1 << 34
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def args(**over):
    v = dict(rows=100, hidden=512, inner=1024, activation=0, dtype=b.QKR_BF16, out_dtype=b.QKR_BF16)
    v.update(over)
    return b.FfArgs(**v)


def forward(a=None, **over):
    a = args() if a is None else a
    fp8 = a.dtype == b.DIT_FF_E4M3
    v = dict(x=A, w_gate=A + FAR, w_up=A + 2 * FAR, xs=A + 3 * FAR if fp8 else 0, gs=A + 4 * FAR if fp8 else 0,
             us=A + 5 * FAR if fp8 else 0, h=A + 6 * FAR, gate=A + 7 * FAR, up=A + 8 * FAR)
    v.update(over)
    return b.load_library().dit_gated_feed_forward(a, *v.values(), 0)


def backward(a=None, **over):
    a = args() if a is None else a
    v = dict(dh=A, x=A + FAR, w_gate=A + 2 * FAR, w_up=A + 3 * FAR, gate=A + 4 * FAR, up=A + 5 * FAR, dx=A + 6 * FAR,
             dw_gate=A + 7 * FAR, dw_up=A + 8 * FAR, ws=A + 9 * FAR, ws_bytes=1 << 40)
    v.update(over)
    return b.load_library().dit_gated_feed_forward_backward(a, *v.values(), 0)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), b.QKR_ERR_SHAPE), (dict(rows=1 << 24), b.QKR_ERR_SHAPE),
    (dict(rows=(1 << 24) - 1, inner=1 << 17), b.QKR_ERR_SHAPE), (dict(rows=(1 << 24) - 1, hidden=1 << 17), b.QKR_ERR_SHAPE),
    (dict(hidden=0), b.QKR_ERR_UNSUPPORTED), (dict(hidden=12), b.QKR_ERR_UNSUPPORTED), (dict(inner=4), b.QKR_ERR_UNSUPPORTED),
    (dict(inner=-8), b.QKR_ERR_UNSUPPORTED), (dict(hidden=(1 << 17) + 8), b.QKR_ERR_UNSUPPORTED),
    (dict(inner=(1 << 17) + 8), b.QKR_ERR_UNSUPPORTED), (dict(activation=2), b.QKR_ERR_ARG), (dict(activation=-1), b.QKR_ERR_ARG),
    (dict(dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED), (dict(dtype=3), b.QKR_ERR_ARG), (dict(dtype=-1), b.QKR_ERR_ARG),
    (dict(out_dtype=b.QKR_FP16), b.QKR_ERR_ARG), (dict(out_dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED),
    (dict(out_dtype=8), b.QKR_ERR_ARG)])
def test_bad_arguments(over, code):
    a = args(**over)
    lib = b.load_library()
    assert forward(a) == code and backward(a) == code
    assert lib.dit_gated_feed_forward_backward_workspace_size(a) == code


def test_8_bits():
    a = args(dtype=b.DIT_FF_E4M3)
    assert backward(a) == b.QKR_ERR_UNSUPPORTED
    assert forward(args(dtype=b.DIT_FF_E4M3, hidden=520)) == b.QKR_ERR_UNSUPPORTED
    assert forward(args(dtype=b.DIT_FF_E4M3, inner=1032)) == b.QKR_ERR_UNSUPPORTED
    for name in ("xs", "gs", "us"):
        assert forward(a, **{name: 0}) == b.QKR_ERR_NULL
        assert forward(a, **{name: A + 3 * FAR + 2}) == b.QKR_ERR_ALIGN
        assert forward(**{name: A + 3 * FAR}) == b.QKR_ERR_ARG
        assert forward(a, **{name: A + 6 * FAR + 64}) == b.QKR_ERR_ARG


def test_missing_and_misaligned():
    lib = b.load_library()
    assert lib.dit_gated_feed_forward_backward_workspace_size(None) == b.QKR_ERR_NULL
    for name in ("x", "w_gate", "w_up", "h", "gate", "up"):
        assert forward(**{name: 0}) == b.QKR_ERR_NULL, name
    for name in ("dh", "x", "w_gate", "w_up", "gate", "up", "dw_gate", "dw_up"):
        assert backward(**{name: 0}) == b.QKR_ERR_NULL, name
    for i, name in enumerate(("x", "w_gate", "w_up")):
        assert forward(**{name: A + i * FAR + 8}) == b.QKR_ERR_ALIGN
    for i, name in enumerate(("h", "gate", "up")):
        assert forward(**{name: A + (6 + i) * FAR + 8}) == b.QKR_ERR_ALIGN
    for i, name in enumerate(("dh", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up", "ws")):
        assert backward(**{name: A + i * FAR + 8}) == b.QKR_ERR_ALIGN, name


def test_outputs_must_not_share_memory():
    for i in range(3):
        for name in ("h", "gate", "up"):
            assert forward(**{name: A + i * FAR}) == b.QKR_ERR_ARG
    assert forward(gate=A + 6 * FAR) == b.QKR_ERR_ARG and forward(up=A + 7 * FAR + 1024) == b.QKR_ERR_ARG
    for i in range(6):
        for name in ("dx", "dw_gate", "dw_up", "ws"):
            assert backward(**{name: A + i * FAR}) == b.QKR_ERR_ARG, (i, name)
    assert backward(dw_up=A + 7 * FAR) == b.QKR_ERR_ARG and backward(ws=A + 6 * FAR) == b.QKR_ERR_ARG


def test_workspaces():
    size = qkr.gated_feed_forward_backward_workspace_size
    need = size(100, 512, 1024)
    assert need >= 4 * 100 * 1024 and need % 16 == 0
    assert backward(ws=0) == b.QKR_ERR_WORKSPACE and backward(ws_bytes=need - 1) == b.QKR_ERR_WORKSPACE
    assert size(0, 512, 1024) == 0 and size(-1, 8, 8) == b.QKR_ERR_SHAPE and size(1, 8, 12) == b.QKR_ERR_UNSUPPORTED
    assert need < size(100, 512, 1024, dtype=b.QKR_FP16) <= need + 4 * 2048
    # products that fill the chip by themselves are not split
    assert size(4608, 6144, 16384) == 4 * 4608 * 16384
    # dx of few rows is, and dw of many rows of narrow weights: partial sums in fp32
    assert size(16, 5120, 13824) > 4 * 16 * 13824 + 2 * 4 * 16 * 5120
    assert size(16384, 512, 2048) > 4 * 16384 * 2048 + 2 * 4 * 2 * 2048 * 512


def test_nothing_to_do():
    assert forward(args(rows=0), x=0, h=0) == b.QKR_OK
    assert backward(dx=0, dw_gate=0, dw_up=0, dh=0) == b.QKR_OK
    assert backward(args(rows=0), dw_gate=0, dw_up=0) == b.QKR_OK


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((32, 64), dtype=torch.bfloat16)
    h = torch.zeros((4, 32), dtype=torch.bfloat16)
    one = torch.ones(4)
    with pytest.raises(ValueError, match="GPU"):
        qkr.gated_feed_forward(x, w, w)
    for a, kw in (((x, w, w[:16]), {}), ((x, w.half(), w), {}), ((x, w[0], w[0]), {}), ((x[:, :32], w, w), {}),
                  ((x.float(), w.float(), w.float()), {}), ((x, w, w), dict(activation="relu")),
                  ((x, w, w), dict(x_scale=one)), ((x, w, w), dict(out_dtype=torch.float16)), ((x, w, w), dict(out=h[:2])),
                  ((x, w, w), dict(gate=h)), ((x, w, w), dict(save=True, up=h.half())),
                  ((torch.zeros((), dtype=torch.bfloat16), w, w), {})):
        with pytest.raises(ValueError):
            qkr.gated_feed_forward(*a, **kw)
    f8 = torch.float8_e4m3fn
    s = dict(x_scale=one, gate_scale=torch.ones(32), up_scale=torch.ones(32))
    for bad in (dict(x_scale=None), dict(gate_scale=one), dict(up_scale=torch.ones(32).half()), dict(out_dtype=torch.float32)):
        with pytest.raises(ValueError):
            qkr.gated_feed_forward(x.to(f8), w.to(f8), w.to(f8), **dict(s, **bad))
    for bad in (dict(dh=h[:2]), dict(gate=h.half()), dict(up=x), dict(dx=h), dict(dw_gate=h), dict(dw_up=w.half()),
                dict(dx=x, input_grad=False), dict(dw_up=w, weight_grads=False), dict(activation="gelu")):
        t = dict(dict(dh=h, gate=h, up=h), **bad)
        with pytest.raises(ValueError):
            qkr.gated_feed_forward_backward(t.pop("dh"), x, w, w, t.pop("gate"), t.pop("up"), **t)
    with pytest.raises(ValueError, match="backward"):
        qkr.gated_feed_forward_backward(h, x.to(f8), w.to(f8), w.to(f8), h, h)


C_PROGRAM = r"""
#include <stdio.h>
#include "feed_forward.h"
#include "rms_norm.h"
int main(void)
{
    dit_ff_args a = {16, 64, 128, DIT_FF_SILU, QKR_BF16, QKR_BF16};
    if (dit_gated_feed_forward_backward_workspace_size(&a) < 4 * 16 * 128) return 1;
    if (dit_gated_feed_forward(&a, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != QKR_ERR_NULL) return 2;
    a.dtype = DIT_FF_E4M3;
    if (dit_gated_feed_forward_backward(&a, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != QKR_ERR_UNSUPPORTED) return 3;
    a.activation = DIT_FF_GELU_TANH, a.rows = 0;
    if (dit_gated_feed_forward(&a, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != QKR_OK) return 4;
    if (dit_rms_norm(0, 0, 0, 0, 0, 0, DIT_RMS_MAX_HIDDEN, 0, QKR_FP32, 1e-6f, QKR_FP16, 0) != QKR_OK) return 5;
    if (dit_rms_norm_backward(0, 0, 0, 0, 1, 64, 0, QKR_FP32, 0, 1e-6f, QKR_FP16, 0, 0, 0) != QKR_ERR_NULL) return 6;
    if (dit_rms_norm_backward_workspace_size(1, 60) != QKR_ERR_UNSUPPORTED) return 7;
    printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_c_program_builds_and_gets_the_documented_codes(tmp_path):
    lib_dir = os.path.dirname(qkr.LIB_PATH)
    src, exe = os.path.join(tmp_path, "check.c"), os.path.join(tmp_path, "check")
    with open(src, "w") as f:
        f.write(C_PROGRAM)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), src, "-L",
                    lib_dir, "-lqknorm_rope", "-ldit_attention", "-Wl,-rpath," + lib_dir, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", (out.returncode, out.stdout, out.stderr)
