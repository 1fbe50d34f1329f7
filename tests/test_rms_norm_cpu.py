"""RMS norm's entry points without a GPU: refusals, workspace sizes and what is
rejected by the binding.  Nothing here reaches a HIP call.
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from diffusion_transformer_qk_amd import binding as b

A = 1 << 20
FAR = 1 << 32


def forward(**over):
    v = dict(x=A, residual=A + FAR, sum=A + 2 * FAR, y=A + 3 * FAR, scales=0, rows=100, hidden=512,
             weight=A + 4 * FAR, param=b.QKR_FP32, eps=1e-6, dtype=b.QKR_BF16)
    v.update(over)
    return b.load_library().dit_rms_norm(v["x"], v["residual"], v["sum"], v["y"], v["scales"], v["rows"],
                                         v["hidden"], v["weight"], v["param"], v["eps"], v["dtype"], 0)


def backward(**over):
    v = dict(dy=A, x=A + FAR, dsum=A + 2 * FAR, dx=A + 3 * FAR, rows=100, hidden=512, weight=A + 4 * FAR,
             param=b.QKR_FP32, dw=A + 5 * FAR, eps=1e-6, dtype=b.QKR_BF16, ws=A + 6 * FAR, ws_bytes=1 << 40)
    v.update(over)
    return b.load_library().dit_rms_norm_backward(
        v["dy"], v["x"], v["dsum"], v["dx"], v["rows"], v["hidden"], v["weight"], v["param"], v["dw"], v["eps"],
        v["dtype"], v["ws"], v["ws_bytes"], 0)


@pytest.mark.parametrize("over,code", [
    (dict(hidden=0), b.QKR_ERR_UNSUPPORTED), (dict(hidden=12), b.QKR_ERR_UNSUPPORTED),
    (dict(hidden=8200), b.QKR_ERR_UNSUPPORTED), (dict(hidden=-8), b.QKR_ERR_UNSUPPORTED),
    (dict(dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED), (dict(dtype=5), b.QKR_ERR_ARG), (dict(param=-1), b.QKR_ERR_ARG),
    (dict(param=3), b.QKR_ERR_ARG), (dict(eps=0.0), b.QKR_ERR_ARG), (dict(eps=float("nan")), b.QKR_ERR_ARG),
    (dict(eps=float("inf")), b.QKR_ERR_ARG), (dict(rows=-1), b.QKR_ERR_SHAPE), (dict(rows=1 << 24), b.QKR_ERR_SHAPE),
    (dict(x=0), b.QKR_ERR_NULL), (dict(x=A + 8), b.QKR_ERR_ALIGN), (dict(weight=A + 4 * FAR + 4), b.QKR_ERR_ALIGN),
    (dict(rows=0, x=0), b.QKR_OK),
])
def test_both_directions(over, code):
    assert forward(**over) == code
    assert backward(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(y=0), b.QKR_ERR_NULL), (dict(sum=0), b.QKR_ERR_NULL), (dict(residual=0), b.QKR_ERR_NULL),
    (dict(y=A + 3 * FAR + 8), b.QKR_ERR_ALIGN), (dict(scales=A + 5 * FAR + 2), b.QKR_ERR_ALIGN),
    (dict(residual=A + FAR + 8), b.QKR_ERR_ALIGN), (dict(sum=A + 2 * FAR + 8), b.QKR_ERR_ALIGN),
    # partly over another buffer, or two outputs in one
    (dict(y=A + 16), b.QKR_ERR_ARG), (dict(y=A + FAR + 16), b.QKR_ERR_ARG), (dict(sum=A + 16), b.QKR_ERR_ARG),
    (dict(y=A + 2 * FAR), b.QKR_ERR_ARG), (dict(weight=A + 2 * FAR), b.QKR_ERR_ARG),
    (dict(weight=A + 3 * FAR + 100 * 1024 - 16), b.QKR_ERR_ARG),
    # 8 bits are never in place
    (dict(y=A, scales=A + 5 * FAR), b.QKR_ERR_ARG), (dict(y=A + FAR, scales=A + 5 * FAR), b.QKR_ERR_ARG),
    (dict(scales=A), b.QKR_ERR_ARG), (dict(scales=A + 3 * FAR), b.QKR_ERR_ARG), (dict(scales=A + 2 * FAR), b.QKR_ERR_ARG),
    (dict(scales=A + 4 * FAR), b.QKR_ERR_ARG), (dict(scales=A + FAR + 4), b.QKR_ERR_ARG)])
def test_forward(over, code):
    assert forward(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dy=0), b.QKR_ERR_NULL), (dict(dx=0), b.QKR_ERR_NULL), (dict(dsum=A + 2 * FAR + 8), b.QKR_ERR_ALIGN),
    (dict(dw=A + 5 * FAR + 4), b.QKR_ERR_ALIGN), (dict(ws=0), b.QKR_ERR_WORKSPACE),
    (dict(ws_bytes=100), b.QKR_ERR_WORKSPACE), (dict(ws=A + 6 * FAR + 8), b.QKR_ERR_ALIGN),
    (dict(dx=A + 16), b.QKR_ERR_ARG), (dict(dx=A + FAR), b.QKR_ERR_ARG), (dict(dx=A + 2 * FAR + 16), b.QKR_ERR_ARG),
    (dict(dw=A + 4 * FAR), b.QKR_ERR_ARG), (dict(dw=A + 3 * FAR), b.QKR_ERR_ARG), (dict(dw=A), b.QKR_ERR_ARG),
    (dict(ws=A + 5 * FAR), b.QKR_ERR_ARG), (dict(ws=A), b.QKR_ERR_ARG), (dict(ws=A + 2 * FAR), b.QKR_ERR_ARG)])
def test_backward(over, code):
    assert backward(**over) == code


def test_workspaces():
    size = qkr.rms_norm_backward_workspace_size
    assert size(1, 512) == 0 and size(4, 512) == 0            # one workgroup: it writes the sums itself
    assert size(0, 512) == 0 and size(-1, 512) == b.QKR_ERR_SHAPE and size(10, 12) == b.QKR_ERR_UNSUPPORTED
    for rows, hidden in ((100, 512), (32760, 5120), (5, 8192), ((1 << 24) - 1, 64)):
        n = size(rows, hidden)
        assert n % (hidden * 4) == 0 and 0 < n <= 1024 * hidden * 4


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        qkr.rms_norm(x, w)
    for f in (qkr.rms_norm, qkr.rms_norm_fp8):
        for kw in (dict(weight=w[:8]), dict(weight=w[None]), dict(residual=x[:2]), dict(residual=x.half()),
                   dict(sum_out=x), dict(residual=x, sum_out=x[:1]), dict(out=x.half()), dict(out=x[:3]),
                   dict(weight=w.double())):
            with pytest.raises(ValueError):
                f(x, **kw)
        with pytest.raises(ValueError):
            f(x.float(), w)
        with pytest.raises(ValueError, match="hidden"):
            f(torch.zeros((), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="scales"):
        qkr.rms_norm_fp8(x, w, scales=torch.zeros(3))
    for kw in (dict(weight=w[:8]), dict(dsum=x[:1]), dict(out=x.half())):
        with pytest.raises(ValueError):
            qkr.rms_norm_backward(x, x, **kw)
    with pytest.raises(ValueError, match="dy"):
        qkr.rms_norm_backward(x[:1], x, w)
