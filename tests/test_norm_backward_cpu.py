"""Layer norm and the backward entry points without a GPU: refusals, workspace
sizes and what is rejected by the binding.  Nothing here reaches a HIP call.
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from diffusion_transformer_qk_amd import binding as b

A = 1 << 20
FAR = 1 << 32


def ln(**over):
    v = dict(x=A, y=A + FAR, rows=100, hidden=512, weight=A + 2 * FAR, bias=A + 3 * FAR, param=b.QKR_FP32,
             eps=1e-6, dtype=b.QKR_BF16)
    v.update(over)
    return b.load_library().dit_layer_norm(v["x"], v["y"], v["rows"], v["hidden"], v["weight"], v["bias"],
                                           v["param"], v["eps"], v["dtype"], 0)


def ln_back(**over):
    v = dict(dy=A, x=A + FAR, dx=A + 2 * FAR, rows=100, hidden=512, per=100, weight=A + 3 * FAR, form=0,
             param=b.QKR_FP32, dw=A + 4 * FAR, db=A + 5 * FAR, eps=1e-6, dtype=b.QKR_BF16, ws=A + 6 * FAR,
             ws_bytes=1 << 40)
    v.update(over)
    return b.load_library().dit_layer_norm_backward(
        v["dy"], v["x"], v["dx"], v["rows"], v["hidden"], v["per"], v["weight"], v["form"], v["param"], v["dw"],
        v["db"], v["eps"], v["dtype"], v["ws"], v["ws_bytes"], 0)


COMMON = [
    (dict(hidden=0), b.QKR_ERR_UNSUPPORTED), (dict(hidden=12), b.QKR_ERR_UNSUPPORTED),
    (dict(hidden=8200), b.QKR_ERR_UNSUPPORTED), (dict(dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED),
    (dict(dtype=5), b.QKR_ERR_ARG), (dict(param=-1), b.QKR_ERR_ARG), (dict(eps=0.0), b.QKR_ERR_ARG),
    (dict(eps=float("nan")), b.QKR_ERR_ARG), (dict(rows=-1), b.QKR_ERR_SHAPE), (dict(rows=1 << 24), b.QKR_ERR_SHAPE),
    (dict(x=0), b.QKR_ERR_NULL), (dict(x=A + 8), b.QKR_ERR_ALIGN), (dict(weight=A + 3 * FAR + 4), b.QKR_ERR_ALIGN),
    (dict(rows=0, x=0), b.QKR_OK),
]


@pytest.mark.parametrize("over,code", COMMON)
def test_both_directions(over, code):
    assert ln(**over) == code
    assert ln_back(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(y=0), b.QKR_ERR_NULL), (dict(y=A + 16), b.QKR_ERR_ARG), (dict(weight=A + FAR), b.QKR_ERR_ARG),
    (dict(bias=A + FAR + 100 * 1024 - 16), b.QKR_ERR_ARG), (dict(bias=A + 4), b.QKR_ERR_ALIGN)])
def test_forward(over, code):
    assert ln(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(per=0), b.QKR_ERR_SHAPE), (dict(form=2), b.QKR_ERR_ARG), (dict(dy=0), b.QKR_ERR_NULL),
    (dict(dx=0), b.QKR_ERR_NULL), (dict(dw=0), b.QKR_ERR_NULL), (dict(db=0), b.QKR_ERR_NULL),
    (dict(ws=0), b.QKR_ERR_WORKSPACE), (dict(ws_bytes=100), b.QKR_ERR_WORKSPACE), (dict(ws=A + 6 * FAR + 8), b.QKR_ERR_ALIGN),
    (dict(dx=A + 16), b.QKR_ERR_ARG), (dict(dx=A + FAR), b.QKR_ERR_ARG), (dict(dw=A + 3 * FAR), b.QKR_ERR_ARG),
    (dict(db=A + 4 * FAR), b.QKR_ERR_ARG), (dict(dw=A + 2 * FAR), b.QKR_ERR_ARG), (dict(ws=A + 5 * FAR), b.QKR_ERR_ARG),
    (dict(ws=A), b.QKR_ERR_ARG)])
def test_backward(over, code):
    assert ln_back(**over) == code


def test_norm_workspaces():
    size = qkr.layer_norm_backward_workspace_size
    assert size(1, 512) == 0                                  # one workgroup: it writes the sums itself
    assert size(0, 512) == 0 and size(-1, 512) == b.QKR_ERR_SHAPE and size(10, 12) == b.QKR_ERR_UNSUPPORTED
    assert size(4000, 512, 4) == 0                            # a workgroup a batch
    for rows, hidden in ((100, 512), (32760, 5120), (5, 8192)):
        n = size(rows, hidden)
        assert n % (2 * hidden * 4) == 0 and 0 < n <= 1024 * 2 * hidden * 4


def test_one_weight_row_for_any_number_of_rows():
    """rows_per_batch may be far above the rows, up to the largest number."""
    size = qkr.layer_norm_backward_workspace_size
    for rows, hidden in ((100, 512), (32760, 5120), ((1 << 24) - 1, 64)):
        for per in (rows, rows + 1, 1 << 40, (1 << 63) - 1):
            assert size(rows, hidden, per) == size(rows, hidden)
    assert ln_back(per=(1 << 63) - 1, ws=0) == b.QKR_ERR_WORKSPACE
    assert ln_back(per=(1 << 63) - 1, ws_bytes=size(100, 512) - 1) == b.QKR_ERR_WORKSPACE
    assert ln_back(per=(1 << 63) - 1, dw=A + 2 * FAR) == b.QKR_ERR_ARG


def qk(**over):
    v = dict(qkv=(A, A + FAR, A + 2 * FAR), q=None, k=None, tokens=100, heads=4, head_dim=64, qg=A + 3 * FAR,
             kg=A + 3 * FAR + 4096, dqg=A + 4 * FAR, dkg=A + 4 * FAR + 4096, eps=1e-6, cos=A + 5 * FAR,
             sin=A + 6 * FAR, layout=0, table=b.QKR_FP32, style=0, dtype=b.QKR_BF16, ws=A + 7 * FAR, ws_bytes=1 << 40)
    v.update(over)
    t = [None if v[n] is None else b.GradTensor(*v[n]) for n in ("qkv", "q", "k")]
    return b.load_library().qknorm_rope_backward(
        *t, v["tokens"], v["heads"], v["head_dim"], v["qg"], v["kg"], v["dqg"], v["dkg"], v["eps"], v["cos"],
        v["sin"], v["layout"], v["table"], v["style"], v["dtype"], v["ws"], v["ws_bytes"], 0)


Q, K = (A, A + FAR, A + 2 * FAR), (A + 8 * FAR, A + 9 * FAR, A + 10 * FAR)


@pytest.mark.parametrize("over,code", [
    (dict(head_dim=96), b.QKR_ERR_UNSUPPORTED), (dict(dtype=b.QKR_FP32), b.QKR_ERR_UNSUPPORTED),
    (dict(table=b.QKR_FP16), b.QKR_ERR_UNSUPPORTED), (dict(dtype=9), b.QKR_ERR_ARG), (dict(table=-1), b.QKR_ERR_ARG),
    (dict(layout=2), b.QKR_ERR_ARG), (dict(style=2), b.QKR_ERR_ARG), (dict(eps=-1.0), b.QKR_ERR_ARG),
    (dict(tokens=-1), b.QKR_ERR_SHAPE), (dict(tokens=1 << 24), b.QKR_ERR_SHAPE), (dict(heads=0), b.QKR_ERR_SHAPE),
    (dict(heads=65537), b.QKR_ERR_SHAPE), (dict(q=Q), b.QKR_ERR_MODE), (dict(qkv=None), b.QKR_ERR_MODE),
    (dict(qg=0), b.QKR_ERR_NULL), (dict(dkg=0), b.QKR_ERR_NULL), (dict(cos=0), b.QKR_ERR_NULL),
    (dict(qkv=(0, A, A)), b.QKR_ERR_NULL), (dict(qkv=None, q=(A, 0, A)), b.QKR_ERR_NULL),
    (dict(ws=0), b.QKR_ERR_WORKSPACE), (dict(ws_bytes=64), b.QKR_ERR_WORKSPACE),
    (dict(qkv=(A + 8, A + FAR, A + 2 * FAR)), b.QKR_ERR_ALIGN), (dict(sin=A + 6 * FAR + 4), b.QKR_ERR_ALIGN),
    (dict(dqg=A + 4 * FAR + 8), b.QKR_ERR_ALIGN), (dict(ws=A + 7 * FAR + 8), b.QKR_ERR_ALIGN),
    (dict(qkv=(A, A + FAR, A + 16)), b.QKR_ERR_ARG), (dict(qkv=(A, A + FAR, A + FAR)), b.QKR_ERR_ARG),
    (dict(qkv=(A, A + FAR, A + 5 * FAR)), b.QKR_ERR_ARG), (dict(dkg=A + 4 * FAR), b.QKR_ERR_ARG),
    (dict(dqg=A), b.QKR_ERR_ARG), (dict(ws=A + FAR), b.QKR_ERR_ARG), (dict(ws=A + 4 * FAR), b.QKR_ERR_ARG),
    (dict(qkv=None, q=Q, k=(K[0], K[1], Q[0])), b.QKR_ERR_ARG), (dict(qkv=None, q=Q, k=(K[0], K[1], Q[2])), b.QKR_ERR_ARG),
    (dict(qkv=None, q=Q, k=(Q[2], K[1], K[2])), b.QKR_ERR_ARG),
])
def test_qk_backward(over, code):
    assert qk(**over) == code


def test_qk_workspace():
    size = qkr.qknorm_rope_backward_workspace_size
    assert size(0, 64) == 0 and size(1, 64) == 2 * 64 * 4 and size(1 << 20, 128) == 2048 * 2 * 128 * 4
    assert size(-1, 64) == b.QKR_ERR_SHAPE and size(5, 100) == b.QKR_ERR_UNSUPPORTED


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros((10, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        qkr.layer_norm(x, w)
    for call in (lambda: qkr.layer_norm(x, w[:32]), lambda: qkr.layer_norm(x, w, w.half()),
                 lambda: qkr.layer_norm(x, w, out=x[:5]), lambda: qkr.layer_norm(x.float(), w),
                 lambda: qkr.layer_norm(x, w.double()),
                 lambda: qkr.layer_norm_backward(x[:5], x, w), lambda: qkr.layer_norm_backward(x.half(), x, w),
                 lambda: qkr.layer_norm_backward(x, x, w[:8]), lambda: qkr.layer_norm_backward(x, x, w, out=x.half()),
                 lambda: qkr.fuse_scale_shift_backward(x, x, w.view(1, 64)[:, :8]),
                 lambda: qkr.fuse_scale_shift_backward(x, x, torch.ones(3, 64)),
                 lambda: qkr.fuse_scale_shift_backward(x, x, torch.ones(3, 64), rows_per_batch=2)):
        with pytest.raises(ValueError):
            call()
    qkv = torch.zeros((10, 3 * 2 * 64), dtype=torch.bfloat16)
    q = torch.zeros((10, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((10, 64))
    ok = dict(q_gamma=w, k_gamma=w, cos=t, sin=t)
    for pos, kw in (((qkv,), ok), ((qkv, qkv, q), ok), ((None, qkv), ok), ((None, None, q), ok),
                    ((), dict(ok, dq=q, k=q)), ((qkv, qkv), dict(ok, cos=t[:5])), ((qkv, qkv), dict(ok, cos=None)),
                    ((qkv, qkv), dict(ok, style="x")), ((qkv, qkv), dict(ok, cos_layout="x")),
                    ((qkv, qkv), dict(ok, q_gamma=w.half())), ((qkv[:5], qkv), ok), ((qkv.half(), qkv), ok),
                    ((qkv, qkv), dict(cos=t, sin=t)), ((qkv, qkv), dict(ok, out=qkv[:, :64])),
                    ((), dict(ok, dq=q, q=q, dk=q[:5], k=q[:5]))):
        with pytest.raises(ValueError):
            qkr.qknorm_rope_backward(*pos, **kw)
