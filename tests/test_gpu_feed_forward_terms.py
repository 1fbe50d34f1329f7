"""The feed-forward backward pass of few rows, and of few numbers, on the GPU: dgate
and dup go into their products in two 16-bit terms, so that gradients are off by
their own rounding, against 64 bits.

Bounds: those of test_gpu_feed_forward.py with u^2 in the place of u for dgate and
dup (the remainder of their rounding is rounded too); in fp16 the remainder of the
smallest numbers ends at 2^-39 of the largest, as the numbers themselves do.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests.gpu_common import same_bits
from tests.test_gpu_feed_forward import act_error, act_of, backward_inputs, slope_of
from tests.test_gpu_layer_norm import F, TYPES, guarded, half_step, tail, untouched

pytestmark = pytest.mark.gpu


def bounds(t, act, u_d):
    """{name: (value, bound)} where dgate and dup are rounded by u_d."""
    x, wg, wu, dh, gate, up = (t[n].double() for n in ("x", "w_gate", "w_up", "dh", "gate", "up"))
    rows, inner = dh.shape
    y, slope = act_of(gate, act), slope_of(gate, act)
    da, db = dh * up * slope, dh * y
    u = half_step(t["x"])
    top = max(float(da.abs().max()), float(db.abs().max()))
    small = top * 2.0 ** -39 if t["x"].dtype == torch.float16 else 0.0
    e = act_error(gate, act)
    e_a = u_d * da.abs() + (dh * up).abs() * 3 * e + small + 2.0 ** -126
    e_b = (u_d + e) * db.abs() + small + 2.0 ** -126
    want = dict(dx=da @ wg + db @ wu, dw_gate=da.t() @ x, dw_up=db.t() @ x)
    # twice as many products in a sum, the second half of them below u of the first
    off = dict(dx=e_a @ wg.abs() + e_b @ wu.abs() + (4 * inner + 80) * F * (da.abs() @ wg.abs() + db.abs() @ wu.abs()),
               dw_gate=e_a.t() @ x.abs() + (2 * rows + 16) * F * (da.abs().t() @ x.abs()),
               dw_up=e_b.t() @ x.abs() + (2 * rows + 16) * F * (db.abs().t() @ x.abs()))
    return {n: (w, u * w.abs() + (1 + u) * off[n] + tail(t["x"])) for n, w in want.items()}


def grads(t, act, **kw):
    return qkr.gated_feed_forward_backward(*(t[n] for n in ("dh", "x", "w_gate", "w_up", "gate", "up")), activation=act,
                                           **kw)


# few rows of any width; few numbers of any shape, at the ends of what counts as that
SIZES = [(1, 8, 8), (1, 5120, 136), (2, 1168, 56), (3, 56, 1160), (5, 512, 2048), (17, 1000, 264), (31, 24, 520),
         (32, 32, 64), (32, 2056, 4104), (1, 8, 4104), (33, 8, 992), (42, 792, 200), (70, 496, 192), (128, 8192, 256),
         (255, 328, 128), (570, 80, 56), (4096, 256, 8)]


@pytest.mark.parametrize("rows,hidden,inner", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_two_terms(rows, hidden, inner, dtype, act):
    t = backward_inputs(71, rows, hidden, inner, dtype)
    made = {n: guarded(t[like].shape, t[like].dtype) for n, like in (("dx", "x"), ("dw_gate", "w_gate"), ("dw_up", "w_up"))}
    need = qkr.gated_feed_forward_backward_workspace_size(rows, hidden, inner, dtype=dict(bf16=0, fp16=1)[dtype])
    workspace, around = guarded((need // 2,), TYPES[dtype])
    grads(t, act, workspace=workspace, **{n: b[0] for n, b in made.items()})
    torch.cuda.synchronize()
    assert untouched(around)
    for n, (want, bound) in bounds(t, act, half_step(t["x"]) ** 2).items():
        assert untouched(made[n][1]), n
        assert bool(((made[n][0].double() - want).abs() <= bound).all()), n
    # each gradient alone
    dx, _, _ = grads(t, act, weight_grads=False)
    _, dg, du = grads(t, act, input_grad=False)
    assert all(same_bits(a, made[n][0]) for n, a in (("dx", dx), ("dw_gate", dg), ("dw_up", du)))


def test_the_bounds_tell_the_terms_apart():
    """One term does not meet them (by the oracle, on the CPU)."""
    t = {n: v.cpu() for n, v in backward_inputs(72, 16, 264, 520, "bf16").items()}
    dh, gate, up, wg, wu = (t[n].double() for n in ("dh", "gate", "up", "w_gate", "w_up"))
    da, db = dh * up * slope_of(gate, "silu"), dh * act_of(gate, "silu")
    want, bound = bounds(t, "silu", half_step(t["x"]) ** 2)["dx"]
    one = [d.to(torch.bfloat16).double() for d in (da, db)]
    two = [o + (d - o).to(torch.bfloat16).double() for o, d in zip(one, (da, db))]
    for (a, b), fits in ((one, False), (two, True)):
        got = (a @ wg + b @ wu).to(torch.bfloat16).double()
        assert bool(((got - want).abs() <= bound).all()) == fits


def test_infinities_stay_in_their_rows():
    for dtype in ("bf16", "fp16"):
        t = backward_inputs(73, 9, 72, 136, dtype)
        dx, _, _ = grads(t, "silu")
        t["dh"][4, 7] = math.inf
        got, _, _ = grads(t, "silu")
        keep = [i for i in range(9) if i != 4]
        assert bool(torch.isfinite(got[keep]).all()) and not bool(torch.isfinite(got[4]).any())
        off = (got[keep].double() - dx[keep].double()).abs()
        assert bool((off <= 2 * half_step(dx) * dx[keep].double().abs() + 2 * tail(dx)).all())
