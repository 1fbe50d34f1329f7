"""The gated feed-forward projection and its backward pass on the GPU against
64 bits, element by element.

Bounds, with u half a step of the output's type and f = 2^-24 of fp32: a sum of
K products in fp32 is off by at most (K + 16) f of the sum of their magnitudes;
act has a slope of at most 1.13 and is itself computed to 32 f (1 + |z|)
relative (the argument of its exponential is off by f |z|, the rest is under 16
operations; |z| counts to 90, where act ends at 0 or x).  dgate and dup are
rounded to the type before the products (u relative; in fp16 at least 2^-39 of
the largest of them, which is stored as 2^14 or more, absolute).

In 8 bits the matrix instruction aligns the eight products of each run of eight k
to the largest of them, and drops what lies below 2^-13 of its power of two
(beside a product of 2^8 one of 2^-5 is kept whole and one of 2^-6 lost, which
the test of that says): seven products of a run are off by less than 2^-13 of
the largest each, and the sums of the runs are fp32's.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests.gpu_common import same_bits
from tests.test_gpu_layer_norm import DEV, F, TYPES, gen, guarded, half_step, tail, untouched

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def tensors(seed, rows, hidden, inner, dtype, by=1.0):
    g = gen(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = TYPES[dtype]
    s = torch.exp((torch.rand((rows, 1), generator=g) * 2 - 1) * math.log(4.0)) * by
    return dict(x=(n(rows, hidden) * s).to(t).to(DEV), w_gate=(n(inner, hidden) / math.sqrt(hidden)).to(t).to(DEV),
                w_up=(n(inner, hidden) / math.sqrt(hidden)).to(t).to(DEV))


def in_8_bits(x):
    scale = x.float().abs().amax(1).clamp(min=1e-30) / 448
    return (x.float() / scale[:, None]).to(FP8), scale


def z_of(a, act):
    return a if act == "silu" else math.sqrt(8 / math.pi) * (a + 0.044715 * a ** 3)


def act_of(a, act):
    return a * torch.sigmoid(z_of(a, act))


def slope_of(a, act):
    a = a.clone().requires_grad_()
    return torch.autograd.grad(act_of(a, act).sum(), a)[0]


def act_error(a, act):
    return 32 * F * (1 + z_of(a, act).abs().clamp(max=90))


def dropped(x, w):
    """What the alignment of the 8-bit products may drop."""
    total = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[1], 8):
        top = torch.zeros_like(total)
        for i in range(k, k + 8):
            top = torch.maximum(top, x[:, i:i + 1].abs() * w[:, i].abs())
        total += top
    return 7 * 2.0 ** -13 * total


def exact(x, wg, wu, act, scales=None):
    """(h, gate, up) in 64 bits and what each may be off by before it is rounded."""
    x, wg, wu = (t.double() for t in (x, wg, wu))
    k = x.shape[1]
    gate, up = x @ wg.t(), x @ wu.t()
    e_g, e_u = (x.abs() @ wg.abs().t() * (k + 16) * F, x.abs() @ wu.abs().t() * (k + 16) * F)
    if scales is not None:
        e_g, e_u = e_g + dropped(x, wg), e_u + dropped(x, wu)
        xs, gs, us = (s.double() for s in scales)
        by_g, by_u = xs[:, None] * gs, xs[:, None] * us
        gate, up, e_g, e_u = gate * by_g, up * by_u, e_g * by_g + 4 * F * (gate * by_g).abs(), e_u * by_u + 4 * F * (
            up * by_u).abs()
    y = act_of(gate, act)
    e_y = 1.13 * e_g + act_error(gate, act) * y.abs()
    return (y * up, gate, up), (e_y * (up.abs() + e_u) + y.abs() * e_u + 2 * F * (y * up).abs(), e_g, e_u)


def check_forward(x, wg, wu, act, scales=None, out_dtype=None):
    want, off = exact(x, wg, wu, act, scales)
    shape = (x.shape[0], wg.shape[0])
    t = out_dtype or x.dtype
    bufs = [guarded(shape, t) for _ in range(3)]
    kw = dict(zip(("x_scale", "gate_scale", "up_scale"), scales)) if scales is not None else {}
    qkr.gated_feed_forward(x, wg, wu, activation=act, out_dtype=out_dtype, save=True, out=bufs[0][0],
                           gate=bufs[1][0], up=bufs[2][0], **kw)
    h = qkr.gated_feed_forward(x, wg, wu, activation=act, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    assert all(untouched(b) for _, b in bufs)
    for (got, _), w, e in zip(bufs, want, off):
        bound = half_step(got) * w.abs() + (1 + half_step(got)) * e + tail(got)
        assert bool(((got.double() - w).abs() <= bound).all())
    assert same_bits(h, bufs[0][0])


SIZES = [(1, 8, 8), (1, 5120, 136), (3, 64, 40), (17, 1000, 264), (31, 24, 520), (32, 32, 64), (33, 8, 8), (40, 40, 72),
         (77, 1000, 328), (128, 64, 64), (129, 96, 136), (255, 328, 1000), (300, 2056, 72), (1, 136, 5120)]


@pytest.mark.parametrize("rows,hidden,inner", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward(rows, hidden, inner, dtype):
    t = tensors(1, rows, hidden, inner, dtype)
    for act in ("silu", "gelu_tanh"):
        check_forward(t["x"], t["w_gate"], t["w_up"], act)


@pytest.mark.parametrize("rows,hidden,inner", [(-(-r // 1), 16 * -(-h // 16), 16 * -(-i // 16)) for r, h, i in SIZES])
def test_forward_in_8_bits(rows, hidden, inner):
    t = tensors(2, rows, hidden, inner, "fp32")
    (x, xs), (wg, gs), (wu, us) = (in_8_bits(t[n]) for n in ("x", "w_gate", "w_up"))
    check_forward(x, wg, wu, "silu", (xs, gs, us), torch.bfloat16)
    check_forward(x, wg, wu, "gelu_tanh", (xs, gs, us), torch.float16)


@pytest.mark.parametrize("rows,hidden,inner", [(4200, 96, 2056), (257, 200, 16392), (5000, 104, 1800)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_tiles(rows, hidden, inner, dtype):
    """Several rounds of tiles, at sizes that end inside one."""
    t = tensors(3, rows, hidden, inner, dtype)
    check_forward(t["x"], t["w_gate"], t["w_up"], "silu")
    t8 = tensors(4, rows, 16 * -(-hidden // 16), 16 * -(-inner // 16), "fp32")
    (x, xs), (wg, gs), (wu, us) = (in_8_bits(t8[n]) for n in ("x", "w_gate", "w_up"))
    check_forward(x, wg, wu, "silu", (xs, gs, us), TYPES[dtype])


def test_alignment_of_8_bit_products():
    """2^8 - 2^8 + small, all within eight k, and the small one in a run of its own."""
    rows, k = 20, 64
    x, w = torch.zeros((rows, k)), torch.zeros((16, k))
    x[:, 0], x[:, 1], w[:, :2] = 256, -256, 1
    w[:, 2] = w[:, 8] = 2.0 ** -6
    one = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    small = 2.0 ** (7 - torch.arange(rows))              # products of 2^7 .. 2^-12
    for place, kept in ((2, small >= 2.0 ** -5), (8, small > 0)):
        x[:, [2, 8]] = 0
        x[:, place] = small * 64
        fits = x[:, place] <= 256                        # that e4m3 has, from 2^-9 on
        fits &= x[:, place] >= 2.0 ** -9
        _, gate, _ = qkr.gated_feed_forward(x.clamp(max=256).to(FP8).to(DEV), w.to(FP8).to(DEV), w.to(FP8).to(DEV),
                                            x_scale=one(rows), gate_scale=one(16), up_scale=one(16), save=True)
        want = torch.where(kept, small, torch.zeros_like(small))
        assert bool((gate.cpu().float() == want[:, None])[fits].all())


def backward_inputs(seed, rows, hidden, inner, dtype, by=1.0):
    t = tensors(seed, rows, hidden, inner, dtype)
    g = gen(seed + 100)
    s = torch.exp((torch.rand((rows, 1), generator=g) * 2 - 1) * math.log(4.0)) / 16 * by
    t["dh"] = (torch.randn((rows, inner), generator=g) * s).to(TYPES[dtype]).to(DEV)
    for n in ("gate", "up"):
        t[n] = (t["x"].double() @ t["w_" + n].double().t()).to(TYPES[dtype])
    return t


def check_backward(t, act):
    x, wg, wu, dh, gate, up = (t[n].double() for n in ("x", "w_gate", "w_up", "dh", "gate", "up"))
    rows, inner = dh.shape
    y, slope = act_of(gate, act), slope_of(gate, act)
    da, db = dh * up * slope, dh * y
    u = half_step(t["x"])
    top = max(float(da.abs().max()), float(db.abs().max())) if rows else 0.0
    small = top * 2.0 ** -39 if t["x"].dtype == torch.float16 else 0.0
    # slope = s + y (1 - s) dz: its parts may cancel; |dz| |y| (1 - s) and s are below 3
    e = act_error(gate, act)
    e_a, e_b = u * da.abs() + (dh * up).abs() * 3 * e + small, (u + e) * db.abs() + small
    made = {}
    for n, like in (("dx", "x"), ("dw_gate", "w_gate"), ("dw_up", "w_up")):
        made[n], made[n + "_buf"] = guarded(t[like].shape, t[like].dtype)
    qkr.gated_feed_forward_backward(t["dh"], t["x"], t["w_gate"], t["w_up"], t["gate"], t["up"], activation=act,
                                    **{n: made[n] for n in ("dx", "dw_gate", "dw_up")})
    torch.cuda.synchronize()
    want = dict(dx=da @ wg + db @ wu, dw_gate=da.t() @ x, dw_up=db.t() @ x)
    off = dict(dx=e_a @ wg.abs() + e_b @ wu.abs() + (2 * inner + 16) * F * (da.abs() @ wg.abs() + db.abs() @ wu.abs()),
               dw_gate=e_a.t() @ x.abs() + (rows + 16) * F * (da.abs().t() @ x.abs()),
               dw_up=e_b.t() @ x.abs() + (rows + 16) * F * (db.abs().t() @ x.abs()))
    for n, w in want.items():
        assert untouched(made[n + "_buf"]), n
        bound = u * w.abs() + (1 + u) * off[n] + tail(t["x"])
        assert bool(((made[n].double() - w).abs() <= bound).all()), n
    return {n: made[n] for n in want}


# dx, dw, or both summed over splits of k, which end inside a stage or have none
SPLITS = [(5, 512, 2048), (2500, 64, 136), (40, 264, 3080), (1100, 72, 1544), (1, 8, 4104), (3000, 520, 40)]


@pytest.mark.parametrize("rows,hidden,inner", SIZES + SPLITS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_backward(rows, hidden, inner, dtype):
    for act in ("silu", "gelu_tanh"):
        t = backward_inputs(5, rows, hidden, inner, dtype)
        all_of = check_backward(t, act)
    a = [t[n] for n in ("dh", "x", "w_gate", "w_up", "gate", "up")]
    dx, dg, du = qkr.gated_feed_forward_backward(*a, activation=act, weight_grads=False)
    assert dg is None and du is None and same_bits(dx, all_of["dx"])
    dx, dg, du = qkr.gated_feed_forward_backward(*a, activation=act, input_grad=False)
    assert dx is None and same_bits(dg, all_of["dw_gate"]) and same_bits(du, all_of["dw_up"])


@pytest.mark.parametrize("rows,hidden,inner", [(4200, 4104, 72), (136, 2056, 4104), (4128, 264, 8200)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_tiles_backward(rows, hidden, inner, dtype):
    check_backward(backward_inputs(6, rows, hidden, inner, dtype), "silu")


@pytest.mark.parametrize("by", [2.0 ** -14, 1.0, 2.0 ** 10])
def test_small_and_large_gradients_in_fp16(by):
    check_backward(backward_inputs(7, 70, 136, 200, "fp16", by), "silu")


# These fill the chip once with 256 x 256 tiles and more than once with 128 x 128 ones, which
# is what the larger tiles are taken for.
@pytest.mark.parametrize("rows,hidden,inner", [(3900, 96, 1960), (300, 200, 16328), (520, 1040, 8008)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_round_of_large_tiles(rows, hidden, inner, dtype):
    for act in ("silu", "gelu_tanh"):
        t = tensors(9, rows, hidden, inner, dtype)
        check_forward(t["x"], t["w_gate"], t["w_up"], act)
        t8 = tensors(10, rows, 16 * -(-hidden // 16), 16 * (inner // 16), "fp32")
        (x, xs), (wg, gs), (wu, us) = (in_8_bits(t8[n]) for n in ("x", "w_gate", "w_up"))
        check_forward(x, wg, wu, act, (xs, gs, us), TYPES[dtype])


# dx; dw; dw over splits of the rows; dx over splits
@pytest.mark.parametrize("rows,hidden,inner", [(3900, 3920, 72), (136, 3920, 1960), (40000, 1480, 744),
                                               (1480, 1480, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_round_of_large_tiles_backward(rows, hidden, inner, dtype):
    check_backward(backward_inputs(11, rows, hidden, inner, dtype), "gelu_tanh")


def test_gradients_against_differences():
    rows, hidden, inner, h = 5, 16, 24, 1e-5
    for act in ("silu", "gelu_tanh"):
        t = backward_inputs(8, rows, hidden, inner, "fp16")
        got = qkr.gated_feed_forward_backward(*(t[n] for n in ("dh", "x", "w_gate", "w_up", "gate", "up")), activation=act)

        def loss(x, wg, wu):
            return float((act_of(x @ wg.t(), act) * (x @ wu.t()) * t["dh"].double()).sum())

        at = [t[n].double() for n in ("x", "w_gate", "w_up")]
        for k, g in enumerate(got):
            size = float(g.double().norm()) / math.sqrt(g.numel())
            for i, j in ((0, 0), (2, 7), (4, 15), (rows - 1 if k == 0 else inner - 1, hidden - 1)):
                e = [torch.zeros_like(a) for a in at]
                e[k][i, j] = h
                d = (loss(*(a + b for a, b in zip(at, e))) - loss(*(a - b for a, b in zip(at, e)))) / (2 * h)
                # kept projections and gradients are rounded to 11 bits, and sums of some 24 of them
                assert abs(float(g[i, j]) - d) <= 2.0 ** -7 * (abs(d) + size)


@pytest.mark.parametrize("rows", [5, 70, 300])
def test_infinities_and_nan_stay_in_their_rows(rows):
    t = backward_inputs(9, rows, 72, 136, "bf16")
    a = [t[n] for n in ("dh", "x", "w_gate", "w_up", "gate", "up")]
    h = qkr.gated_feed_forward(t["x"], t["w_gate"], t["w_up"])
    dx, _, _ = qkr.gated_feed_forward_backward(*a)
    bad = {n: v.clone() for n, v in t.items()}
    bad["x"][2, 5] = math.inf
    bad["x"][3, 71] = math.nan
    bad["dh"][1, 100] = math.nan
    keep = [i for i in range(rows) if i not in (1, 2, 3)]
    got = qkr.gated_feed_forward(bad["x"], t["w_gate"], t["w_up"])
    assert same_bits(got[keep], h[keep]) and bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got[2]).any())
    got, dwg, _ = qkr.gated_feed_forward_backward(*(bad[n] for n in ("dh", "x", "w_gate", "w_up", "gate", "up")))
    assert same_bits(got[keep], dx[keep]) and bool(torch.isnan(got[1]).all())
    assert bool(torch.isnan(dwg[:, 71]).all()) and bool(torch.isnan(dwg[100]).all())
    # in fp16 a row that is lost does not unscale the others
    t = backward_inputs(10, rows, 72, 136, "fp16", 2.0 ** -12)
    a = [t[n] for n in ("dh", "x", "w_gate", "w_up", "gate", "up")]
    dx, _, _ = qkr.gated_feed_forward_backward(*a)
    a[0] = t["dh"].clone()
    a[0][1, 3] = math.inf
    # (the largest finite value may have been the lost row's: the power of two, but no row's bits, may differ)
    got, _, _ = qkr.gated_feed_forward_backward(*a)
    keep = [i for i in range(rows) if i != 1]
    assert float((got[keep].double() - dx[keep].double()).abs().max()) <= 2.0 ** -9 * float(dx[keep].double().abs().max())


@pytest.mark.parametrize("value", [-3e38, -1e20, -100.0, -89.0, 89.0, 1e20, 3e38])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_projections_far_from_zero(value, act):
    """The activation ends at 0 or x, its slope at 0 or 1, up to bf16's largest numbers."""
    one = torch.zeros((40, 8), dtype=torch.bfloat16, device=DEV)
    one[:, 0] = 1
    wg, wu = torch.zeros((16, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((16, 8), dtype=torch.bfloat16, device=DEV)
    wg[:, 0] = value
    wu[:, 0] = 0.5
    h, gate, up = qkr.gated_feed_forward(one, wg, wu, activation=act, save=True)
    v = float(wg[0, 0])
    assert bool((gate.double() == v).all())
    assert bool(((h.double() - (0.5 * v if v > 0 else 0)).abs() <= 2.0 ** -8 * max(0, v) + 1e-30).all())
    dh = torch.ones_like(h) * 2.0 ** -6
    dx, dg, _ = qkr.gated_feed_forward_backward(dh, one, wg, wu, gate, up, activation=act, input_grad=True)
    assert bool((dg[:, 0].double() == (40 * 2.0 ** -7 if v > 0 else 0)).all())


def test_halves_of_one_weight_and_leading_dimensions():
    t = tensors(11, 6 * 7, 64, 48, "bf16")
    both = torch.cat([t["w_gate"], t["w_up"]])
    wg, wu = both.chunk(2)
    x = t["x"].view(6, 7, 64)
    h, gate, up = qkr.gated_feed_forward(x, wg, wu, save=True)
    assert h.shape == (6, 7, 48)
    assert same_bits(h.view(42, 48), qkr.gated_feed_forward(t["x"], t["w_gate"], t["w_up"]))
    grads = torch.empty_like(both)
    dg, du = grads.chunk(2)
    dx, a, b = qkr.gated_feed_forward_backward(h, x, wg, wu, gate, up, dw_gate=dg, dw_up=du)
    want = qkr.gated_feed_forward_backward(h, x, t["w_gate"], t["w_up"], gate, up)
    assert dx.shape == x.shape and same_bits(grads, torch.cat(want[1:])) and a is dg and b is du
    # shared: both projections by one weight
    same = qkr.gated_feed_forward(t["x"], t["w_up"], t["w_up"])
    assert same.shape == (42, 48)


def test_no_rows():
    t = tensors(12, 0, 64, 48, "fp16")
    h, gate, up = qkr.gated_feed_forward(t["x"], t["w_gate"], t["w_up"], save=True)
    assert h.shape == gate.shape == up.shape == (0, 48)
    dx, dg, du = qkr.gated_feed_forward_backward(h, t["x"], t["w_gate"], t["w_up"], gate, up)
    assert dx.shape == (0, 64) and bool((dg == 0).all()) and bool((du == 0).all())


@pytest.mark.parametrize("rows", [4, 200])
def test_streams_and_graphs(rows):
    s = backward_inputs(13, rows, 136, 200, "fp16")
    names = ("dh", "x", "w_gate", "w_up", "gate", "up")

    def step():
        h, gate, up = qkr.gated_feed_forward(s["x"], s["w_gate"], s["w_up"], save=True)
        return [h, gate, up, *qkr.gated_feed_forward_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], gate, up)]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        h, gate, up = qkr.gated_feed_forward(s["x"], s["w_gate"], s["w_up"], save=True, stream=stream)
        got = qkr.gated_feed_forward_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], gate, up, stream=stream)
        side.synchronize()
        assert all(same_bits(a, b) for a, b in zip((h, gate, up, *got), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        new = backward_inputs(20 + i, rows, 136, 200, "fp16")
        for n in names:
            s[n].copy_(new[n])
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(kept, want))
