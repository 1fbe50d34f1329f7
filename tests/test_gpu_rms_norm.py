"""RMS norm with the residual's addition and an output in 8 bits, and its
backward pass, on the GPU against 64 bits.

Bounds, with u half a step of the 16-bit type and c = 64 * 2^-24: a row's sums
are trees of at most 44 fp32 operations one after another (16 to 32 products a
thread, 6 lane moves, 4 waves), the rest of a value's path is under 12, so n = s
rstd is off by c |n|; the other bounds carry that through the formulas.
dweight: at most 200 additions one after another for the rows here (the rows of
a chunk, then its chunks in 32 runs).  The values in 8 bits do not depend on
any sum and are exact products and quotients of fp32: they have to be equal.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests.gpu_common import same_bits
from tests.test_gpu_layer_norm import DEV, EPS, F, TYPES, C, gen, guarded, half_step, rows_of, tail, untouched

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def weight_of(seed, hidden, dtype):
    if dtype is None:
        return None
    return (1 + 0.3 * torch.randn(hidden, generator=gen(seed))).to(TYPES[dtype]).to(DEV)


def summed(x, residual):
    """Rounded once: both have so few bits that the sum in 64 bits is exact."""
    return x if residual is None else (x.double() + residual.double()).to(x.dtype)


def normalised(s, eps=EPS):
    s = s.double()
    rstd = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return s * rstd, rstd


def in_8_bits(s, w):
    """The bytes, by the formula in fp32 on the CPU, of rows times a power of two
    that brings their largest value below 1: it changes no mantissa, and keeps
    448 / top of the smallest rows in fp32's range."""
    s = s.double().cpu()
    s = torch.ldexp(s, -torch.frexp(s.abs().amax(-1, keepdim=True)).exponent)
    t = s.float() * (1.0 if w is None else w.float().cpu())
    top = t.abs().amax(-1, keepdim=True)
    # (a number over a tensor would be its reciprocal times the number: two roundings)
    return (t * (torch.full_like(top, 448.0) / torch.where(top == 0, torch.ones_like(top), top))).to(FP8)


def check_forward(x, residual, w, eps=EPS):
    s = summed(x, residual)
    n, _ = normalised(s, eps)
    want = n * (1.0 if w is None else w.double())
    y, buf = guarded(x.shape, x.dtype)
    sums, sbuf = guarded(x.shape, x.dtype)
    qkr.rms_norm(x, w, residual=residual, sum_out=None if residual is None else sums, out=y, eps=eps)
    torch.cuda.synchronize()
    assert untouched(buf) and untouched(sbuf)
    if residual is not None:
        assert same_bits(sums, s)
    bound = half_step(x) * want.abs() + 2 * C * want.abs() + tail(x)
    assert bool(((y.double() - want).abs() <= bound).all())
    # 8 bits
    bytes_, bbuf = guarded(x.shape, torch.uint8)
    found = qkr.rms_norm_fp8(x, w, residual=residual, out=bytes_.view(FP8), eps=eps)
    torch.cuda.synchronize()
    assert untouched(bbuf)
    assert torch.equal(bytes_.cpu(), in_8_bits(s, w).view(torch.uint8))
    top = (s.double() * (1.0 if w is None else w.double())).abs().amax(-1)
    rstd = normalised(s, eps)[1][:, 0]
    scale = torch.where(top == 0, torch.ones_like(top), top) * rstd / 448
    assert bool(((found[1].double() - scale).abs() <= 2 * C * scale + 2.0 ** -149).all())
    if residual is not None:
        assert same_bits(found[2], s)


@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 64), (5, 512), (70, 520), (2, 1000), (9, 1024), (6, 1032),
                                         (1, 2048), (33, 2056), (4, 4104), (1025, 5120), (3, 6152), (7, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward(rows, hidden, dtype):
    x, r = rows_of(1, rows, hidden, dtype), rows_of(2, rows, hidden, dtype)
    for param in (None, "fp32", "bf16", "fp16"):
        check_forward(x, r, weight_of(3, hidden, param))
    check_forward(x, None, weight_of(4, hidden, "fp32"))


def check_backward(dy, s, dsum, w, eps=EPS):
    n, rstd = normalised(s, eps)
    wd = 1.0 if w is None else w.double()
    dyd = dy.double()
    g = dyd * wd
    mean = (g * n).mean(-1, keepdim=True)
    want = rstd * (g - n * mean) + (0 if dsum is None else dsum.double())
    off = C * rstd * (g.abs() + 3 * n.abs() * (g * n).abs().mean(-1, keepdim=True))
    dx, buf = guarded(s.shape, s.dtype)
    _, dw = qkr.rms_norm_backward(dy, s, w, dsum=dsum, out=dx, eps=eps, param_grads=True)
    torch.cuda.synchronize()
    assert untouched(buf)
    bound = (half_step(s) + F) * want.abs() + (1 + half_step(s)) * off + tail(s)
    assert bool(((dx.double() - want).abs() <= bound).all())
    dwant = (dyd * n).sum(0)
    assert bool(((dw.double() - dwant).abs() <= (200 * F + C) * (dyd * n).abs().sum(0) + 2.0 ** -126).all())
    return dx, dw


@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 64), (5, 512), (70, 520), (2, 1000), (2500, 1024), (6, 1032),
                                         (1, 2048), (33, 2056), (4, 4104), (1025, 5120), (3, 6152), (515, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_backward(rows, hidden, dtype):
    s, dy, ds = rows_of(5, rows, hidden, dtype), rows_of(6, rows, hidden, dtype, 1 / 16), rows_of(7, rows, hidden, dtype)
    for param in (None, "fp32", "bf16", "fp16"):
        check_backward(dy, s, ds, weight_of(8, hidden, param))
    check_backward(dy, s, None, weight_of(9, hidden, "fp32"))
    dx, dw = qkr.rms_norm_backward(dy, s, weight_of(9, hidden, "fp32"), dsum=ds, param_grads=False)
    assert dw is None and same_bits(dx, check_backward(dy, s, ds, weight_of(9, hidden, "fp32"))[0])


def test_gradient_against_differences():
    """dx and dweight of sum(y dy) + sum(s dsum), by central differences of the
    64-bit formula."""
    rows, hidden, h = 3, 24, 1e-5
    s, dy, ds = (rows_of(i, rows, hidden, "fp16") for i in (10, 11, 12))
    w = weight_of(13, hidden, "fp32")
    dx, dw = qkr.rms_norm_backward(dy, s, w, dsum=ds)

    def loss(sv, wv):
        return float((normalised(sv)[0] * wv * dy.double()).sum() + (sv * ds.double()).sum())

    sd, wd = s.double(), w.double()
    for i in range(rows):
        for j in range(hidden):
            e = torch.zeros_like(sd)
            e[i, j] = h
            d = (loss(sd + e, wd) - loss(sd - e, wd)) / (2 * h)
            assert abs(float(dx[i, j]) - d) <= 2.0 ** -10 * (abs(d) + 1)
    for j in range(hidden):
        e = torch.zeros_like(wd)
        e[j] = h
        d = (loss(sd, wd + e) - loss(sd, wd - e)) / (2 * h)
        assert abs(float(dw[j]) - d) <= 1e-5 * (abs(d) + 1)


@pytest.mark.parametrize("hidden", [64, 1024, 2048, 8192])
@pytest.mark.parametrize("by", [1e37, 1e20, 1e-15, 1e-19, 1e-37])
def test_rows_whose_squares_leave_the_range(hidden, by):
    """bf16 rows up to its largest and down to its smallest numbers, beside ordinary ones."""
    x = rows_of(14, 6, hidden, "bf16")
    x[1::2] = (x[1::2].double() * by).to(x.dtype)
    w = weight_of(15, hidden, "fp32")
    for eps in (1e-6, 1e-38):
        check_forward(x, None, w, eps)
        dy = rows_of(16, 6, hidden, "bf16", 1 / 16)
        check_backward(dy, x, None, w, eps) if by < 1 or eps < 1e-30 or by == 1e20 else None


def test_gradients_whose_products_leave_the_range():
    s, dy = rows_of(17, 4, 2048, "bf16"), rows_of(18, 4, 2048, "bf16")
    s[1] *= 1e17
    dy[1] *= 1e22
    s[2] *= 1e-17
    dy[2] *= 1e-20
    w = weight_of(19, 2048, "fp32")
    for r in range(4):
        check_backward(dy[r:r + 1].contiguous(), s[r:r + 1].contiguous(), None, w)


@pytest.mark.parametrize("hidden", [512, 5120])
def test_rows_of_zeros_infinities_and_nan(hidden):
    x = rows_of(20, 5, hidden, "bf16")
    x[0] = 0
    x[1, 3] = math.inf
    x[2, hidden - 1] = math.nan
    x[4] = -0.0
    w = weight_of(21, hidden, "bf16")
    y = qkr.rms_norm(x, w)
    want = x.float() / torch.sqrt(x.float().square().mean(1, keepdim=True) + EPS)
    assert bool((y[[0, 4]] == 0).all()) and bool(torch.isnan(y[2]).all())
    assert torch.equal(torch.isnan(y[1]), torch.isnan(want[1])) and bool((y[1, 4:] == 0).all())
    q, scales = qkr.rms_norm_fp8(x, w)
    assert bool((q[[0, 4]].float() == 0).all()) and bool(torch.isnan(scales[1:3]).all())
    assert math.isfinite(float(scales[0])) and float(scales[0]) > 0
    # the others as without them
    for a, b in ((y[3:4], qkr.rms_norm(x[3:4].contiguous(), w)), (scales[3:4], qkr.rms_norm_fp8(x[3:4].contiguous(), w)[1])):
        assert same_bits(a, b)
    # a weight of zeros
    q, scales = qkr.rms_norm_fp8(x[3:4].contiguous(), torch.zeros_like(w))
    assert bool((q.float() == 0).all()) and bool(torch.isfinite(scales).all())
    # weights as large and as small as their type has
    for value in (3e38, 1e-38):
        big = torch.full((hidden,), value, device=DEV)
        q, scales = qkr.rms_norm_fp8(x[3:4].contiguous(), big)
        n = normalised(x[3:4])[0] * float(big[0])
        assert bool(torch.isfinite(q.float()).all())
        assert float((q.double() * scales.double()[:, None] - n).abs().max()) <= float(n.abs().max()) * (
            2.0 ** -4 if value > 1 else 1.0)


@pytest.mark.parametrize("hidden", [256, 2048])
def test_in_place_and_dimensions(hidden):
    x, r = rows_of(22, 12, hidden, "bf16").view(3, 4, hidden), rows_of(23, 12, hidden, "bf16").view(3, 4, hidden)
    w = weight_of(24, hidden, "bf16")
    y, s = qkr.rms_norm(x, w, residual=r)
    assert y.shape == s.shape == x.shape
    a, b = x.clone(), r.clone()
    out, total = qkr.rms_norm(a, w, residual=b, sum_out=b, out=a)
    assert out is a and total is b and same_bits(a, y) and same_bits(b, s)
    a, b = x.clone(), r.clone()
    out, total = qkr.rms_norm(a, w, residual=b, sum_out=a, out=b)
    assert same_bits(b, y) and same_bits(a, s)
    q, scales, total = qkr.rms_norm_fp8(x, w, residual=r)
    assert q.shape == x.shape and scales.shape == (3, 4) and same_bits(total, s)
    b = r.clone()
    assert torch.equal(qkr.rms_norm_fp8(x, w, residual=b, sum_out=b)[0].view(torch.uint8), q.view(torch.uint8))
    assert same_bits(b, s)
    dx, dw = qkr.rms_norm_backward(x, s, w, dsum=r)
    for name in ("dy", "dsum"):
        t = dict(dy=x.clone(), dsum=r.clone())
        got, gw = qkr.rms_norm_backward(t["dy"], s, w, dsum=t["dsum"], out=t[name])
        assert got is t[name] and same_bits(got, dx) and same_bits(gw, dw)
    # one tensor as both gradients
    both, _ = qkr.rms_norm_backward(x, s, w, dsum=x)
    t = x.clone()
    assert same_bits(qkr.rms_norm_backward(t, s, w, dsum=t, out=t)[0], both)


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    y, s = qkr.rms_norm(x, w, residual=x)
    q, scales = qkr.rms_norm_fp8(x, w)
    dx, dw = qkr.rms_norm_backward(x, x, w)
    assert y.shape == s.shape == dx.shape == q.shape == (0, 64) and scales.shape == (0,) and bool((dw == 0).all())


def test_streams_and_graphs():
    """The same bits on another stream and from a graph replayed on new rows."""
    s = dict(x=rows_of(25, 300, 2048, "bf16"), r=rows_of(26, 300, 2048, "bf16"), dy=rows_of(27, 300, 2048, "bf16"))
    w = weight_of(28, 2048, "fp32")

    def step():
        y, total = qkr.rms_norm(s["x"], w, residual=s["r"])
        q, scales = qkr.rms_norm_fp8(total, w)
        dx, dw = qkr.rms_norm_backward(s["dy"], total, w, dsum=s["r"])
        return [y, total, q.view(torch.int16), scales, dx, dw]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        y, total = qkr.rms_norm(s["x"], w, residual=s["r"], stream=stream)
        dx, dw = qkr.rms_norm_backward(s["dy"], total, w, dsum=s["r"], stream=stream)
        side.synchronize()
        assert same_bits(y, want[0]) and same_bits(dx, want[4]) and same_bits(dw, want[5])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        for j, t in enumerate(s.values()):
            t.copy_(rows_of(30 + 3 * i + j, 300, 2048, "bf16"))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(kept, want))


def test_tensors_past_4_gib():
    """Offsets of 2^32 bytes and more: the last rows equal those of a small call."""
    rows, hidden = 270000, 8192
    x = torch.empty((rows, hidden), dtype=torch.bfloat16, device=DEV)
    x.view(-1)[:1 << 20].normal_()
    x.view(-1)[-(1 << 20):].normal_()
    x[128:-128] = 0.5
    w = weight_of(29, hidden, "bf16")
    last = x[-64:].clone()
    y, s = qkr.rms_norm(x, w, residual=x)
    ys, ss = qkr.rms_norm(last, w, residual=last)
    assert same_bits(y[-64:], ys) and same_bits(s[-64:], ss)
    q, scales = qkr.rms_norm_fp8(x, w)
    qs, scale = qkr.rms_norm_fp8(last, w)
    assert torch.equal(q[-64:].view(torch.uint8), qs.view(torch.uint8)) and same_bits(scales[-64:], scale)
    dx, _ = qkr.rms_norm_backward(y, x, w, dsum=s)
    assert same_bits(dx[-64:], qkr.rms_norm_backward(ys, last, w, dsum=ss)[0])
