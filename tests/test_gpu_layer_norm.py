"""Layer norm forward and backward, and the backward pass of the AdaLN
modulation, on the GPU against 64 bits.

Bounds, with u half a step of the 16-bit type and c = 64 * 2^-24 (the sums of a
row are trees of at most 44 fp32 additions, the rest of a value's path is
under 20 operations): the mean is off by c avg|x|, so n = (x - mean) rstd by
e_n = c (avg|x| rstd + |n|); the other bounds carry that through the formulas.
dweight and dbias: at most 200 additions one after another (the rows of a
chunk, then its chunks in 16 runs).
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests.gpu_common import same_bits

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
F = 2.0 ** -24
C = 64 * F
PAD = 4096


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows_of(seed, rows, hidden, dtype, by=1.0):
    g = gen(seed)
    s = torch.exp((torch.rand((rows, 1), generator=g) * 2 - 1) * math.log(10.0))
    return ((torch.randn((rows, hidden), generator=g) + 0.5 * torch.randn(hidden, generator=g)) * s * by).to(
        TYPES[dtype]).to(DEV)


def params_of(seed, shape, dtype):
    g = gen(seed)
    return tuple((a + 0.3 * torch.randn(shape, generator=g)).to(TYPES[dtype]).to(DEV) for a in (1, 0))


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def tail(t):
    return torch.finfo(t.dtype).smallest_normal * torch.finfo(t.dtype).eps / 2


def normalised(x, eps=EPS):
    x = x.double()
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    n = (x - mean) * rstd
    e_n = C * (x.abs().mean(-1, keepdim=True) * rstd + n.abs())
    return n, rstd, e_n


def guarded(shape, dtype, fill=7.0):
    size = math.prod(shape)
    buf = torch.full((size + 2 * PAD,), fill, dtype=dtype, device=DEV)
    return buf[PAD:PAD + size].view(shape), buf


def untouched(buf, fill=7.0):
    return bool((buf[:PAD] == fill).all() and (buf[-PAD:] == fill).all())


def check_forward(x, w, b, eps=EPS):
    y, buf = guarded(x.shape, x.dtype)
    qkr.layer_norm(x, w, b, out=y, eps=eps)
    torch.cuda.synchronize()
    assert untouched(buf)
    n, _, e_n = normalised(x, eps)
    wd = 1.0 if w is None else w.double()
    bd = 0.0 if b is None else b.double()
    want = n * wd + bd
    size = (n * wd).abs() + abs(bd)
    bound = half_step(x) * want.abs() + e_n * abs(wd) + 4 * F * size + tail(x)
    assert ((y.double() - want).abs() <= bound).all(), float(((y.double() - want).abs() - bound).max())
    return y


def check_backward(dy, x, w, one, per, got, eps=EPS):
    """w: [batches, hidden] or None; one: added to it; per: rows of a batch."""
    dx, dw, db = got
    rows, hidden = x.shape
    n, rstd, e_n = normalised(x, eps)
    d = dy.double()
    at = torch.arange(rows, device=DEV) // per
    g = d if w is None else d * (w.double() + one)[at]
    e_g = 2 * F * g.abs()
    c1, c2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    want = rstd * (g - c1 - n * c2)
    e_c1 = C * g.abs().mean(1, keepdim=True)
    e_c2 = C * (g * n).abs().mean(1, keepdim=True) + (g.abs() * e_n).mean(1, keepdim=True)
    size = g.abs() + c1.abs() + (n * c2).abs()
    bound = (half_step(x) * want.abs() + tail(x)
             + rstd * (e_g + e_c1 + n.abs() * e_c2 + e_n * (c2.abs() + e_c2) + C * size))
    off = (dx.double() - want).abs()
    assert (off <= bound).all(), "dx: %g" % float((off - bound).max())
    if w is None:
        assert dw is None and db is None
        return
    batches = w.shape[0]
    sums = [torch.zeros((batches, hidden), dtype=torch.float64, device=DEV) for _ in range(4)]
    for s, v in zip(sums, (d * n, d, (d * n).abs() * 200 * F + d.abs() * e_n, d.abs() * 200 * F)):
        s.index_add_(0, at, v)
    assert ((dw.double().view_as(sums[0]) - sums[0]).abs() <= sums[2] + 1e-30).all(), "dweight"
    assert ((db.double().view_as(sums[1]) - sums[1]).abs() <= sums[3] + 1e-30).all(), "dbias"


WIDTHS = [8, 64, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4088, 5120, 6144, 6152, 8192]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_forward_and_backward_by_width(hidden, dtype):
    rows = 37
    x, dy = rows_of(hidden, rows, hidden, dtype), rows_of(hidden + 1, rows, hidden, dtype, 1 / 16)
    w, b = params_of(hidden, (hidden,), "fp32")
    keep = [t.clone() for t in (x, dy, w, b)]
    check_forward(x, w, b)
    dx, buf = guarded(x.shape, x.dtype)
    got = qkr.layer_norm_backward(dy, x, w, out=dx)
    torch.cuda.synchronize()
    assert untouched(buf) and got[0] is dx
    check_backward(dy, x, w[None], 0.0, rows, got)
    assert all(same_bits(a, c) for a, c in zip(keep, (x, dy, w, b)))


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 767, 769, 5000])
@pytest.mark.parametrize("hidden", [72, 1160])
def test_row_counts(rows, hidden):
    x, dy = rows_of(rows, rows, hidden, "bf16"), rows_of(rows + 1, rows, hidden, "bf16", 1 / 16)
    w, b = params_of(rows, (hidden,), "bf16")
    check_forward(x, w, b)
    check_backward(dy, x, w[None], 0.0, rows, qkr.layer_norm_backward(dy, x, w))


@pytest.mark.parametrize("param", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_parameter_types(dtype, param):
    x, dy = rows_of(3, 50, 640, dtype), rows_of(4, 50, 640, dtype)
    w, b = params_of(5, (640,), param)
    check_forward(x, w, b)
    check_backward(dy, x, w[None], 0.0, 50, qkr.layer_norm_backward(dy, x, w))


def test_without_weight_or_bias():
    x, dy = rows_of(6, 50, 1200, "bf16"), rows_of(7, 50, 1200, "bf16")
    w, b = params_of(8, (1200,), "fp32")
    check_forward(x, None, None)
    check_forward(x, w, None)
    check_forward(x, None, b)
    check_backward(dy, x, None, 0.0, 50, qkr.layer_norm_backward(dy, x))


@pytest.mark.parametrize("rows,batches,per", [(120, 4, None), (120, 120, None), (100, 3, 40), (100, 7, 15),
                                              (1000, 2, None), (5, 1, 9), (3000, 1000, None)])
@pytest.mark.parametrize("hidden", [256, 2560])
def test_modulation_gradients(rows, batches, per, hidden):
    """Whole batches, one row each, a short last batch, more batches than workgroups."""
    x, dy = rows_of(9, rows, hidden, "bf16"), rows_of(10, rows, hidden, "bf16", 1 / 16)
    scale = params_of(11, (batches, hidden), "fp32")[1]
    got = qkr.fuse_scale_shift_backward(dy, x, scale, rows_per_batch=per)
    check_backward(dy, x, scale, 1.0, per or rows // batches, got)


@pytest.mark.parametrize("param", ["bf16", "fp16"])
def test_modulation_of_16_bits(param):
    """1 + scale is formed in fp32, not in the scale's type."""
    x, dy = rows_of(9, 60, 512, "bf16"), rows_of(10, 60, 512, "bf16", 1 / 16)
    scale = (params_of(11, (2, 512), "fp32")[1] / 100).to(TYPES[param])
    check_backward(dy, x, scale, 1.0, 30, qkr.fuse_scale_shift_backward(dy, x, scale))


def test_modulation_rows_that_no_row_uses_get_zeros():
    x, dy = rows_of(12, 20, 128, "bf16"), rows_of(13, 20, 128, "bf16")
    scale = params_of(14, (5, 128), "fp32")[1]
    got = qkr.fuse_scale_shift_backward(dy, x, scale, rows_per_batch=9)
    check_backward(dy, x, scale, 1.0, 9, got)
    assert (got[1][3:] == 0).all() and (got[2][3:] == 0).all()


@pytest.mark.parametrize("hidden", [200, 3000])
def test_in_place(hidden):
    x, dy = rows_of(15, 400, hidden, "bf16"), rows_of(16, 400, hidden, "bf16")
    w, b = params_of(17, (hidden,), "fp32")
    y, z = qkr.layer_norm(x, w, b), x.clone()
    assert qkr.layer_norm(z, w, b, out=z) is z and same_bits(y, z)
    want, d = qkr.layer_norm_backward(dy, x, w), dy.clone()
    got = qkr.layer_norm_backward(d, x, w, out=d)
    assert all(same_bits(a, c) for a, c in zip(got, want)) and got[0] is d


@pytest.mark.parametrize("hidden", [256, 2560])
@pytest.mark.parametrize("eps", [1e-6, 1e-35])
def test_values_at_the_ends_of_the_range(hidden, eps):
    """Rows whose squares overflow or sink below fp32's normal range, constant
    rows and zeros, beside ordinary ones."""
    x = rows_of(18, 12, hidden, "bf16")
    big = 2.0 ** 110 * rows_of(19, 12, hidden, "bf16").double()
    small = 2.0 ** -120 * rows_of(20, 12, hidden, "bf16").double()
    x[1] = big[1].to(x.dtype)
    x[3] = small[3].to(x.dtype)
    x[5] = 3.0
    x[7] = 0.0
    x[9] = 1e38
    w, b = params_of(21, (hidden,), "fp32")
    y = check_forward(x, w, b, eps)
    assert same_bits(y[7], b.to(x.dtype)) and same_bits(y[5], b.to(x.dtype))
    dy = rows_of(22, 12, hidden, "bf16", 1e-3)
    ordinary = [0, 1, 2, 4, 6, 8, 10, 11]       # the others' dx is as large as rstd: 1 / sqrt(eps)
    got = qkr.layer_norm_backward(dy[ordinary], x[ordinary], w, eps=eps)
    check_backward(dy[ordinary], x[ordinary], w[None], 0.0, 12, got, eps)


def test_a_nan_stays_in_its_row():
    x, dy = rows_of(23, 30, 1096, "bf16"), rows_of(24, 30, 1096, "bf16")
    w, b = params_of(25, (1096,), "fp32")
    y = qkr.layer_norm(x, w, b)
    x[7, 5] = math.nan
    y2 = qkr.layer_norm(x, w, b)
    dx = qkr.layer_norm_backward(dy, x, w)[0]
    others = [i for i in range(30) if i != 7]
    assert torch.isnan(y2[7]).all() and same_bits(y2[others], y[others])
    assert torch.isnan(dx[7]).all() and torch.isfinite(dx[others]).all()


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    assert qkr.layer_norm(x, w).shape == (0, 64)
    dx, dw, db = qkr.layer_norm_backward(x, x, w)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_leading_dimensions():
    x, dy = rows_of(26, 24, 320, "bf16"), rows_of(27, 24, 320, "bf16")
    w, _ = params_of(28, (320,), "fp32")
    a = qkr.layer_norm_backward(dy.view(2, 3, 4, 320), x.view(2, 3, 4, 320), w)
    c = qkr.layer_norm_backward(dy, x, w)
    assert a[0].shape == (2, 3, 4, 320) and same_bits(a[0].view(24, 320), c[0])
    assert same_bits(a[1], c[1]) and same_bits(a[2], c[2])


def test_against_differences_of_the_64_bit_forward():
    x, dy = rows_of(29, 20, 96, "bf16"), rows_of(30, 20, 96, "bf16")
    w, b = params_of(31, (96,), "fp32")
    dx, dw, db = (t.double() for t in qkr.layer_norm_backward(dy, x, w))

    def loss(x, w, b):
        return float(((normalised(x)[0] * w + b) * dy.double()).sum())

    args, h = [t.double() for t in (x, w, b)], 1e-6
    for i, g in enumerate((dx, dw, db)):
        t = torch.randn(args[i].shape, generator=gen(i), dtype=torch.float64).to(DEV)
        ends = [loss(*[a + s * h * t if j == i else a for j, a in enumerate(args)]) for s in (1, -1)]
        slack = (half_step(x) if i == 0 else 200 * F) * float((g.abs() * t.abs()).sum())
        # the elementwise bounds above, dominated by the roundings of dx, plus h^2 terms
        assert abs((ends[0] - ends[1]) / (2 * h) - float((g * t).sum())) <= 2 * slack + 1e-3


def test_runs_streams_and_graph_replays_give_the_same_bits():
    x, dy = rows_of(32, 3000, 1280, "bf16"), rows_of(33, 3000, 1280, "bf16")
    w, b = params_of(34, (1280,), "fp32")
    scale = params_of(35, (3, 1280), "fp32")[1]

    def step():
        return (qkr.layer_norm(x, w, b), *qkr.layer_norm_backward(dy, x, w),
                *qkr.fuse_scale_shift_backward(dy, x, scale))

    want = step()
    assert all(same_bits(a, c) for a, c in zip(step(), want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = qkr.layer_norm_backward(dy, x, w, stream=st)
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    assert all(same_bits(a, c) for a, c in zip(other, want[1:4]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(3):
        x.copy_(rows_of(40 + i, 3000, 1280, "bf16"))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, c) for a, c in zip(kept, want))


@pytest.mark.parametrize("hidden", [256, 2560])
@pytest.mark.parametrize("eps", [1e-6, 1e-35])
def test_gradients_at_the_ends_of_the_range(hidden, eps):
    """The rows of test_values_at_the_ends_of_the_range, backwards: dx is as
    large as rstd, at most 1 / sqrt(eps), which bf16 holds."""
    x = rows_of(18, 12, hidden, "bf16")
    big = 2.0 ** 110 * rows_of(19, 12, hidden, "bf16").double()
    small = 2.0 ** -120 * rows_of(20, 12, hidden, "bf16").double()
    x[1] = big[1].to(x.dtype)
    x[3] = small[3].to(x.dtype)
    x[5] = 3.0
    x[7] = 0.0
    x[9] = 1e38
    w = params_of(21, (hidden,), "fp32")[0]
    dy = rows_of(22, 12, hidden, "bf16", 1e-3)
    got = qkr.layer_norm_backward(dy, x, w, eps=eps)
    check_backward(dy, x, w[None], 0.0, 12, got, eps)


@pytest.mark.parametrize("one", [0.0, 1.0])
@pytest.mark.parametrize("hidden", [256, 2560])
@pytest.mark.parametrize("eps", [1e-6, 1e-35, 1e-37, 3e-45])
def test_gradients_of_constant_rows(hidden, eps, one):
    """A row of one value has n = 0 exactly (up to 8192 copies of a 16-bit value
    add up without rounding), so dx = (g - avg g) / sqrt(eps) whatever the
    value, dweight is 0 and dbias the sum of dy.  eps is the fp32 number."""
    values = [3.0, 0.0, 1024.0, -1e38, 1e18, 2.0 ** -100, 3e38, -2.0 ** -126, 1e30]
    x = torch.tensor(values)[:, None].expand(-1, hidden).bfloat16().to(DEV)
    dy = rows_of(36, len(values), hidden, "bf16", 1e-3)
    w = params_of(37, (1, hidden), "fp32")[0]
    if one:
        dx, dw, db = qkr.fuse_scale_shift_backward(dy, x, w, eps=eps)
    else:
        dx, dw, db = qkr.layer_norm_backward(dy, x, w[0], eps=eps)
    g = dy.double() * (w.double() + one)
    c1 = g.mean(1, keepdim=True)
    rstd = float(torch.tensor(eps, dtype=torch.float32).double()) ** -0.5
    want = rstd * (g - c1)
    bound = half_step(x) * want.abs() + tail(x) + rstd * (
        C * g.abs().mean(1, keepdim=True) + C * (g.abs() + c1.abs()))
    off = (dx.double() - want).abs()
    assert (off <= bound).all(), [float(v) for v in (off - bound).amax(1)]
    assert (dw == 0).all()
    assert ((db.double().view(-1) - dy.double().sum(0)).abs() <= 200 * F * dy.double().abs().sum(0)).all()


def test_products_of_large_values_and_gradients():
    """x of 1e17, whose squares still add up in fp32, times gradients of 1e22,
    whose products with it do not: dx is about 1e5."""
    for hidden in (256, 2560):
        x = rows_of(38, 12, hidden, "bf16", 1e17)
        dy = rows_of(39, 12, hidden, "bf16", 1e22)
        w = params_of(40, (hidden,), "fp32")[0]
        check_backward(dy, x, w[None], 0.0, 12, qkr.layer_norm_backward(dy, x, w))


@pytest.mark.parametrize("rows,hidden", [(50, 1200), (3, 64), (2000, 512)])
def test_sums_are_to_be_had_without_a_weight(rows, hidden):
    """A layer norm with a bias alone has a bias gradient: the weight of ones' bits."""
    x, dy = rows_of(6, rows, hidden, "bf16"), rows_of(7, rows, hidden, "bf16")
    ones = torch.ones(hidden, device=DEV)
    want = qkr.layer_norm_backward(dy, x, ones)
    got = qkr.layer_norm_backward(dy, x, param_grads=True)
    check_backward(dy, x, ones[None], 0.0, rows, got)
    assert all(same_bits(a, b) for a, b in zip(got, want))
    dx, dw, db = qkr.layer_norm_backward(dy, x, ones, param_grads=False)
    assert same_bits(dx, want[0]) and dw is None and db is None


def test_errors_name_the_tensor_of_the_wrong_type():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    for call, names in ((lambda: qkr.layer_norm(x, w.double()), "^weight/bias must"),
                        (lambda: qkr.layer_norm(x, None, w.int()), "^weight/bias must"),
                        (lambda: qkr.layer_norm(x.float(), w), "^x must"),
                        (lambda: qkr.layer_norm_backward(x, x, w.double()), "^weight must"),
                        (lambda: qkr.layer_norm_backward(x.float(), x.float(), w), "^x must"),
                        (lambda: qkr.fuse_scale_shift_backward(x, x, w.double()), "^scale must"),
                        (lambda: qkr.attention(*[x.float().view(1, 1, 4, 64)] * 3), "^q/k/v must")):
        with pytest.raises(ValueError, match=names):
            call()


def test_rows_past_4_gib():
    """x, dy and dx of more than 2^32 bytes: rows at either end and around the
    border have a small call's bits, and the sums hold every row (512 rows of a
    chunk one after another, then its chunks in 16 runs: 600 additions)."""
    rows, hidden = 262500, 8192
    g = torch.Generator(device=DEV).manual_seed(41)
    x = torch.randn((rows, hidden), generator=g, device=DEV, dtype=torch.bfloat16)
    dy = torch.randn((rows, hidden), generator=g, device=DEV, dtype=torch.bfloat16)
    w, b = params_of(42, (hidden,), "fp32")
    some = torch.tensor([0, 1, 262143, 262144, 262145, rows - 2, rows - 1], device=DEV)
    assert same_bits(qkr.layer_norm(x, w, b)[some], qkr.layer_norm(x[some], w, b))
    dx, dw, db = qkr.layer_norm_backward(dy, x, w)
    assert same_bits(dx[some], qkr.layer_norm_backward(dy[some], x[some], w)[0])
    del dx
    sums = [torch.zeros(hidden, dtype=torch.float64, device=DEV) for _ in range(4)]
    for at in range(0, rows, 8192):
        n, _, e_n = normalised(x[at:at + 8192])
        d = dy[at:at + 8192].double()
        for s, v in zip(sums, (d * n, d, (d * n).abs() * 600 * F + d.abs() * e_n, d.abs() * 600 * F)):
            s += v.sum(0)
    assert ((dw.double() - sums[0]).abs() <= sums[2]).all() and ((db.double() - sums[1]).abs() <= sums[3]).all()
