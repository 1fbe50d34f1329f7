"""The backward pass of QK-norm + RoPE on the GPU against 64 bits.

Bounds, with u half a step of the 16-bit type and c = 64 * 2^-24 (a head's sums
are 8 additions in a lane and at most 5 across lanes; the rest of a value's
path is under 20 operations): dn is off by c times the sum of its terms'
magnitudes, u_d = x r by c |u_d|, and so on through the formulas.  dgamma: at
most 400 additions one after another (the heads and tokens of a lane, then
the workgroups in 64 runs).
"""
import math

import numpy as np
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
import workloads as wl
from tests.gpu_common import same_bits

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F = 2.0 ** -24
C = 64 * F
EPS = 1e-6


def tables(tokens, heads, d, style, layout, dtype):
    """Not rotations: cosines and sines that differ between the two of a pair."""
    g = torch.Generator().manual_seed(tokens * 7 + d)
    rows = (tokens, heads, d) if layout == "per_head" else (tokens, d)
    return [torch.randn(rows, generator=g).to(torch.float32 if dtype == "fp32" else torch.bfloat16).to(DEV)
            for _ in range(2)]


def pair(style, d):
    i = torch.arange(d)
    if style == "interleaved":
        return i ^ 1, torch.where(i % 2 == 0, 1.0, -1.0).double()
    return (i + d // 2) % d, torch.where(i < d // 2, 1.0, -1.0).double()


def reference(x, do, gamma, cos, sin, style, eps=EPS):
    """x, do [tokens, heads, d] -> dx and dgamma with their bounds, 64 bits."""
    d = x.shape[2]
    partner, sign = pair(style, d)
    sign = sign.to(DEV)
    c, s = (t.double().view(t.shape[0], -1, d) for t in (cos, sin))
    xd, g0 = x.double(), do.double()
    one, two = g0 * c, sign * g0[..., partner] * s[..., partner]
    dn, e_dn = one + two, C * (one.abs() + two.abs())
    r = 1 / torch.sqrt(xd.square().mean(2, keepdim=True) + eps)
    u = xd * r
    g, e_g = dn * gamma.double(), (e_dn + 2 * F * dn.abs()) * gamma.double().abs()
    m = (g * u).mean(2, keepdim=True)
    e_m = (e_g * u.abs() + C * (g * u).abs()).mean(2, keepdim=True)
    want = r * (g - u * m)
    step = torch.finfo(x.dtype).eps / 2
    bound = (step * want.abs() + r * (e_g + u.abs() * e_m + C * (g.abs() + (u * m).abs()))
             + torch.finfo(x.dtype).smallest_normal * step * 2)
    dgamma = (dn * u).sum((0, 1))
    e_dgamma = (e_dn * u.abs() + (400 * F + C) * (dn * u).abs()).sum((0, 1))
    return want, bound, dgamma, e_dgamma


def inputs(seed, tokens, heads, d, dtype):
    g = torch.Generator().manual_seed(seed)
    s = torch.exp((torch.rand((tokens, 1, 1, 1), generator=g) * 2 - 1) * math.log(10.0))
    x = (torch.randn((tokens, 3, heads, d), generator=g) * s).to(TYPES[dtype]).to(DEV)
    do = (torch.randn((tokens, 3, heads, d), generator=g) / 16).to(TYPES[dtype]).to(DEV)
    gam = [(1 + 0.3 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    return x, do, gam


def check(x, do, gam, cos, sin, style, layout, eps=EPS):
    tokens, _, heads, d = x.shape
    kw = dict(q_gamma=gam[0], k_gamma=gam[1], cos=cos, sin=sin, eps=eps, style=style, cos_layout=layout)
    flat = do.clone().view(tokens, -1)
    before = x.clone()
    dg = qkr.qknorm_rope_backward(flat, x.view(tokens, -1), **kw)
    torch.cuda.synchronize()
    got = flat.view(tokens, 3, heads, d)
    assert same_bits(x, before) and same_bits(got[:, 2].contiguous(), do[:, 2].contiguous())
    for i in range(2):
        want, bound, dgamma, e_dgamma = reference(x[:, i], do[:, i], gam[i], cos, sin, style, eps)
        off = (got[:, i].double() - want).abs()
        assert (off <= bound).all(), float((off - bound).max())
        assert ((dg[i].double() - dgamma).abs() <= e_dgamma + 1e-30).all()
    return got, dg


@pytest.mark.parametrize("table", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["shared", "per_head"])
@pytest.mark.parametrize("style", ["interleaved", "rotate_half"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_form(d, dtype, style, layout, table):
    x, do, gam = inputs(d, 43, 5, d, dtype)
    check(x, do, gam, *tables(43, 5, d, style, layout, table), style, layout)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (2, 40), (3, 3), (255, 24), (4095, 5), (5000, 2), (9, 97)])
def test_sizes(tokens, heads):
    x, do, gam = inputs(tokens, tokens, heads, 128, "bf16")
    check(x, do, gam, *tables(tokens, heads, 128, "interleaved", "shared", "fp32"), "interleaved", "shared")


def test_separate_tensors_and_outputs_of_their_own():
    x, do, gam = inputs(1, 75, 7, 64, "bf16")
    cos, sin = tables(75, 7, 64, "rotate_half", "shared", "fp32")
    got, dg = check(x, do, gam, cos, sin, "rotate_half", "shared")
    kw = dict(q_gamma=gam[0], k_gamma=gam[1], cos=cos, sin=sin, eps=EPS, style="rotate_half")
    q, k, dq, dk = (t[:, i].contiguous() for t in (x, do) for i in range(2))
    keep = dq.clone()
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    g2 = qkr.qknorm_rope_backward(dq=dq, dk=dk, q=q, k=k, dq_out=oq, dk_out=ok, **kw)
    want = [got[:, i].contiguous() for i in range(2)]
    assert same_bits(oq, want[0]) and same_bits(ok, want[1]) and same_bits(dq, keep)
    # the sums of dgamma are taken over other runs of tokens only when one tensor is given
    assert same_bits(g2[0], dg[0]) and same_bits(g2[1], dg[1])
    only, none = qkr.qknorm_rope_backward(dq=dq, q=q, **kw)
    assert none is None and same_bits(dq, want[0])
    torch.testing.assert_close(only, dg[0], rtol=1e-4, atol=1e-4)
    none, only = qkr.qknorm_rope_backward(dk=dk, k=k, **kw)
    assert none is None and same_bits(dk, want[1])
    out = torch.full((75, 3 * 7 * 64), 5.0, dtype=x.dtype, device=DEV)
    src = do.clone().view(75, -1)
    qkr.qknorm_rope_backward(src, x.view(75, -1), out=out, **kw)
    assert same_bits(src, do.view(75, -1)) and (out[:, 2 * 7 * 64:] == 5).all()
    assert same_bits(out.view(75, 3, 7, 64)[:, 1].contiguous(), want[1])


@pytest.mark.parametrize("eps", [1e-6, 1e-35])
def test_heads_at_the_ends_of_the_range(eps):
    """Heads whose squares overflow or sink below fp32's normal range, and
    zeros, beside ordinary ones."""
    x, do, gam = inputs(2, 20, 4, 128, "bf16")
    x[3, :, 1] = (x[3, :, 1].double() * 2.0 ** 100).to(x.dtype)
    x[5, :, 2] = (x[5, :, 2].double() * 2.0 ** -90).to(x.dtype)
    if eps == 1e-6:
        x[7, :, 0] = 0.0
    check(x, do, gam, *tables(20, 4, 128, "interleaved", "shared", "fp32"), "interleaved", "shared", eps)


def test_a_nan_stays_in_its_head():
    x, do, gam = inputs(3, 30, 4, 64, "bf16")
    cos, sin = tables(30, 4, 64, "interleaved", "shared", "fp32")
    kw = dict(q_gamma=gam[0], k_gamma=gam[1], cos=cos, sin=sin, eps=EPS)
    a, b = do.clone().view(30, -1), do.clone().view(30, -1)
    qkr.qknorm_rope_backward(a, x.view(30, -1), **kw)
    x[4, 0, 2, 9] = math.nan
    qkr.qknorm_rope_backward(b, x.view(30, -1), **kw)
    a, b = a.view(30, 3, 4, 64), b.view(30, 3, 4, 64)
    assert torch.isnan(b[4, 0, 2]).all()
    b[4, 0, 2] = a[4, 0, 2]
    assert same_bits(a, b)


def test_no_tokens():
    kw = dict(q_gamma=torch.ones(64, device=DEV), k_gamma=torch.ones(64, device=DEV),
              cos=torch.empty((0, 64), device=DEV), sin=torch.empty((0, 64), device=DEV))
    x = torch.empty((0, 3 * 2 * 64), dtype=torch.bfloat16, device=DEV)
    a, b = qkr.qknorm_rope_backward(x, x, **kw)
    assert (a == 0).all() and (b == 0).all()


@pytest.mark.parametrize("style", ["interleaved", "rotate_half"])
def test_against_the_forward_kernel(style):
    """With a true rotation the forward pass keeps each head's norm, so x and dx
    are orthogonal up to eps: sum_d x dx = r^3 eps sum_d x g.  And the pass is
    linear along x: differences of the forward kernel's own 64-bit oracle."""
    import oracle

    t, h, d = 12, 3, 64
    x, do, gam = inputs(4, t, h, d, "fp16")
    cos, sin = wl.rope_tables(np.arange(t) * 3, (d // 2,), d, style)
    flat = do.clone().view(t, -1)
    qkr.qknorm_rope_backward(flat, x.view(t, -1), q_gamma=gam[0], k_gamma=gam[1], cos=cos.to(DEV),
                             sin=sin.to(DEV), eps=EPS, style=style)
    dx = flat.view(t, 3, h, d)[:, :2].double().cpu()
    gen = torch.Generator().manual_seed(5)
    step = torch.randint(-2, 3, (t, 3, h, d), generator=gen).double() * 2.0 ** -9
    losses = []
    for sign in (1, -1):
        # a step that 16 bits hold exactly would round: the oracle takes 16-bit
        # inputs, so both ends are rounded and their true difference is used
        xs = (x.double().cpu() + sign * step).half()
        q, k = oracle.fused_qk(wl.u16(xs.view(t, -1)), "fp16", heads=h, head_dim=d,
                               q_gamma=gam[0].cpu().numpy(), k_gamma=gam[1].cpu().numpy(), eps=EPS,
                               cos=cos.numpy(), sin=sin.numpy(), style=style)
        o = torch.stack([torch.from_numpy(np.asarray(v)).view(t, h, d) for v in (q, k)], 1)
        losses.append((float((o * do[:, :2].double().cpu()).sum()), xs.double()))
    along = float((dx * (losses[0][1] - losses[1][1])[:, :2]).sum())
    # roundings of dx along the step, and the third-order terms of the
    # difference: (|step| r)^3 of each head, |step| r <= 2^-8 / 0.08
    slack = float((dx.abs() * (losses[0][1] - losses[1][1])[:, :2].abs()).sum()) * 2.0 ** -11
    cubic = float(do.double().abs().sum()) * 2 * (2.0 ** -8 / 0.08) ** 3
    assert abs(losses[0][0] - losses[1][0] - along) <= slack + cubic


def test_runs_streams_and_graph_replays_give_the_same_bits():
    x, do, gam = inputs(6, 700, 8, 128, "bf16")
    cos, sin = tables(700, 8, 128, "interleaved", "shared", "fp32")
    out = torch.zeros((700, 3 * 8 * 128), dtype=x.dtype, device=DEV)
    xf, df = x.view(700, -1), do.view(700, -1)

    def step(**kw):
        return qkr.qknorm_rope_backward(df, xf, out=out, q_gamma=gam[0], k_gamma=gam[1], cos=cos, sin=sin,
                                        eps=EPS, **kw)

    want = (*step(), out.clone())
    assert all(same_bits(a, c) for a, c in zip((*step(), out), want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = step(stream=st)
    st.synchronize()
    assert all(same_bits(a, c) for a, c in zip((*got, out), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(3):
        x.copy_(inputs(50 + i, 700, 8, 128, "bf16")[0])
        want = (*step(), out.clone())
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, c) for a, c in zip((*kept, out), want))


def test_products_of_large_values_and_gradients():
    """x of 1e17, whose squares still add up in fp32, times gradients of 1e23,
    whose products with it do not: dx is about 1e6."""
    x, do, gam = inputs(7, 20, 4, 128, "bf16")
    x, do = (x.double() * 1e17).to(x.dtype), (do.double() * 1e24).to(x.dtype)
    check(x, do, gam, *tables(20, 4, 128, "interleaved", "shared", "fp32"), "interleaved", "shared")


def test_tokens_past_4_gib():
    """A fused buffer of more than 2^32 bytes: tokens at either end and around
    the border have a small call's bits, and dgamma holds every token (a lane's
    35 tokens of 10 heads, then the waves, 32 parts of a run and 18 for the runs:
    404 additions, for which the bound has 400 and what C leaves of 64)."""
    tokens, heads, d = 139900, 40, 128
    g = torch.Generator(device=DEV).manual_seed(8)
    x, do = (torch.randn((tokens, 3 * heads * d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    gam = inputs(9, 1, 1, d, "bf16")[2]
    cos, sin = (torch.randn((tokens, d), generator=g, device=DEV) for _ in range(2))
    some = torch.tensor([0, 1, 139808, 139809, 139810, 139811, tokens - 2, tokens - 1], device=DEV)
    kw = dict(q_gamma=gam[0], k_gamma=gam[1], eps=EPS)
    few = do[some]
    qkr.qknorm_rope_backward(few, x[some], cos=cos[some], sin=sin[some], **kw)
    out = torch.full_like(x, 3.0)
    dg = qkr.qknorm_rope_backward(do, x, cos=cos, sin=sin, out=out, **kw)
    n = 2 * heads * d
    assert same_bits(out[some][:, :n].contiguous(), few[:, :n].contiguous()) and (out[:, n:] == 3).all()
    del out
    sums = torch.zeros((2, 2, d), dtype=torch.float64, device=DEV)
    for at in range(0, tokens, 4096):
        run = slice(at, at + 4096)
        parts = [t[run].view(-1, 3, heads, d) for t in (x, do)]
        for i in range(2):
            _, _, dgamma, e_dgamma = reference(parts[0][:, i], parts[1][:, i], gam[i], cos[run], sin[run], "interleaved")
            sums[i, 0] += dgamma
            sums[i, 1] += e_dgamma
    for i in range(2):
        assert ((dg[i].double() - sums[i, 0]).abs() <= sums[i, 1]).all()
