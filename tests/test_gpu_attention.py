"""Attention and its backward pass on the GPU against 64 bits.

Every element is held to the bound of tests/attention_reference.py, which
counts the roundings of the 16-bit operands and outputs and the fp32 sums.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests import attention_reference as ref
from tests.gpu_common import same_bits

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def draw(seed, *shape, dtype="bf16", by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * by).to(TYPES[dtype]).to(DEV)


def within(got, want, bound, what):
    """got [batch, tokens, heads, d] (16 bits), want and bound heads first."""
    got = got.double().permute(0, 2, 1, 3)
    assert torch.isfinite(got).all(), what + ": not finite"
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, "%s: %g over its bound at %s" % (
        what, worst, [int(i) for i in torch.unravel_index(over.argmax(), over.shape)])


def lengths_tensor(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)


def check(q, k, v, dout, causal=False, lengths=None, scale=None, grads=True):
    kw = dict(causal=causal, kv_lengths=lengths_tensor(lengths), scale=scale)
    used = None if lengths is None else [max(0, min(n, k.shape[1])) for n in lengths]
    out, lse = qkr.attention(q, k, v, **kw)
    torch.cuda.synchronize()
    want = ref.forward(q, k, v, causal, used, scale)
    within(out, want["out"], want["bound"], "out")
    none = ~want["some"]
    assert (lse[none] == -math.inf).all() and (out.permute(0, 2, 1, 3)[none] == 0).all()
    assert ((lse.double() - want["lse"]).abs() <= want["lse_bound"])[~none].all(), "lse"
    if not grads:
        return out, lse
    got = qkr.attention_backward(dout, q, k, v, out, lse, **kw)
    torch.cuda.synchronize()
    grad = ref.backward(want, dout, out, q.dtype)
    for name, g in zip(("dq", "dk", "dv"), got):
        within(g, *grad[name], name)
    assert (got[0].permute(0, 2, 1, 3)[none] == 0).all()
    return out, lse, got


def tensors(seed, dtype, batch, sq, sk, h, hk, d, by=1.0):
    return (draw(seed, batch, sq, h, d, dtype=dtype, by=by), draw(seed + 1, batch, sk, hk, d, dtype=dtype, by=by),
            draw(seed + 2, batch, sk, hk, d, dtype=dtype), draw(seed + 3, batch, sq, h, d, dtype=dtype, by=1 / 16))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sq,sk", [(1, 1), (1, 65), (33, 31), (64, 64), (129, 200), (257, 1)])
def test_sizes(dtype, d, sq, sk):
    check(*tensors(sq * 1000 + sk, dtype, 2, sq, sk, 3, 3, d))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sq,sk", [(1, 1), (65, 65), (200, 130), (70, 333), (256, 256), (300, 20)])
def test_causal(dtype, d, sq, sk):
    """Square, more queries than keys (the first see none), more keys than queries."""
    check(*tensors(sq * 1000 + sk, dtype, 2, sq, sk, 2, 2, d), causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 256), ("fp16", 128)])
def test_key_lengths(dtype, d, causal):
    """None, one, a tile's edge and either side, all, and lengths out of range."""
    lengths = [0, 1, 63, 64, 65, 200, 1 << 30, -5]
    check(*tensors(7, dtype, len(lengths), 150, 200, 2, 2, d), causal=causal, lengths=lengths)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("h,hk", [(6, 2), (5, 1), (8, 8), (12, 4)])
def test_shared_key_heads(h, hk, causal):
    check(*tensors(h, "bf16", 2, 97, 161, h, hk, 64), causal=causal, lengths=[161, 90])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("by", [0.0, 6.0, 30.0])
def test_scores_from_flat_to_peaked(dtype, by):
    """Equal scores, and scores of hundreds, where one key takes all the weight."""
    check(*tensors(11, dtype, 1, 150, 300, 2, 2, 128, by=by))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rising_scores_move_the_maximum(dtype):
    """Every tile raises the running maximum of every row."""
    q, k, v, dout = tensors(12, dtype, 1, 70, 640, 1, 1, 64)
    k = (k.float() * 0.01 + torch.arange(640, device=DEV).view(1, -1, 1, 1) / 80).to(k.dtype)
    q = (q.float().abs() + 0.5).to(q.dtype)
    check(q, k, v, dout)


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 10])
def test_fp16_gradients_keep_their_precision(size):
    """Gradients far below and above 1 over 2000 keys: ds is far below fp16's
    normal range, or p (dp - delta) above it, unless it is scaled."""
    q, k, v, dout = tensors(13, "fp16", 1, 64, 2000, 1, 1, 64)
    check(q, k, v, (dout.float() * size).half())


def test_rows_of_very_different_gradients_keep_theirs_in_fp16():
    q, k, v, dout = tensors(14, "fp16", 1, 96, 500, 2, 2, 64)
    by = 2.0 ** torch.linspace(-10, 10, 96, device=DEV).view(1, -1, 1, 1)
    out, lse = qkr.attention(q, k, v)
    dout = (dout.float() * by).half()
    dq, _, _ = qkr.attention_backward(dout, q, k, v, out, lse)
    want = ref.forward(q, k, v)
    grad = ref.backward(want, dout, out, torch.float16)["dq"][0]
    # two roundings (ds, dq) at half a step each, statistically far below their
    # sum; and dq's own subnormals: half of 2^-24 in each of 64 elements
    off = (dq.double().permute(0, 2, 1, 3) - grad).norm(dim=3)
    assert (off <= 2 * 2.0 ** -11 * grad.norm(dim=3) + 64 ** 0.5 * 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_query_with_one_key_moves_neither(dtype, d):
    """Its probability is 1 whatever q and k are: their gradients are 0, not
    what two sums of dout . v differ by."""
    for sq, sk, h, hk, lengths, causal in ((1, 1, 3, 3, None, False), (70, 1, 4, 2, None, False),
                                           (40, 90, 2, 1, [1, 0, 1], False), (1, 1, 2, 2, None, True)):
        q, k, v, dout = tensors(35, dtype, 3, sq, sk, h, hk, d)
        _, _, (dq, dk, _) = check(q, k, v, dout, lengths=lengths, causal=causal)
        assert (dq == 0).all() and (dk == 0).all()
    q, k, v, dout = tensors(36, dtype, 1, 64, 64, 1, 1, d)
    dq = check(q, k, v, dout, causal=True)[2][0]
    assert (dq[:, 0] == 0).all()


@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_scale(scale):
    check(*tensors(15, "bf16", 1, 40, 70, 2, 2, 64), scale=scale)


def test_three_dimensions_are_one_sample():
    q, k, v, dout = tensors(16, "bf16", 1, 50, 70, 4, 2, 64)
    out, lse = qkr.attention(q, k, v)
    out3, lse3 = qkr.attention(q[0], k[0], v[0])
    assert out3.shape == (50, 4, 64) and lse3.shape == (4, 50)
    assert same_bits(out[0], out3) and same_bits(lse[0], lse3)
    g = qkr.attention_backward(dout, q, k, v, out, lse)
    g3 = qkr.attention_backward(dout[0], q[0], k[0], v[0], out3, lse3)
    assert all(same_bits(a[0], b) for a, b in zip(g, g3))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_fused_buffers_and_other_layouts_give_the_same_bits(d):
    """Slices of one QKV buffer, gradients into slices of another, heads-first
    storage, rows with gaps: all as the contiguous call, and nothing else of
    the buffers is written."""
    b, s, h = 2, 131, 3
    qkv = draw(17, b, s, 3, h, d)
    dout = draw(18, b, s, h, d)
    q, k, v = (qkv[:, :, i].contiguous() for i in range(3))
    out, lse = qkr.attention(q, k, v)
    want = qkr.attention_backward(dout, q, k, v, out, lse)

    views = [qkv[:, :, i] for i in range(3)]
    before = qkv.clone()
    out2, lse2 = qkr.attention(*views)
    assert same_bits(out, out2) and same_bits(lse, lse2)
    grads = torch.full((b, s, 3, h, d), 9.0, dtype=qkv.dtype, device=DEV)
    qkr.attention_backward(dout, *views, out, lse, dq=grads[:, :, 0], dk=grads[:, :, 1], dv=grads[:, :, 2])
    assert all(same_bits(grads[:, :, i].contiguous(), want[i]) for i in range(3))
    assert same_bits(qkv, before)

    first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v, dout, out)]
    out3, lse3 = qkr.attention(*first[:3])
    got = qkr.attention_backward(first[3], *first[:3], first[4], lse3)
    assert same_bits(out3.contiguous(), out) and all(same_bits(x, y) for x, y in zip(got, want))

    wide = torch.full((b, s + 2, h, d + 8), 7.0, dtype=qkv.dtype, device=DEV)
    target = wide[:, 1:-1, :, :d]
    qkr.attention(q, k, v, out=target)
    assert same_bits(target.contiguous(), out)
    assert (wide[:, :, :, d:] == 7).all() and (wide[:, (0, -1)] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("stride", [0, 8])
def test_one_token_of_any_stride(dtype, stride):
    """A single token's stride is never stepped over: 0 and less than a row give
    the contiguous call's bits, though kernels stage tiles of many rows."""
    for sq, sk, h, hk in ((1, 70, 4, 2), (70, 1, 2, 2), (1, 1, 3, 1)):
        x = tensors(37, dtype, 2, sq, sk, h, hk, 128)
        odd = [t.as_strided(t.shape, (t.stride(0), stride, *t.stride()[2:])) if t.shape[1] == 1 else t for t in x]
        out, lse = qkr.attention(*x[:3])
        out2, lse2 = qkr.attention(*odd[:3])
        assert same_bits(out, out2) and same_bits(lse, lse2)
        want = qkr.attention_backward(x[3], *x[:3], out, lse)
        got = qkr.attention_backward(odd[3], *odd[:3], out, lse)
        assert all(same_bits(a, b) for a, b in zip(got, want))


def test_expanded_heads_and_samples_as_inputs():
    """k and v of one sample and head, expanded without memory of their own."""
    q, _, _, dout = tensors(19, "bf16", 3, 40, 90, 4, 4, 64)
    k, v = (draw(20 + i, 1, 90, 1, 64).expand(3, 90, 4, 64) for i in range(2))
    out, lse = qkr.attention(q, k, v)
    out2, lse2 = qkr.attention(q, k.contiguous(), v.contiguous())
    assert same_bits(out, out2) and same_bits(lse, lse2)
    got = qkr.attention_backward(dout, q, k, v, out, lse)
    want = qkr.attention_backward(dout, q, k.contiguous(), v.contiguous(), out, lse)
    assert all(same_bits(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_padding_keys_are_not_read(dtype, bad):
    lengths = [0, 37, 64, 130]
    q, k, v, dout = tensors(21, dtype, 4, 70, 150, 2, 2, 64)
    for i, n in enumerate(lengths):
        k[i, n:] = bad
        v[i, n:] = -bad
    _, _, (dq, dk, dv) = check(q, k, v, dout, lengths=lengths)
    for i, n in enumerate(lengths):
        assert (dk[i, n:] == 0).all() and (dv[i, n:] == 0).all()


def test_no_queries_or_no_keys():
    q, k, v, dout = tensors(22, "bf16", 2, 5, 7, 2, 2, 64)
    none = q[:, :0]
    out, lse = qkr.attention(none, k, v)
    assert out.shape == none.shape and lse.shape == (2, 2, 0)
    dq, dk, dv = qkr.attention_backward(none, none, k, v, none, lse, dk=torch.ones_like(k),
                                        dv=torch.ones_like(v))
    assert (dk == 0).all() and (dv == 0).all()
    out, lse = qkr.attention(q, k[:, :0], v[:, :0])
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, _, _ = qkr.attention_backward(dout, q, k[:, :0], v[:, :0], out, lse, dq=torch.ones_like(q))
    assert (dq == 0).all()


def test_missing_tensors_without_tokens():
    """From C a tensor of no tokens may be NULL."""
    from diffusion_transformer_qk_amd import binding as b

    lib = b.load_library()
    q, _, _, dout = tensors(22, "fp16", 2, 5, 7, 2, 2, 64)
    args = b.AttnArgs(2, 5, 0, 2, 2, 64, 0, b.QKR_FP16, 0.125, None)
    t = lambda x: b._attn_tensor(x, "x")  # noqa: E731
    out, lse, dq = torch.ones_like(q), torch.ones((2, 2, 5), device=DEV), torch.ones_like(q)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.dit_attention(args, t(q), None, None, t(out), lse.data_ptr(), 0, 0, st) == 0
    assert lib.dit_attention_backward(args, t(dout), t(q), None, None, t(out), lse.data_ptr(), t(dq), None, None,
                                      ws.data_ptr(), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -math.inf).all() and (dq == 0).all()


@pytest.mark.parametrize("dtype,sq,sk,h,hk,causal", [
    ("bf16", 1, 4000, 8, 2, False), ("fp16", 60, 3000, 2, 1, False), ("fp16", 1500, 130, 4, 4, True),
    ("bf16", 900, 900, 3, 3, True)])
def test_workspaces_of_any_contents(dtype, sq, sk, h, hk, causal):
    """NaN patterns in the workspace, and one larger than needed, change nothing
    (calls that cut the keys, the queries, both, and neither)."""
    q, k, v, dout = tensors(34, dtype, 1, sq, sk, h, hk, 128)
    out, lse = qkr.attention(q, k, v, causal=causal)
    want = qkr.attention_backward(dout, q, k, v, out, lse, causal=causal)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    out2, lse2 = qkr.attention(q, k, v, causal=causal, workspace=ws)
    ws.fill_(255)
    got = qkr.attention_backward(dout, q, k, v, out, lse, causal=causal, workspace=ws)
    assert same_bits(out, out2) and same_bits(lse, lse2)
    assert all(same_bits(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("causal", [False, True])
def test_results_do_not_change_from_run_to_run(causal):
    q, k, v, dout = tensors(23, "fp16", 2, 700, 700, 4, 2, 128)
    out, lse = qkr.attention(q, k, v, causal=causal)
    grads = qkr.attention_backward(dout, q, k, v, out, lse, causal=causal)
    for _ in range(3):
        out2, lse2 = qkr.attention(q, k, v, causal=causal)
        grads2 = qkr.attention_backward(dout, q, k, v, out, lse, causal=causal)
        assert same_bits(out, out2) and same_bits(lse, lse2)
        assert all(same_bits(a, b) for a, b in zip(grads, grads2))


@pytest.mark.parametrize("batch,sq,sk,h,hk,lengths", [
    (1, 1, 5000, 10, 2, None), (3, 1, 3000, 4, 4, [0, 1, 2999]), (1, 7, 4100, 4, 1, None),
    (2, 20, 2500, 2, 2, [2500, 100])])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_few_queries_over_many_keys(dtype, d, batch, sq, sk, h, hk, lengths):
    check(*tensors(24, dtype, batch, sq, sk, h, hk, d), lengths=lengths)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
def test_head_dim_256_in_many_workgroups(dtype, causal):
    """More workgroups than CUs, where a wave keeps all columns of dk and dv
    (smaller calls share them between two)."""
    check(*tensors(38, dtype, 5, 300, 290, 16, 8, 256), causal=causal, lengths=[290, 129, 0, 64, 257])
    check(*tensors(39, dtype, 30, 3, 140, 16, 8, 256), causal=causal)


def test_few_queries_over_many_keys_causal():
    check(*tensors(25, "bf16", 1, 9, 3000, 4, 2, 128), causal=True)


def test_few_keys_under_many_queries():
    check(*tensors(26, "bf16", 1, 3000, 20, 2, 2, 128))


def test_a_longer_call():
    check(*tensors(27, "bf16", 1, 2000, 2000, 3, 3, 128))


def test_rows_past_4_gib():
    """Tokens 2^21 elements apart: the last lies beyond 2^32 bytes."""
    rows, stride = 1100, 1 << 21
    buf = torch.zeros(rows * stride, dtype=torch.bfloat16, device=DEV)
    x = [draw(28 + i, 1, rows, 1, 64) for i in range(4)]
    far = []
    for i, t in enumerate(x):
        view = buf.as_strided(t.shape, (rows * stride, stride, 64, 1), 64 * i)
        view.copy_(t)
        far.append(view)
    out, lse = qkr.attention(*far[:3])
    want, want_lse = qkr.attention(*x[:3])
    assert same_bits(out, want) and same_bits(lse, want_lse)
    o_far = buf.as_strided(out.shape, (rows * stride, stride, 64, 1), 64 * 4)
    qkr.attention(*far[:3], out=o_far)
    assert same_bits(o_far.contiguous(), want)
    grads = [buf.as_strided(out.shape, (rows * stride, stride, 64, 1), 64 * (5 + i)) for i in range(3)]
    qkr.attention_backward(far[3], *far[:3], o_far, lse, dq=grads[0], dk=grads[1], dv=grads[2])
    for a, b in zip(grads, qkr.attention_backward(x[3], *x[:3], want, want_lse)):
        assert same_bits(a.contiguous(), b)


def test_directional_differences():
    """The gradients against central differences of the 64-bit forward pass
    along random directions.  Differences are exact to about h^2; the bound is
    the sum of the gradients' elementwise bounds along the direction."""
    q, k, v, dout = tensors(31, "bf16", 1, 40, 60, 4, 2, 64)
    out, lse = qkr.attention(q, k, v, causal=True)
    got = qkr.attention_backward(dout, q, k, v, out, lse, causal=True)
    base = ref.forward(q, k, v, True)
    bounds = ref.backward(base, dout, out, q.dtype)
    do = dout.double().permute(0, 2, 1, 3)
    for i, (name, g) in enumerate(zip(("dq", "dk", "dv"), got)):
        t = torch.randn((q, k, v)[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64).to(DEV)
        h = 1e-5
        loss = []
        for sign in (1, -1):
            x = [y.double() for y in (q, k, v)]
            x[i] = x[i] + sign * h * t
            loss.append(float((ref_out(*x) * do).sum()))
        along = float((g.double() * t).sum())
        slack = float((bounds[name][1].permute(0, 2, 1, 3) * t.abs()).sum())
        assert abs((loss[0] - loss[1]) / (2 * h) - along) <= slack + 1e-6


def ref_out(q, k, v):
    """The causal forward pass in 64 bits, for values that need not be 16-bit."""
    group = q.shape[2] // k.shape[2]
    qh, kh, vh = (x.permute(0, 2, 1, 3).repeat_interleave(n, 1).contiguous()
                  for x, n in ((q, 1), (k, group), (v, group)))
    s = (qh @ kh.transpose(2, 3)) / math.sqrt(q.shape[3])
    seen = ref.visible(q.shape[1], k.shape[1], q.shape[0], True, None, q.device)
    return torch.softmax(s.masked_fill(~seen, -math.inf), 3) @ vh


def test_another_stream_and_graph_replays():
    """Captured forward and backward passes, two graphs that share nothing,
    replayed between eager calls with changed inputs."""
    q, k, v, dout = tensors(32, "fp16", 2, 90, 1500, 4, 2, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step():
        out, lse = qkr.attention(q, k, v)
        return (out, lse, *qkr.attention_backward(dout, q, k, v, out, lse))

    with torch.cuda.stream(st):
        step()
    by_hand = qkr.attention(q, k, v, stream=st)
    st.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept = step()
        graphs.append((g, kept))
    for i in range(4):
        for x in (q, k, v, dout):
            x.copy_(draw(100 + i, *x.shape, dtype="fp16"))
        want = step()
        for g, kept in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(same_bits(a, b) for a, b in zip(kept, want))
    assert torch.isfinite(by_hand[0]).all()


def test_an_infinity_reaches_no_pair_far_from_it_in_fp16():
    """Under causality an infinite dout row or v row of one position leaves the
    gradients of pairs 192 or more positions on the hidden side as they are,
    also where p (dp - delta) lies above fp16's range unless it is scaled."""
    s, far = 500, 192
    q, k, v, dout = tensors(44, "fp16", 1, s, s, 2, 2, 64)
    dout = (dout.float() * 2048).half()
    out, lse = qkr.attention(q, k, v, causal=True)
    for at in (0, 130):
        # query `at` has nothing to do with the keys behind it
        bad, zero = dout.clone(), dout.clone()
        bad[:, at], zero[:, at] = math.inf, 0
        _, dk, dv = qkr.attention_backward(bad, q, k, v, out, lse, causal=True)
        _, dk0, dv0 = qkr.attention_backward(zero, q, k, v, out, lse, causal=True)
        assert torch.isfinite(dk0).all()
        assert same_bits(dk[:, at + far:], dk0[:, at + far:]) and same_bits(dv[:, at + far:], dv0[:, at + far:])
    for at in (s - 1, s - 140):
        # key `at` has nothing to do with the queries before it
        bad, zero = v.clone(), v.clone()
        bad[:, at], zero[:, at] = -math.inf, 0
        dq = qkr.attention_backward(dout, q, k, bad, out, lse, causal=True)[0]
        dq0 = qkr.attention_backward(dout, q, k, zero, out, lse, causal=True)[0]
        assert torch.isfinite(dq0).all() and same_bits(dq[:, :at - far], dq0[:, :at - far])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 64), ("bf16", 128), ("bf16", 256)])
def test_a_hidden_value_reaches_192_positions_at_most(dtype, d, bad):
    """A NaN or infinity in a key or query takes part, with p = 0, in the rows
    of its workgroup and tile that causality hides from it, and in no others."""
    s, at, far = 700, 350, 192
    q, k, v, dout = tensors(45, dtype, 1, s, s, 2, 2, d)
    v[:, at], dout[:, at] = 0, 0            # so that fp16's scaling is the same
    out, lse = qkr.attention(q, k, v, causal=True)
    want = qkr.attention_backward(dout, q, k, v, out, lse, causal=True)
    for name in ("k", "v"):
        x = dict(k=k.clone(), v=v.clone())
        x[name][:, at] = bad
        out2, lse2 = qkr.attention(q, x["k"], x["v"], causal=True)
        dq = qkr.attention_backward(dout, q, x["k"], x["v"], out, lse, causal=True)[0]
        n = at - far + 1
        assert same_bits(out2[:, :n], out[:, :n]) and same_bits(lse2[:, :, :n].contiguous(), lse[:, :, :n].contiguous())
        assert same_bits(dq[:, :n], want[0][:, :n])
    for name in ("q", "dout"):
        x = dict(q=q.clone(), dout=dout.clone())
        x[name][:, at] = bad
        _, dk, dv = qkr.attention_backward(x["dout"], x["q"], k, v, out, lse, causal=True)
        n = at + far
        assert same_bits(dk[:, n:], want[1][:, n:]) and same_bits(dv[:, n:], want[2][:, n:])


@pytest.mark.parametrize("order", ["sbthd", "bshtd", "btshd", "bthsd", "thbsd"])
@pytest.mark.parametrize("hk", [4, 2])
def test_slices_of_buffers_of_any_order(order, hk):
    """q, k, v and out, and the gradients, as slices of one buffer whose
    dimensions (batch, sequence, tensor, head, element) stand in any order: the
    contiguous calls' bits, and every other element as it was."""
    b, s, h, d = 2, 100, 4, 64
    size = dict(b=b, s=s, t=5, h=h, d=d)

    def buffer(*values):
        """A buffer and its four slices, with these values in the first of them."""
        buf = torch.full([size[c] for c in order], 9.0, dtype=torch.bfloat16, device=DEV)
        whole = buf.permute([order.index(c) for c in "tbshd"])
        views = [whole[i, :, :, :n] for i, n in enumerate((h, hk, hk, h))]
        for view, value in zip(views, values):
            view.copy_(value)
        return buf, views

    q, k, v, dout = tensors(41, "bf16", b, s, s, h, hk, d)
    out, lse = qkr.attention(q, k, v)
    grads = qkr.attention_backward(dout, q, k, v, out, lse)

    buf, (vq, vk, vv, vo) = buffer(q, k, v)
    assert same_bits(qkr.attention(vq, vk, vv, out=vo)[1], lse)
    assert same_bits(buf, buffer(q, k, v, out)[0])
    for given in ((dout, q, k, v, out), (dout, vq, vk, vv, vo)):
        buf, (vdq, vdk, vdv, _) = buffer()
        qkr.attention_backward(*given, lse, dq=vdq, dk=vdk, dv=vdv)
        assert same_bits(buf, buffer(*grads)[0])


def test_gradients_over_the_buffer_they_were_cut_from_are_refused():
    """dq in the place of q, k's slice one element on, two gradients in one place."""
    buf = draw(42, 100, 2, 3, 4, 64)
    q, k, v = buf.permute(2, 1, 0, 3, 4).unbind(0)
    out, lse = qkr.attention(q, k, v)
    grads = torch.empty_like(buf).permute(2, 1, 0, 3, 4)
    for dq, dk in ((q, grads[1]), (grads[0], v), (grads[0], grads[0]), (grads[0], grads[2])):
        with pytest.raises(qkr.QkrError):
            qkr.attention_backward(out, q, k, v, out, lse, dq=dq, dk=dk, dv=grads[2])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_strides_of_a_dimension_of_one_do_not_count(dtype):
    """One token, one sample and one head of strides that nothing steps over
    (above the limits, negative in C, odd) give the contiguous call's bits."""
    for batch, sq, sk, h, hk in ((2, 1, 70, 4, 2), (1, 70, 1, 2, 2), (1, 1, 1, 1, 1), (1, 40, 70, 3, 1)):
        x = tensors(43, dtype, batch, sq, sk, h, hk, 128)
        out, lse = qkr.attention(*x[:3])
        want = qkr.attention_backward(x[3], *x[:3], out, lse)
        for stride in (5242880, 3, 1 << 39):
            odd = [t.as_strided(t.shape, [stride if n == 1 else st for n, st in zip(t.shape, t.stride())])
                   for t in (*x, torch.empty_like(out), *map(torch.empty_like, want))]
            out2, lse2 = qkr.attention(*odd[:3], out=odd[4])
            assert same_bits(out, out2.contiguous()) and same_bits(lse, lse2)
            got = qkr.attention_backward(odd[3], *odd[:3], odd[4], lse, dq=odd[5], dk=odd[6], dv=odd[7])
            assert all(same_bits(a, b.contiguous()) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128), ("bf16", 256)])
def test_keys_cut_for_dq_beside_whole_runs_of_queries(dtype, d):
    """Few causal queries over many keys of many heads: dq's keys are cut into
    runs that its masks leave uneven, dk's and dv's queries are not cut."""
    check(*tensors(46, dtype, 1, 100, 3000, 12, 12, d), causal=True)
    check(*tensors(47, dtype, 2, 130, 2100, 12, 6, d), causal=True, lengths=[2100, 1500])


@pytest.mark.parametrize("causal", [False, True])
def test_more_than_6000_tokens(causal):
    check(*tensors(48, "bf16", 1, 6200, 6200, 2, 1, 64), causal=causal)
