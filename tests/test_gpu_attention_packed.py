"""Attention of packed sequences and its backward pass on the GPU, sequence by
sequence against 64 bits with the bounds of attention_reference.py.

How many terms p is rounded in goes by the whole call here (up to 32 rows a key
head and sequence in the mean: two, forward; one in the backward pass), not by
the sequence, so the reference is told.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests import attention_reference as ref
from tests.gpu_common import same_bits

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
NAN = math.nan


def offsets_of(lengths, lead=0):
    return torch.tensor([0, *lengths]).cumsum(0).add(lead).to(torch.int32).to(DEV)


def inputs(seed, lengths, kv_lengths, heads, kv_heads, d, dtype, lead=0, rest=0, fill=NAN):
    """Packed tensors whose rows of no sequence hold `fill`."""
    g = torch.Generator().manual_seed(seed)

    def rows(lens, h, by=1.0):
        t = (torch.randn((lead + sum(lens) + rest, h, d), generator=g) * by).to(dtype)
        t[:lead] = fill
        t[lead + sum(lens):] = fill
        return t.to(DEV)

    return dict(q=rows(lengths, heads), k=rows(kv_lengths, kv_heads), v=rows(kv_lengths, kv_heads),
                dout=rows(lengths, heads, 0.25))


def slices(lengths, lead):
    at = lead
    for n in lengths:
        yield slice(at, at + n)
        at += n


def check(seed, lengths, kv_lengths, heads, kv_heads, d, dtype, causal, monkeypatch, lead=0, rest=0, backward=True):
    t = inputs(seed, lengths, kv_lengths or lengths, heads, kv_heads, d, dtype, lead, rest)
    offsets = offsets_of(lengths, lead)
    kw = dict(kv_offsets=offsets_of(kv_lengths, lead) if kv_lengths else None, causal=causal)
    out, lse = qkr.attention_packed(t["q"], t["k"], t["v"], offsets, **kw)
    given = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    qkr.attention_packed(t["q"], t["k"], t["v"], offsets, out=given[0], lse=given[1], **kw)
    torch.cuda.synchronize()
    end = lead + sum(lengths)
    none = torch.ones(out.shape[0], dtype=torch.bool, device=DEV)
    none[lead:end] = False
    assert bool((out[none] == 0).all()) and bool((lse[:, none] == -math.inf).all())
    assert bool((given[0][none] == 7).all()) and bool((given[1][:, none] == 7).all())
    assert same_bits(out[~none], given[0][~none]) and same_bits(lse[:, ~none].contiguous(), given[1][:, ~none].contiguous())
    grads = None
    if backward:
        o, s = out.clone(), lse.clone()
        o[none] = NAN
        s[:, none] = NAN
        a = (t["dout"], t["q"], t["k"], t["v"], o, s, offsets)
        grads = dict(zip(("dq", "dk", "dv"), qkr.attention_packed_backward(*a, **kw)))
        kept = {n: torch.full_like(t[n[1]], 7.0) for n in grads}
        qkr.attention_packed_backward(*a, **kw, **kept)
        torch.cuda.synchronize()
        for n, g in grads.items():
            part = slice(lead, lead + sum(lengths if n == "dq" else kv_lengths or lengths))
            for made, value in ((g, 0), (kept[n], 7)):
                assert bool((made[:part.start] == value).all()) and bool((made[part.stop:] == value).all()), n
            assert same_bits(g[part], kept[n][part])
    two = sum(lengths) + lead + rest
    monkeypatch.setattr(ref, "two_terms", lambda q, k: two * (heads // kv_heads) <= 32 * len(lengths))
    for rows, keys in zip(slices(lengths, lead), slices(kv_lengths or lengths, lead)):
        if rows.stop == rows.start:
            if grads:
                assert bool((grads["dk"][keys] == 0).all()) and bool((grads["dv"][keys] == 0).all())
            continue
        one = [t[n][s][None] for n, s in (("q", rows), ("k", keys), ("v", keys))]
        r = ref.forward(*one, causal=causal)
        got = out[rows].double().permute(1, 0, 2)
        assert bool(((got - r["out"][0]).abs() <= r["bound"][0]).all()), (rows, keys)
        s = lse[:, rows].double()
        some = r["some"][0]
        assert bool((s[~some] == -math.inf).all())
        assert bool(((s - r["lse"][0]).abs()[some] <= r["lse_bound"][0][some]).all())
        if not grads:
            continue
        with monkeypatch.context() as m:
            m.setattr(ref, "two_terms", lambda q, k: False)
            r = ref.forward(*one, causal=causal)
            for n, (want, bound) in ref.backward(r, t["dout"][rows][None], out[rows][None], dtype).items():
                g = grads[n][rows if n == "dq" else keys].double().permute(1, 0, 2)
                assert bool(((g - want[0]).abs() <= bound[0]).all()), (n, rows, keys)


LENGTHS = [
    ([1], None), ([17], None), ([5, 0, 3], None), ([130, 1, 64, 0, 33, 300], None), ([0, 0, 200], None), ([129, 0], None),
    ([128, 256, 128], None), ([40, 7, 0, 90], [1, 200, 50, 0]), ([33, 150], [400, 65]), ([0, 3], [70, 0]),
    ([200, 31, 32, 1], [64, 31, 33, 129]),
]


@pytest.mark.parametrize("lengths,kv", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,dtype", [(64, 4, 4, "bfloat16"), (128, 6, 2, "float16"), (256, 2, 2, "bfloat16"),
                                                    (64, 5, 1, "float16"), (128, 9, 9, "bfloat16"), (256, 3, 1, "float16")])
def test_sequences(lengths, kv, causal, d, heads, kv_heads, dtype, monkeypatch):
    lead = 3 if len(lengths) % 2 else 0
    check(1, lengths, kv, heads, kv_heads, d, getattr(torch, dtype), causal, monkeypatch, lead, rest=130 if d == 64 else 5)


@pytest.mark.parametrize("count", [63, 64, 65, 300, 5000])
@pytest.mark.parametrize("causal", [False, True])
def test_many_sequences(count, causal, monkeypatch):
    """More than the lanes of a wave, in one step of the search and in several."""
    g = torch.Generator().manual_seed(count)
    lengths = torch.randint(0, 4, (count,), generator=g).tolist()
    kv = torch.randint(0, 9, (count,), generator=g).tolist()
    t = inputs(2, lengths, kv, 2, 1, 64, torch.bfloat16, 1, 2)
    offsets, kv_offsets = offsets_of(lengths, 1), offsets_of(kv, 1)
    out, lse = qkr.attention_packed(t["q"], t["k"], t["v"], offsets, kv_offsets=kv_offsets, causal=causal)
    grads = qkr.attention_packed_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, offsets, kv_offsets=kv_offsets,
                                          causal=causal)
    # the same as padded samples: 3 queries (the last ones, under causality) and 8 keys each
    q, k, v, dout = (torch.zeros((count, n, h, 64), dtype=torch.bfloat16, device=DEV) for n, h in ((3, 2), (8, 1), (8, 1), (3, 2)))
    lens = torch.tensor(kv, dtype=torch.int32, device=DEV)
    want = torch.zeros_like(out, dtype=torch.float32), torch.full_like(lse, -math.inf)
    wants = [torch.zeros_like(x, dtype=torch.float32) for x in grads]
    a, b = 1, 1
    qf, kf, vf, df = (t[n].double() for n in ("q", "k", "v", "dout"))
    picks = set(range(0, count, max(1, count // 100))) | {count - 1}
    for i, (nq, nk) in enumerate(zip(lengths, kv)):
        if i in picks and nq and nk:
            for h in range(2):
                s = qf[a:a + nq, h] @ kf[b:b + nk, 0].t() / 8
                if causal:
                    s = s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(nk - nq + 1), -math.inf)
                p = torch.softmax(s, 1).nan_to_num(0.0)
                o = p @ vf[b:b + nk, 0]
                assert float((out[a:a + nq, h].double() - o).abs().max()) <= 2.0 ** -7 * 4
                ds = p * ((df[a:a + nq, h] @ vf[b:b + nk, 0].t()) - (df[a:a + nq, h] * o).sum(1, keepdim=True))
                dq = ds @ kf[b:b + nk, 0] / 8
                assert float((grads[0][a:a + nq, h].double() - dq).abs().max()) <= 2.0 ** -6
        elif i in picks:
            assert bool((out[a:a + nq] == 0).all()) and bool((lse[:, a:a + nq] == -math.inf).all())
            assert all(bool((x[b:b + nk] == 0).all()) for x in grads[1:]) or nq
        a, b = a + nq, b + nk
    assert bool(torch.isfinite(out.float()).all()) and all(bool(torch.isfinite(x.float()).all()) for x in grads)


@pytest.mark.parametrize("lengths,kv", [([1], [6000]), ([1, 1, 1], [3000, 0, 5001]), ([4, 1, 2, 0], [1, 7000, 900, 12]),
                                        ([300], [5000]), ([150, 40], [70, 6000])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_queries_over_many_keys(lengths, kv, d, monkeypatch):
    """Keys are cut into splits, of which short sequences leave most without a key."""
    for causal, dtype in ((False, torch.bfloat16), (True, torch.float16)):
        check(3, lengths, kv, 4, 2, d, dtype, causal, monkeypatch, lead=2, rest=1)
    assert qkr.attention_packed_workspace_size(len(lengths), sum(lengths), sum(kv), 4, 2, d) > 0


def test_equal_to_samples_of_one_length():
    """Packed samples of one length are the padded call's, bit for bit where both cut alike."""
    b, s, h, d = 3, 256, 24, 64
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((b, s, 3, h, d), generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = qkv.unbind(2)
    out, lse = qkr.attention(q, k, v, causal=True)
    pq, pk, pv = qkv.view(b * s, 3, h, d).unbind(1)
    got, plse = qkr.attention_packed(pq, pk, pv, offsets_of([s] * b), causal=True)
    assert same_bits(got.view(b, s, h, d), out)
    assert same_bits(plse.view(h, b, s).permute(1, 0, 2).contiguous(), lse)


def test_slices_of_fused_buffers(monkeypatch):
    lengths, h, d = [70, 0, 130], 3, 128
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((200, 3, h, d), generator=g).to(torch.float16).to(DEV)
    q, k, v = qkv.unbind(1)
    offsets = offsets_of(lengths)
    out, lse = qkr.attention_packed(q, k, v, offsets)
    dout = torch.randn((200, h, d), generator=g).to(torch.float16).to(DEV)
    want = qkr.attention_packed_backward(dout, *(x.contiguous() for x in (q, k, v)), out, lse, offsets)
    assert same_bits(out, qkr.attention_packed(*(x.contiguous() for x in (q, k, v)), offsets)[0])
    grads = torch.full_like(qkv, 5.0)
    dq, dk, dv = grads.unbind(1)
    qkr.attention_packed_backward(dout, q, k, v, out, lse, offsets, dq=dq, dk=dk, dv=dv)
    assert all(same_bits(a.contiguous(), b) for a, b in zip((dq, dk, dv), want))
    # heads first, and an out of that order
    qh = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    oh = torch.empty((h, 200, d), dtype=q.dtype, device=DEV).permute(1, 0, 2)
    assert same_bits(qkr.attention_packed(qh, k, v, offsets, out=oh, lse=torch.empty_like(lse))[0].contiguous(), out)


def test_infinities_and_nan_stay_in_their_sequences():
    lengths = [100, 37, 200]
    t = inputs(6, lengths, lengths, 4, 2, 64, torch.float16, fill=0.0)
    offsets = offsets_of(lengths)
    out, lse = qkr.attention_packed(t["q"], t["k"], t["v"], offsets)
    grads = qkr.attention_packed_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, offsets)
    for bad in (math.inf, NAN):
        b = {n: x.clone() for n, x in t.items()}
        for n in b:
            b[n][110] = bad
        o, s = qkr.attention_packed(b["q"], b["k"], b["v"], offsets)
        g = qkr.attention_packed_backward(b["dout"], b["q"], b["k"], b["v"], o, s, offsets)
        for got, want in zip((o, *g), (out, *grads)):
            assert same_bits(got[:100], want[:100]) and same_bits(got[137:], want[137:])


def test_nothing_to_attend():
    for rows, kv_rows, sequences in ((0, 0, 0), (0, 9, 2), (9, 0, 2), (4, 4, 0)):
        q = torch.ones((rows, 2, 64), dtype=torch.bfloat16, device=DEV)
        k = torch.ones((kv_rows, 2, 64), dtype=torch.bfloat16, device=DEV)
        offsets = torch.zeros(sequences + 1, dtype=torch.int32, device=DEV)
        kv = torch.zeros_like(offsets)
        offsets[1:], kv[1:] = rows, kv_rows
        out, lse = qkr.attention_packed(q, k, k, offsets, kv_offsets=kv)
        dq, dk, dv = qkr.attention_packed_backward(q, q, k, k, out, lse, offsets, kv_offsets=kv)
        for x in (out, dq, dk, dv):
            assert bool((x == 0).all())
        assert bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_streams_and_graphs(dtype):
    """The same bits on another stream, and from a graph replayed on other tensors
    and other lengths."""
    cases = [[100, 37, 200, 3], [0, 340, 0, 0], [85, 85, 85, 85], [1, 2, 300, 0], [340, 0, 0, 0]]
    s = inputs(7, [340], [340], 6, 2, 64, dtype)
    s["offsets"] = offsets_of(cases[0])

    def step():
        out, lse = qkr.attention_packed(s["q"], s["k"], s["v"], s["offsets"], causal=True)
        return [out, lse, *qkr.attention_packed_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["offsets"],
                                                         causal=True)]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        out, lse = qkr.attention_packed(s["q"], s["k"], s["v"], s["offsets"], causal=True, stream=stream)
        got = qkr.attention_packed_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["offsets"], causal=True,
                                            stream=stream)
        side.synchronize()
        assert all(same_bits(a, b) for a, b in zip((out, lse, *got), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i, lengths in enumerate(cases[1:]):
        for n, x in inputs(10 + i, [340], [340], 6, 2, 64, dtype).items():
            s[n].copy_(x)
        s["offsets"].copy_(offsets_of(lengths))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(kept, want))


def test_offsets_past_the_buffers_are_clamped():
    """Not what a program should pass, but nothing is read or written outside."""
    q = torch.randn((50, 2, 64), device=DEV).to(torch.bfloat16)
    for offsets in ([0, 20, 90], [-5, 10, 50], [0, 50, 1 << 30], [60, 70, 80], [-9, -3, 0]):
        o = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        c = o.clamp(0, 50)
        got, want = (qkr.attention_packed(q, q, q, x, causal=True) for x in (o, c))
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
        for a, b in zip(*(qkr.attention_packed_backward(q, q, q, q, *want, x, causal=True) for x in (o, c))):
            assert same_bits(a, b)
