"""The gated feed-forward projection and packed attention on buffers past 4 GiB:
the last rows, which lie beyond every 32-bit byte offset, against 64 bits with
the bounds of their own tests.
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests import attention_reference as ref
from tests import test_gpu_feed_forward as ff
from tests.test_gpu_attention_packed import slices
from tests.test_gpu_layer_norm import DEV, F, half_step, tail

pytestmark = pytest.mark.gpu


def rows_of(seed, shape, by=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * by)


@pytest.mark.parametrize("rows,hidden,inner", [(270001, 8192, 8), (140001, 8, 16384)])
def test_feed_forward(rows, hidden, inner):
    x, wg, wu = rows_of(1, (rows, hidden)), rows_of(2, (inner, hidden), hidden ** -0.5), rows_of(3, (inner, hidden), hidden ** -0.5)
    h, gate, up = qkr.gated_feed_forward(x, wg, wu, save=True)
    end = slice(rows - 64, rows)
    want, off = ff.exact(x[end], wg, wu, "silu")
    for got, w, e in zip((h, gate, up), want, off):
        assert bool(((got[end].double() - w).abs() <= half_step(got) * w.abs() + (1 + half_step(got)) * e + tail(got)).all())
    dh = rows_of(4, (rows, inner), 1 / 16)
    dx, dwg, dwu = qkr.gated_feed_forward_backward(dh, x, wg, wu, gate, up)

    def parts(r, c):
        """dgate and dup of these rows and columns, and what they may be off by."""
        a, b, d = gate[r, c].double(), up[r, c].double(), dh[r, c].double()
        y, slope = ff.act_of(a, "silu"), ff.slope_of(a, "silu")
        e = ff.act_error(a, "silu")
        da, db = d * b * slope, d * y
        return (da, half_step(x) * da.abs() + (d * b).abs() * 3 * e), (db, (half_step(x) + e) * db.abs())

    (da, e_a), (db, e_b) = parts(end, slice(None))
    g, u = wg.double(), wu.double()
    want = da @ g + db @ u
    off = e_a @ g.abs() + e_b @ u.abs() + (2 * inner + 16) * F * (da.abs() @ g.abs() + db.abs() @ u.abs())
    assert bool(((dx[end].double() - want).abs() <= half_step(x) * want.abs() + (1 + half_step(x)) * off + tail(x)).all())
    last, few = slice(inner - 8, inner), slice(hidden - 8, hidden)
    xs = x[:, few].double()
    for got, (d, e) in zip((dwg, dwu), parts(slice(None), last)):
        want = d.t() @ xs
        off = e.t() @ xs.abs() + (rows + 16) * F * (d.abs().t() @ xs.abs())
        got = got[last, few].double()
        assert bool(((got - want).abs() <= half_step(x) * want.abs() + (1 + half_step(x)) * off + tail(x)).all())


@pytest.mark.parametrize("causal", [False, True])
def test_packed_attention(causal, monkeypatch):
    """Sequences behind 150000 rows that are none's: 40 heads of 128 on a fused buffer."""
    lead, lengths, heads, d = 150000, [70, 33, 200], 40, 128
    tokens = lead + sum(lengths)
    qkv = rows_of(5, (tokens, 3, heads, d))
    q, k, v = qkv.unbind(1)
    offsets = torch.tensor([0, *lengths]).cumsum(0).add(lead).to(torch.int32).to(DEV)
    out, lse = qkr.attention_packed(q, k, v, offsets, causal=causal)
    dout = rows_of(6, (tokens, heads, d), 0.25)
    grad = torch.zeros_like(qkv)
    qkr.attention_packed_backward(dout, q, k, v, out, lse, offsets, causal=causal, dq=grad[:, 0], dk=grad[:, 1], dv=grad[:, 2])
    torch.cuda.synchronize()
    assert bool((out[:lead] == 0).all()) and bool((grad[:lead] == 0).all())
    monkeypatch.setattr(ref, "two_terms", lambda q, k: False)
    for rows in slices(lengths, lead):
        r = ref.forward(*(t[rows][None] for t in (q, k, v)), causal=causal)
        assert bool(((out[rows].double().permute(1, 0, 2) - r["out"][0]).abs() <= r["bound"][0]).all())
        assert bool(((lse[:, rows].double() - r["lse"][0]).abs() <= r["lse_bound"][0]).all())
        back = ref.backward(r, dout[rows][None], out[rows][None], torch.bfloat16)
        for i, n in enumerate(("dq", "dk", "dv")):
            want, bound = back[n]
            assert bool(((grad[rows, i].double().permute(1, 0, 2) - want[0]).abs() <= bound[0]).all()), n
