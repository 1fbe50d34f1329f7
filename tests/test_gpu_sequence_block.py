"""The halves of a block over packed sequences in one run, as they are used:
RMS norm with the residual, packed attention on the fused buffer that it wrote,
RMS norm, gated feed-forward, and back; and the step in 8 bits.  Each operator
is held to its bounds against 64 bits on what the one before it gave, and a
captured run to the eager one.  (What a model has between them, projections, is
views and copies here.)
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests import attention_reference as ref
from tests import test_gpu_feed_forward as ff
from tests import test_gpu_rms_norm as rms
from tests.gpu_common import same_bits
from tests.test_gpu_attention_packed import offsets_of, slices
from tests.test_gpu_layer_norm import DEV, TYPES, gen, rows_of

pytestmark = pytest.mark.gpu

HEADS, D = 4, 64
WIDTH = 3 * HEADS * D
LENGTHS, REST = [70, 1, 0, 129, 33], 5
TOKENS = sum(LENGTHS) + REST


def parameters(dtype):
    g = gen(20)
    made = {n: rms.weight_of(21 + i, WIDTH, "fp32") for i, n in enumerate(("w1", "w2"))}
    for n in ("w_gate", "w_up"):
        made[n] = (torch.randn((WIDTH, WIDTH), generator=g) / WIDTH ** 0.5).to(TYPES[dtype]).to(DEV)
    return made


def run(t, p, offsets, causal):
    """Everything that the block computes, by name."""
    f = dict(t)
    f["n1"], f["s1"] = qkr.rms_norm(t["x"], p["w1"], residual=t["r"])
    f["q"], f["k"], f["v"] = f["n1"].view(TOKENS, 3, HEADS, D).unbind(1)
    f["out"], f["lse"] = qkr.attention_packed(f["q"], f["k"], f["v"], offsets, causal=causal)
    f["a"] = f["out"].view(TOKENS, -1).repeat(1, 3)
    f["n2"], f["s2"] = qkr.rms_norm(f["a"], p["w2"], residual=f["s1"])
    f["h"], f["gate"], f["up"] = qkr.gated_feed_forward(f["n2"], p["w_gate"], p["w_up"], save=True)
    # the output is s2 + h: its gradient reaches both
    f["dn2"], f["dw_gate"], f["dw_up"] = qkr.gated_feed_forward_backward(
        t["dy"], f["n2"], p["w_gate"], p["w_up"], f["gate"], f["up"])
    f["ds2"], f["dw2"] = qkr.rms_norm_backward(f["dn2"], f["s2"], p["w2"], dsum=t["dy"])
    f["dout"] = f["ds2"].view(TOKENS, 3, HEADS, D).sum(1)
    dqkv = torch.zeros_like(f["n1"]).view(TOKENS, 3, HEADS, D)
    qkr.attention_packed_backward(f["dout"], f["q"], f["k"], f["v"], f["out"], f["lse"], offsets, causal=causal,
                                  dq=dqkv[:, 0], dk=dqkv[:, 1], dv=dqkv[:, 2])
    f["dn1"] = dqkv.view(TOKENS, WIDTH)
    f["ds1"], f["dw1"] = qkr.rms_norm_backward(f["dn1"], f["s1"], p["w1"], dsum=f["ds2"])
    return f


def inputs(seed, dtype):
    return dict(x=rows_of(seed, TOKENS, WIDTH, dtype), r=rows_of(seed + 1, TOKENS, WIDTH, dtype),
                dy=rows_of(seed + 2, TOKENS, WIDTH, dtype, 1 / 16))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_block(dtype, causal, monkeypatch):
    p, offsets = parameters(dtype), offsets_of(LENGTHS)
    f = run(inputs(30, dtype), p, offsets, causal)
    torch.cuda.synchronize()
    for x, r, w in (("x", "r", "w1"), ("a", "s1", "w2")):
        rms.check_forward(f[x], f[r], p[w])
    ff.check_forward(f["n2"], p["w_gate"], p["w_up"], "silu")
    t = dict(dh=f["dy"], x=f["n2"], gate=f["gate"], up=f["up"], w_gate=p["w_gate"], w_up=p["w_up"])
    grads = ff.check_backward(t, "silu")
    for n, name in (("dx", "dn2"), ("dw_gate", "dw_gate"), ("dw_up", "dw_up")):
        assert same_bits(grads[n], f[name]), n
    for dy, s, ds, w, dx in (("dn2", "s2", "dy", "w2", "ds2"), ("dn1", "s1", "ds2", "w1", "ds1")):
        got, dw = rms.check_backward(f[dy], f[s], f[ds], p[w])
        assert same_bits(got, f[dx]) and same_bits(dw, f["d" + w])
    # both passes round p once: there are more than 32 rows a sequence in the mean
    monkeypatch.setattr(ref, "two_terms", lambda q, k: False)
    given = f["dn1"].view(TOKENS, 3, HEADS, D)
    for rows in slices(LENGTHS, 0):
        if rows.stop == rows.start:
            continue
        one = [f[n][rows][None] for n in "qkv"]
        r = ref.forward(*one, causal=causal)
        assert bool(((f["out"][rows].double().permute(1, 0, 2) - r["out"][0]).abs() <= r["bound"][0]).all())
        back = ref.backward(r, f["dout"][rows][None], f["out"][rows][None], TYPES[dtype])
        for i, n in enumerate(("dq", "dk", "dv")):
            want, bound = back[n]
            assert bool(((given[rows, i].double().permute(1, 0, 2) - want[0]).abs() <= bound[0]).all()), n
    assert bool((f["out"][-REST:] == 0).all()) and bool((given[-REST:] == 0).all())


def quantised(p):
    return {n: ff.in_8_bits(p[n]) for n in ("w_gate", "w_up")}


def run_8_bits(t, p, weights):
    f = {}
    f["n"], f["scales"], f["s"] = qkr.rms_norm_fp8(t["x"], p["w1"], residual=t["r"])
    f["h"] = qkr.gated_feed_forward(f["n"], weights["w_gate"][0], weights["w_up"][0], x_scale=f["scales"],
                                    gate_scale=weights["w_gate"][1], up_scale=weights["w_up"][1])
    return f


@pytest.mark.parametrize("rows", [1, 8, TOKENS])
def test_step_in_8_bits(rows):
    p = parameters("bf16")
    weights = quantised(p)
    t = {n: v[:rows] for n, v in inputs(40, "bf16").items()}
    f = run_8_bits(t, p, weights)
    rms.check_forward(t["x"], t["r"], p["w1"])
    ff.check_forward(f["n"], weights["w_gate"][0], weights["w_up"][0], "silu",
                     (f["scales"], weights["w_gate"][1], weights["w_up"][1]), torch.bfloat16)
    # what the norm gives is the 16-bit norm but for the 8 bits: half a step of e4m3 (of 2^-6 below it) and the other's
    n = qkr.rms_norm(t["x"], p["w1"], residual=t["r"])[0].double()
    got, scale = f["n"].double() * f["scales"].double()[:, None], f["scales"].double()[:, None]
    off = torch.maximum(got.abs() * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -4) + n.abs() * 2.0 ** -8 * 1.01
    assert bool(((got - n).abs() <= off + n.abs() * 4 * rms.C).all())


def test_captured_runs():
    """Two graphs, replayed in turn with eager calls between them."""
    p, offsets = parameters("bf16"), offsets_of(LENGTHS)
    weights = quantised(p)
    t = inputs(50, "bf16")
    small = {n: v[:8].clone() for n, v in t.items()}
    run(t, p, offsets, True), run_8_bits(small, p, weights)
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: run(t, p, offsets, True), lambda: run_8_bits(small, p, weights)):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            found = call()
        graphs.append((graph, found, call))
    for turn in range(4):
        new = inputs(60 + turn, "bf16")
        for n in t:
            t[n].copy_(new[n])
            small[n].copy_(new[n][:8])
        wants = [{n: v.clone() for n, v in call().items()} for _, _, call in graphs]
        for (graph, found, _), want in zip(graphs[::1 if turn % 2 else -1], wants[::1 if turn % 2 else -1]):
            graph.replay()
            torch.cuda.synchronize()
            for n, v in want.items():
                assert same_bits(found[n].contiguous(), v.contiguous()), (turn, n)
