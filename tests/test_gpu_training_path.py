"""The operators of a DiT block's attention half in a row, as a training step
uses them: modulation -> QKV -> QK-norm + RoPE -> attention, and back.

The projection is left out (the modulated row is the QKV row), so that every
step is the library's.  End to end the results are compared in the 2-norm: at
most 16 roundings lie between the inputs and a gradient, each at most half a
step of the type, and a norm, softmax or rotation passes one on by at most a
factor of 2 at these inputs: 32 half steps.
"""
import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests.gpu_common import same_bits

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
B, S, H, D = 2, 173, 4, 64
WIDTH = 3 * H * D


def inputs(seed, dtype):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    angle = torch.arange(B * S)[:, None] % S * 100.0 ** (-torch.arange(D // 2) / (D // 2))
    angle = angle.repeat_interleave(2, 1)
    return dict(x=n(B * S, WIDTH).to(dtype).to(DEV), scale=(0.3 * n(B, WIDTH)).to(DEV),
                shift=(0.3 * n(B, WIDTH)).to(DEV), qg=(1 + 0.1 * n(D)).to(DEV), kg=(1 + 0.1 * n(D)).to(DEV),
                cos=angle.cos().float().to(DEV), sin=angle.sin().float().to(DEV),
                dout=(n(B, S, H, D) / 4).to(dtype).to(DEV),
                lengths=torch.tensor([S, 100], dtype=torch.int32, device=DEV))


def step(s):
    """One forward and backward pass; the gradients of x, scale, shift and gammas."""
    raw = qkr.fuse_scale_shift(s["x"], s["scale"], s["shift"])
    qkv = raw.clone()
    rope = dict(q_gamma=s["qg"], k_gamma=s["kg"], cos=s["cos"], sin=s["sin"])
    qkr.qknorm_rope_fused(qkv, **rope)
    q, k, v = qkv.view(B, S, 3, H, D).unbind(2)
    out, lse = qkr.attention(q, k, v, kv_lengths=s["lengths"])
    grad = torch.empty_like(qkv)
    dq, dk, dv = grad.view(B, S, 3, H, D).unbind(2)
    qkr.attention_backward(s["dout"], q, k, v, out, lse, kv_lengths=s["lengths"], dq=dq, dk=dk, dv=dv)
    dqg, dkg = qkr.qknorm_rope_backward(grad, raw, **rope)
    dx, dscale, dshift = qkr.fuse_scale_shift_backward(grad, s["x"], s["scale"])
    return dict(out=out, dx=dx, dscale=dscale, dshift=dshift, dqg=dqg, dkg=dkg)


def exact(s):
    """The same by automatic differentiation in 64 bits."""
    p = {n: s[n].double().requires_grad_() for n in ("x", "scale", "shift", "qg", "kg")}
    n = torch.nn.functional.layer_norm(p["x"], (WIDTH,), eps=1e-6).view(B, S, WIDTH)
    qkv = (n * (1 + p["scale"][:, None]) + p["shift"][:, None]).view(B, S, 3, H, D)
    cos, sin = (s[t].double().view(B, S, 1, D) for t in ("cos", "sin"))

    def turn(t, gamma):
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * gamma
        other = torch.stack([-t[..., 1::2], t[..., ::2]], -1).flatten(-2)
        return t * cos + other * sin

    q, k, v = (t.permute(0, 2, 1, 3).contiguous()
               for t in (turn(qkv[:, :, 0], p["qg"]), turn(qkv[:, :, 1], p["kg"]), qkv[:, :, 2]))
    w = (q @ k.transpose(2, 3).contiguous()) / D ** 0.5
    hidden = torch.arange(S, device=DEV)[None] >= s["lengths"][:, None]
    out = (torch.softmax(w.masked_fill(hidden[:, None, None], -torch.inf), 3) @ v).permute(0, 2, 1, 3)
    out.backward(s["dout"].double())
    return dict(out=out.detach(), dx=p["x"].grad, dscale=p["scale"].grad, dshift=p["shift"].grad,
                dqg=p["qg"].grad, dkg=p["kg"].grad)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_gradients_of_the_whole_path(dtype):
    s = inputs(1, dtype)
    got, want = step(s), exact(s)
    for name, w in want.items():
        rel = float((got[name].double().view_as(w) - w).norm() / w.norm())
        assert rel <= 32 * torch.finfo(dtype).eps / 2, (name, rel)


def test_the_whole_path_in_a_graph():
    """Captured once, replayed on new inputs between eager steps."""
    s = inputs(2, torch.bfloat16)
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(s)
    for i in range(4):
        for name, t in inputs(10 + i, torch.bfloat16).items():
            s[name].copy_(t)
        want = step(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(kept[n], want[n]) for n in want)
