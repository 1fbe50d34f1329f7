"""Attention and its gradients in 64 bits, with elementwise error bounds for a
16-bit implementation (no test functions here).

The bounds follow from the arithmetic.  With u half a step of the 16-bit type
(relative) and f = 2^-24 of fp32:
  scores: D products summed in fp32: |error| <= e_s = (D + 4) f scale sum|q k|
    (plus the rounding of the exponent's argument, 2 f |s|), so p is off by a
    relative e_p = 2 e_s + (keys + 16) f (numerator, denominator, exp2);
  p is rounded to 16 bits before it is multiplied (u), the output once (u);
  fp16 products of p below its normal range add 2^-24 / 2^7 of the largest p.
Calls of up to 32 query rows a key head round p and ds in two terms: u^2 in the
place of u there (two_terms).
Backward, p comes from lse (its rounding: 2 f |lse|), ds = p (dp - delta) is
rounded to 16 bits, dp is off by (D + 4) f sum|dout v| and delta by the
rounding of out (u sum|dout out|, out being a 16-bit input) and its own sum.
Values below 2^-126 are rounded to zero (fp32's smallest normal number, and
bf16's): each p by less than TINY, each ds by less than TINY (1 + |dp - delta|).
"""
import math

import torch

F32 = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def subnormal_step(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _heads(x, group=1):
    return x.double().permute(0, 2, 1, 3).repeat_interleave(group, 1).contiguous()


def visible(q_tokens, kv_tokens, batch, causal, lengths, device):
    """[batch, 1, q, k] truth values."""
    j = torch.arange(kv_tokens, device=device)
    seen = torch.ones((batch, 1, q_tokens, kv_tokens), dtype=torch.bool, device=device)
    if lengths is not None:
        seen &= (j[None] < torch.as_tensor(lengths, device=device)[:, None])[:, None, None]
    if causal:
        seen &= j[None] <= torch.arange(q_tokens, device=device)[:, None] + kv_tokens - q_tokens
    return seen


def clean(x, lengths):
    """x with the rows past each sample's length set to zero (they may hold anything)."""
    if lengths is None:
        return x
    keep = torch.arange(x.shape[1], device=x.device)[None] < torch.as_tensor(
        lengths, device=x.device)[:, None]
    return torch.where(keep[:, :, None, None], x, torch.zeros_like(x))


def two_terms(q, k):
    return q.shape[1] * q.shape[2] // k.shape[2] <= 32


def forward(q, k, v, causal=False, lengths=None, scale=None):
    """dict of out, lse, p (64 bits, heads first) and the bounds of out and lse."""
    group = q.shape[2] // k.shape[2]
    d, keys = q.shape[3], k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    qh, kh, vh = _heads(q), _heads(clean(k, lengths), group), _heads(clean(v, lengths), group)
    seen = visible(q.shape[1], keys, q.shape[0], causal, lengths, q.device)
    s = (qh @ kh.transpose(2, 3)) * scale
    s = torch.where(seen, s, torch.tensor(-math.inf, dtype=torch.float64, device=q.device))
    some = seen.any(3, keepdim=True).expand(*s.shape[:3], 1)
    lse = torch.logsumexp(s, 3, keepdim=True) if keys else torch.full_like(some, -math.inf,
                                                                          dtype=torch.float64)
    p = torch.where(some & seen, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))),
                    torch.zeros_like(s))
    out = p @ vh
    u, f = half_step(q.dtype), F32
    u_p = u * u if two_terms(q, k) else u
    mag = (qh.abs() @ kh.abs().transpose(2, 3)) * scale
    e_s = ((d + 4) * f * mag + 2 * f * mag).amax(3, keepdim=True) if keys else torch.zeros_like(lse)
    e_p = 2 * e_s + (keys + 16) * f
    pv = p @ vh.abs()
    bound = (u * out.abs() + (1 + u) * (u_p + e_p) * pv + subnormal_step(q.dtype)
             + 2 * TINY * vh.abs().sum(2, keepdim=True))
    if q.dtype == torch.float16:
        bound = bound + 2.0 ** -31 * vh.abs().sum(2, keepdim=True) * p.amax(3, keepdim=True) if keys else bound
    lse_bound = e_s + (keys + 16) * f + 4 * f * torch.where(some, lse.abs(), torch.zeros_like(lse))
    return dict(out=out, lse=lse[..., 0], p=p, some=some[..., 0], e_p=e_p, scale=scale, bound=bound,
                lse_bound=lse_bound[..., 0], q=qh, k=kh, v=vh, group=group,
                u_p=u_p)


def backward(ref, dout, out16, dtype):
    """dq, dk, dv (heads first) of forward()'s dict and their bounds.  out16:
    the 16-bit out that the implementation is given."""
    q, k, v, p, scale, group = (ref[n] for n in ("q", "k", "v", "p", "scale", "group"))
    u, f, d = half_step(dtype), F32, q.shape[3]
    do = _heads(dout)
    o16 = _heads(out16)
    dp = do @ v.transpose(2, 3)
    delta = (do * ref["out"]).sum(3, keepdim=True)
    ds = p * (dp - delta)
    e_dp = (d + 4) * f * (do.abs() @ v.abs().transpose(2, 3))
    # what the given out differs by from the exact one, and the fp32 sum
    e_delta = (do * (o16 - ref["out"])).sum(3, keepdim=True).abs() + (d + 4) * f * (
        do.abs() * o16.abs()).sum(3, keepdim=True)
    e_p = ref["e_p"] + 4 * f * torch.where(ref["some"], ref["lse"].abs(),
                                           torch.zeros_like(ref["lse"]))[..., None]
    u_p = ref["u_p"]
    e_ds = (u_p + e_p) * ds.abs() + (1 + u) * p * (e_dp + e_delta) + TINY * (1 + (dp - delta).abs())
    keys, rows = k.shape[2], q.shape[2] * group
    small = torch.zeros((), dtype=torch.float64, device=q.device)
    if dtype == torch.float16 and p.numel():
        # operands below fp16's normal range: 2^-24 / 2^15 of the bound on |dp - delta|
        worst = 2 * do.norm(dim=3).amax() * v.norm(dim=3).amax() * 4
        small = worst * 2.0 ** -39

    def joined(x):
        b, h, n, e = x.shape
        return x.view(b, h // group, group, n, e).sum(2)

    tail = subnormal_step(dtype)
    got = {}
    dq = scale * (ds @ k)
    got["dq"] = dq, (u * dq.abs() + scale * (e_ds @ k.abs()) * (1 + u) + keys * f * scale * (ds.abs() @ k.abs())
                     + scale * small * k.abs().sum(2, keepdim=True) + tail)
    dk = joined(scale * (ds.transpose(2, 3) @ q))
    got["dk"] = dk, (u * dk.abs() + (1 + u) * joined(scale * (e_ds.transpose(2, 3) @ q.abs()))
                     + rows * f * joined(scale * (ds.abs().transpose(2, 3) @ q.abs()))
                     + joined(scale * small * q.abs().sum(2, keepdim=True).expand_as(k)) + tail)
    dv = joined(p.transpose(2, 3) @ do)
    e_pr = (u_p + e_p) * p + 2 * TINY
    got["dv"] = dv, (u * dv.abs() + (1 + u) * joined(e_pr.transpose(2, 3) @ do.abs())
                     + rows * f * joined(p.transpose(2, 3) @ do.abs())
                     + joined(2.0 ** -39 * do.abs().sum(2, keepdim=True).expand_as(v)) + tail)
    return got
