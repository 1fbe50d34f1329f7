"""Cases of the training path of a DiT block's attention half: attention
forward and backward, layer norm forward and backward, and the backward pass
of QK-norm + RoPE, each with its plain form in elementary torch operations.

Tensors are laid out as a program that uses the library holds them: q, k and v
are views of one fused QKV buffer where the case says so, gradients arrive and
leave in the activations' type, the gradients of norm weights in fp32.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def attend(name, grad, dtype, batch, q_tokens, kv_tokens, heads, kv_heads, head_dim, causal=False,
           lengths="", fused=False):
    """lengths: keys in use per sample ("" for all of them); fused: q, k and v
    are slices of one [batch, tokens, 3 * heads * head_dim] buffer."""
    return dict(name=name, op="attend", grad=grad, dtype=dtype, batch=batch, q_tokens=q_tokens,
                kv_tokens=kv_tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                causal=causal, lengths=lengths, fused=fused)


def norm(name, grad, dtype, param, rows, hidden, batches=0):
    """batches: 0 for an affine layer norm (one weight row for all rows), else
    the number of modulation rows (weight 1 + scale, one row per sample)."""
    return dict(name=name, op="norm", grad=grad, dtype=dtype, param=param, rows=rows,
                hidden=hidden, batches=batches)


def qk(name, dtype, tokens, heads, head_dim, style="interleaved", layout="shared", table="fp32",
       fused=True):
    return dict(name=name, op="qk", grad=True, dtype=dtype, tokens=tokens, heads=heads,
                head_dim=head_dim, style=style, layout=layout, table=table, fused=fused)


def listed():
    return [
        # self-attention of one of eight head shards of a 21x30x52 video latent: the long end
        attend("attend_video_shard", False, "bf16", 1, 32760, 32760, 5, 5, 128, fused=True),
        # cross-attention of a token shard to two padded prompts
        attend("attend_padded_text", False, "fp16", 2, 4095, 512, 40, 40, 128, lengths="512,77"),
        # one query token over a long sequence whose key heads are shared: latency and split work
        attend("attend_one_token", False, "bf16", 1, 1, 32760, 40, 8, 128, lengths="32749"),
        # the backward pass of the first case
        attend("attend_grad_video_shard", True, "bf16", 1, 32760, 32760, 5, 5, 128, fused=True),
        # 512 text and 64x64 image tokens, 48 heads: an ordinary training call
        attend("attend_grad_image", True, "bf16", 1, 4608, 4608, 48, 48, 128, fused=True),
        # a padded causal batch with shared key heads, an odd length, one sample without any key
        attend("attend_grad_causal_padded", True, "fp16", 3, 1021, 1021, 12, 4, 64, causal=True,
               lengths="1021,0,640"),
        # 256 tokens of 24 heads of 64: a small call, where launches count
        attend("attend_grad_small", True, "bf16", 1, 256, 256, 24, 24, 64, fused=True),
        # the affine layer norm in front of a video block's cross-attention
        norm("norm_affine_video", False, "bf16", "fp32", 32760, 5120),
        # the gradient of the modulated layer norm of two guidance branches of that block
        norm("norm_grad_modulated_video", True, "bf16", "fp32", 65520, 5120, batches=2),
        # a prompt's tokens at an odd width
        norm("norm_grad_affine_text", True, "fp16", "fp16", 77, 1000),
        # the gradient of the QK pass over the whole fused video buffer
        qk("qk_grad_video", "bf16", 32760, 40, 128),
        # a small call with a table row per head, the other pairing, 16-bit tables
        qk("qk_grad_small", "fp16", 255, 24, 64, style="rotate_half", layout="per_head",
           table="bf16", fused=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend_grad", "attend_grad", "norm", "norm_grad", "qk"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind.startswith("attend"):
        head_dim = rng.choice([64, 128, 256])
        batch = rng.randint(1, 3)
        kv_heads = rng.randint(1, 10)
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        fused = heads == kv_heads and rng.random() < 0.5
        q_tokens = _log(rng, 1, 6000)
        kv_tokens = q_tokens if fused or rng.random() < 0.4 else _log(rng, 1, 6000)
        lengths = ""
        if rng.random() < 0.5:
            lengths = ",".join(str(rng.randint(0, kv_tokens)) for _ in range(batch))
        c = attend("", kind == "attend_grad", dtype, batch, q_tokens, kv_tokens, heads, kv_heads,
                   head_dim, rng.random() < 0.3, lengths, fused)
    elif kind.startswith("norm"):
        hidden = 8 * _log(rng, 1, 1024)
        batches = rng.choice([0, 0, 1, 2, 3]) if kind == "norm_grad" else 0
        rows = max(1, batches) * _log(rng, 1, 20000)
        c = norm("", kind == "norm_grad", dtype, rng.choice(["fp32", "bf16", "fp16"]), rows, hidden,
                 batches)
    else:
        c = qk("", dtype, _log(rng, 1, 30000), rng.randint(1, 40), rng.choice([64, 128, 256]),
               rng.choice(["interleaved", "rotate_half"]), rng.choice(["shared", "shared", "per_head"]),
               rng.choice(["fp32", "bf16"]), rng.random() < 0.6)
        while c["tokens"] * c["heads"] * c["head_dim"] > 32760 * 40 * 128:
            c["tokens"] = (c["tokens"] + 1) // 2
    del c["name"]
    return c


def _lengths(case):
    if not case["lengths"]:
        return [case["kv_tokens"]] * case["batch"]
    return [int(n) for n in case["lengths"].split(",")]


def _visible_pairs(case):
    """(query, key) pairs of one head that the masks leave, over all samples."""
    total = 0
    sq, sk = case["q_tokens"], case["kv_tokens"]
    for n in _lengths(case):
        if not case["causal"]:
            total += sq * n
            continue
        # query i sees min(n, i + 1 + sk - sq) keys, none where that is negative
        first = min(max(0, sq - sk), sq)              # queries before this one see nothing
        full = min(max(first, n - 1 + sq - sk), sq)   # queries from this one on see all n
        a, z = first + 1 + sk - sq, full - 1 + 1 + sk - sq
        total += (a + z) * (full - first) // 2 + (sq - full) * n
    return total


def work(case):
    if case["op"] == "attend":
        d, h, hk = case["head_dim"], case["heads"], case["kv_heads"]
        q = case["batch"] * case["q_tokens"] * h * d * 2
        kv = sum(_lengths(case)) * hk * d * 2
        whole_kv = case["batch"] * case["kv_tokens"] * hk * d * 2
        lse = case["batch"] * h * case["q_tokens"] * 4
        pairs = _visible_pairs(case) * h
        if case["grad"]:   # reads q, out, dout, k, v, lse; writes dq, dk, dv
            return {"bytes": 4 * q + 2 * kv + lse + 2 * whole_kv, "flops": 10 * d * pairs}
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * pairs}
    if case["op"] == "norm":
        x = case["rows"] * case["hidden"] * 2
        params = max(1, case["batches"]) * case["hidden"]
        size = 4 if case["param"] == "fp32" else 2
        if case["grad"]:   # reads x, dy, the weight; writes dx and two fp32 rows a sample
            return {"bytes": 3 * x + params * (size + 8), "flops": 14 * case["rows"] * case["hidden"]}
        return {"bytes": 2 * x + 2 * params * size, "flops": 7 * case["rows"] * case["hidden"]}
    n = case["tokens"] * case["heads"] * case["head_dim"]
    rows = case["tokens"] * (case["heads"] if case["layout"] == "per_head" else 1)
    table = 2 * rows * case["head_dim"] * (4 if case["table"] == "fp32" else 2)
    return {"bytes": 2 * 3 * n * 2 + table + 4 * case["head_dim"] * 4, "flops": 2 * 14 * n}


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _token_scales(g, rows, spread=10.0):
    u = torch.rand((rows, 1), generator=g, device="cuda")
    return torch.exp((2 * u - 1) * math.log(spread))


def prepare(case, seed):
    g = _generator(seed)
    t = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "attend":
        b, sq, sk = case["batch"], case["q_tokens"], case["kv_tokens"]
        h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
        if case["fused"]:
            # normalised and rotated q and k, as the QK pass leaves them, and v
            qkv = _normal(g, b, sq, 3, h, d).to(t)
            s["q"], s["k"], s["v"] = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
        else:
            s["q"] = _normal(g, b, sq, h, d).to(t)
            s["k"] = _normal(g, b, sk, hk, d).to(t)
            s["v"] = _normal(g, b, sk, hk, d).to(t)
        s["kv_lengths"] = (torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
                           if case["lengths"] else None)
        if case["grad"]:
            s["out"], s["lse"] = _attention(s)
            s["dout"] = (_normal(g, b, sq, h, d) * _token_scales(g, b * sq, 4.0).view(b, sq, 1, 1)
                         / 16).to(t)
            if case["fused"]:   # the gradients land in the slices of one buffer too
                grads = torch.empty((b, sq, 3, h, d), dtype=t, device="cuda")
                s["dq"], s["dk"], s["dv"] = grads[:, :, 0], grads[:, :, 1], grads[:, :, 2]
            else:
                s["dq"] = s["dk"] = s["dv"] = None
    elif case["op"] == "norm":
        rows, c, p = case["rows"], case["hidden"], TYPES[case["param"]]
        s["x"] = ((_normal(g, rows, c) + 0.5 * _normal(g, c)) * _token_scales(g, rows)).to(t)
        if case["batches"]:
            s["weight"] = (0.5 * _normal(g, case["batches"], c)).to(p)      # the scale
        else:
            s["weight"] = (1 + 0.1 * _normal(g, c)).to(p)
            s["bias"] = (0.1 * _normal(g, c)).to(p)
        if case["grad"]:
            s["dy"] = (_normal(g, rows, c) * _token_scales(g, rows, 4.0) / 16).to(t)
    else:
        n, h, d = case["tokens"], case["heads"], case["head_dim"]
        scale, slope = _token_scales(g, n), _token_scales(g, n, 4.0) / 16
        if case["fused"]:
            s["x"] = (_normal(g, n, 3 * h * d) * scale).to(t)
            s["do"] = (_normal(g, n, 3 * h * d) * slope).to(t)
            s["dx"] = torch.zeros_like(s["x"])     # its third slice belongs to v's gradient
        else:
            for k in ("q", "k"):
                s["x" + k] = (_normal(g, n, h * d) * scale).to(t).view(n, h, d)
                s["do" + k] = (_normal(g, n, h * d) * slope).to(t).view(n, h, d)
        s["q_gamma"], s["k_gamma"] = 1 + 0.1 * _normal(g, d), 1 + 0.1 * _normal(g, d)
        rows = n * (h if case["layout"] == "per_head" else 1)
        at = torch.arange(rows, device="cuda") // (h if case["layout"] == "per_head" else 1)
        start = torch.randint(0, 1000, (1,), generator=g, device="cuda")
        freq = 10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))
        angle = (at + start).double()[:, None] * freq
        angle = (angle.repeat_interleave(2, 1) if case["style"] == "interleaved"
                 else torch.cat([angle, angle], 1))
        shape = (n, h, d) if case["layout"] == "per_head" else (n, d)
        s["cos"] = angle.cos().to(TYPES[case["table"]]).view(shape)
        s["sin"] = angle.sin().to(TYPES[case["table"]]).view(shape)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _own(s)
    if case["op"] == "attend":
        if case["grad"]:
            return _attention_backward(s)
        out, lse = _attention(s)
        return {"out": out, "lse": lse}
    if case["op"] == "norm":
        return _layer_norm_backward(s) if case["grad"] else {"y": _layer_norm(s)}
    return _qknorm_rope_backward(s)


def _own(s):
    import diffusion_transformer_qk_amd as qkr

    case = s["case"]
    if case["op"] == "attend":
        kw = dict(causal=case["causal"], kv_lengths=s["kv_lengths"])
        if case["grad"]:
            dq, dk, dv = qkr.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"],
                                                s["lse"], dq=s["dq"], dk=s["dk"], dv=s["dv"], **kw)
            return {"dq": dq, "dk": dk, "dv": dv}
        out, lse = qkr.attention(s["q"], s["k"], s["v"], **kw)
        return {"out": out, "lse": lse}
    if case["op"] == "norm":
        if not case["grad"]:
            return {"y": qkr.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)}
        if case["batches"]:
            dx, dw, db = qkr.fuse_scale_shift_backward(s["dy"], s["x"], s["weight"], eps=EPS)
        else:
            dx, dw, db = qkr.layer_norm_backward(s["dy"], s["x"], s["weight"], eps=EPS)
        return {"dx": dx, "dweight": dw, "dbias": db}
    kw = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], cos=s["cos"], sin=s["sin"], eps=EPS,
              cos_layout=case["layout"], style=case["style"])
    if case["fused"]:
        dqg, dkg = qkr.qknorm_rope_backward(s["do"], s["x"], out=s["dx"], **kw)
        return {"dx": s["dx"], "dq_gamma": dqg, "dk_gamma": dkg}
    dxq, dxk = torch.empty_like(s["xq"]), torch.empty_like(s["xk"])
    dqg, dkg = qkr.qknorm_rope_backward(dq=s["doq"], dk=s["dok"], q=s["xq"], k=s["xk"],
                                        dq_out=dxq, dk_out=dxk, **kw)
    return {"dx": {"q": dxq, "k": dxk}, "dq_gamma": dqg, "dk_gamma": dkg}


# ------------------------------------------------------------------ plain forms

def _heads_first(x, groups=1):
    """[batch, tokens, heads, head_dim] -> contiguous fp32 [batch, heads * groups, tokens, head_dim]."""
    return x.float().permute(0, 2, 1, 3).repeat_interleave(groups, 1).contiguous()


def _hidden_pairs(s):
    """True where a key is hidden from a query, [batch or 1, 1, q, k]; None if none is."""
    case = s["case"]
    sq, sk = case["q_tokens"], case["kv_tokens"]
    j = torch.arange(sk, device="cuda")
    hidden = None
    if s["kv_lengths"] is not None:
        hidden = (j >= s["kv_lengths"][:, None])[:, None, None, :]
    if case["causal"]:
        late = (j > torch.arange(sq, device="cuda")[:, None] + (sk - sq))[None, None]
        hidden = late if hidden is None else hidden | late
    return hidden


def _scores(s, q, k):
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(q.shape[-1]))
    hidden = _hidden_pairs(s)
    return scores if hidden is None else scores.masked_fill_(hidden, -math.inf)


def _attention(s):
    case = s["case"]
    groups = case["heads"] // case["kv_heads"]
    q, k, v = _heads_first(s["q"]), _heads_first(s["k"], groups), _heads_first(s["v"], groups)
    p = _scores(s, q, k)
    top = p.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = p.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    lse = (top + total.log()).squeeze(3)
    out = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return out.permute(0, 2, 1, 3).to(s["q"].dtype).contiguous(), lse


def _attention_backward(s):
    case = s["case"]
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
    groups = h // hk
    q, k, v = _heads_first(s["q"]), _heads_first(s["k"], groups), _heads_first(s["v"], groups)
    do, out = _heads_first(s["dout"]), _heads_first(s["out"])
    lse = s["lse"][..., None]
    lse = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    p = _scores(s, q, k).sub_(lse).exp_()
    delta = (do * out).sum(3, keepdim=True)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous()).sub_(delta).mul_(p)
    del p
    ds.mul_(1 / math.sqrt(d))
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    grads = {"dq": dq}
    for name, x in (("dk", dk), ("dv", dv)):
        grads[name] = x.view(b, hk, groups, -1, d).sum(2)
    return {n: x.permute(0, 2, 1, 3).to(s["q"].dtype).contiguous() for n, x in grads.items()}


def _normalised(s):
    x = s["x"].float()
    x = x - x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    return x * rstd, rstd


def _layer_norm(s):
    n, _ = _normalised(s)
    return (n * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)


def _layer_norm_backward(s):
    batches, c = s["case"]["batches"], s["case"]["hidden"]
    n, rstd = _normalised(s)
    dy = s["dy"].float()
    each = max(1, batches)
    w = 1 + s["weight"].float() if batches else s["weight"].float()[None]
    g = (dy.view(each, -1, c) * w[:, None]).view(-1, c)
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    dw = (dy * n).view(each, -1, c).sum(1, dtype=torch.float64).float()
    db = dy.view(each, -1, c).sum(1, dtype=torch.float64).float()
    if not batches:
        dw, db = dw[0], db[0]
    return {"dx": dx.to(s["x"].dtype), "dweight": dw, "dbias": db}


def _turned_back(do, cos, sin, style):
    """The transposed rotation: pairs (a, b) give do_a c_a + do_b s_b and do_b c_b - do_a s_a."""
    t = do * sin
    if style == "interleaved":
        t = t.unflatten(-1, (-1, 2))
        t = torch.stack([t[..., 1], -t[..., 0]], -1).flatten(-2)
    else:
        a, b = t.chunk(2, -1)
        t = torch.cat([b, -a], -1)
    return do * cos + t


def _qknorm_rope_backward(s):
    case = s["case"]
    n, h, d = case["tokens"], case["heads"], case["head_dim"]
    if case["fused"]:
        x, do = (s[k].view(n, 3, h, d)[:, :2].float() for k in ("x", "do"))
    else:
        x, do = (torch.stack([s[k + "q"], s[k + "k"]], 1).float() for k in ("x", "do"))
    shape = (n, 1, h, d) if case["layout"] == "per_head" else (n, 1, 1, d)
    dn = _turned_back(do, s["cos"].float().view(shape), s["sin"].float().view(shape), case["style"])
    r = 1 / torch.sqrt((x * x).mean(3, keepdim=True) + EPS)
    u = x * r
    g = dn * torch.stack([s["q_gamma"], s["k_gamma"]])[:, None]
    dx = (r * (g - u * (g * u).mean(3, keepdim=True))).to(TYPES[case["dtype"]])
    dgamma = (dn * u).sum((0, 2), dtype=torch.float64).float()
    if case["fused"]:
        v = torch.zeros_like(dx[:, :1])
        dx = torch.cat([dx, v], 1).view(n, 3 * h * d)
    else:
        dx = {"q": dx[:, 0].contiguous(), "k": dx[:, 1].contiguous()}
    return {"dx": dx, "dq_gamma": dgamma[0], "dk_gamma": dgamma[1]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attention(s)
    return _exact_norm(s) if case["op"] == "norm" else _exact_qk(s)


def _exact_attention(s):
    """Head by head; the backward pass from q, k, v and dout alone."""
    case = s["case"]
    b, sq, sk = case["batch"], case["q_tokens"], case["kv_tokens"]
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros((b, sq, h, d), **f64), torch.full((b, h, sq), -math.inf, **f64)
    dq, dk, dv = (torch.zeros((b, t, n, d), **f64) for t, n in ((sq, h), (sk, hk), (sk, hk)))
    for i, length in enumerate(_lengths(case)):
        if length == 0:
            continue
        seen = torch.arange(length, device="cuda")[None] <= (
            torch.arange(sq, device="cuda")[:, None] + (sk - sq) if case["causal"]
            else torch.full((sq, 1), sk, device="cuda"))
        some = seen.any(1, keepdim=True)
        for j in range(h):
            q = s["q"][i, :, j].double()
            k, v = (s[n][i, :length, j // (h // hk)].double() for n in ("k", "v"))
            x = q @ k.T
            x = torch.where(seen, x / math.sqrt(d), torch.tensor(-math.inf, **f64))
            total = torch.logsumexp(x, 1, keepdim=True)
            lse[i, j] = total[:, 0]
            x = torch.where(some, torch.exp(x - total), torch.tensor(0.0, **f64))
            if not case["grad"]:
                out[i, :, j] = x @ v
                continue
            do = s["dout"][i, :, j].double()
            dv[i, :length, j // (h // hk)] += x.T @ do
            y = do @ v.T
            y -= (x * y).sum(1, keepdim=True)
            x *= y
            del y
            dq[i, :, j] = x @ k / math.sqrt(d)
            dk[i, :length, j // (h // hk)] += x.T @ q / math.sqrt(d)
    return {"dq": dq, "dk": dk, "dv": dv} if case["grad"] else {"out": out, "lse": lse}


def _exact_norm(s):
    case = s["case"]
    x = s["x"].double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    w = s["weight"].double()
    if not case["grad"]:
        return {"y": (x - mean) / torch.sqrt(var + EPS) * w + s["bias"].double()}
    sd = torch.sqrt(var + EPS)
    n = (x - mean) / sd
    each, c = max(1, case["batches"]), case["hidden"]
    dy = s["dy"].double()
    dw = (dy * n).reshape(each, -1, c).sum(1)
    db = dy.reshape(each, -1, c).sum(1)
    g = dy * (1 + w if case["batches"] else w.view(1, c)).repeat_interleave(case["rows"] // each, 0)
    dx = (g - (g + n * (g * n).mean(1, keepdim=True)).mean(1, keepdim=True)
          - n * (g * n).mean(1, keepdim=True)) / sd
    return {"dx": dx, "dweight": dw if case["batches"] else dw[0],
            "dbias": db if case["batches"] else db[0]}


def _exact_qk(s):
    case = s["case"]
    n, h, d = case["tokens"], case["heads"], case["head_dim"]
    first = (torch.arange(0, d, 2, device="cuda") if case["style"] == "interleaved"
             else torch.arange(d // 2, device="cuda"))
    second = first + (1 if case["style"] == "interleaved" else d // 2)
    c, t = (s[k].double().view(n, -1, d) for k in ("cos", "sin"))
    found, gammas = [], []
    for i, name in enumerate(("q", "k")):
        if case["fused"]:
            x, do = (s[k][:, i * h * d:(i + 1) * h * d].double().view(n, h, d) for k in ("x", "do"))
        else:
            x, do = s["x" + name].double(), s["do" + name].double()
        dn = do * c
        dn[..., first] += do[..., second] * t[..., second]
        dn[..., second] -= do[..., first] * t[..., first]
        ms = x.square().mean(2, keepdim=True) + EPS
        gammas.append((dn * x / ms.sqrt()).sum((0, 1)))
        g = dn * s[name + "_gamma"].double()
        found.append((g - x * (g * x).mean(2, keepdim=True) / ms) / ms.sqrt())
    if case["fused"]:
        dx = torch.cat([x.reshape(n, h * d) for x in found + [torch.zeros_like(found[0])]], 1)
    else:
        dx = {"q": found[0], "k": found[1]}
    return {"dx": dx, "dq_gamma": gammas[0], "dk_gamma": gammas[1]}
