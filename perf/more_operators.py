"""Cases for the passes around the block-scaled linear layers: what a pass
computes, in plain torch operations and as calls of the library.

Each path has its own `op`:

  norm     what stands between two sublayers of a transformer block: the
           sublayer's output h is normed (if it has a norm of its own), gated
           and added to the scaled residual, and the sum normed for the next
           sublayer.
             u = post_norm(h) or h;  r' = res_scale r + gate u;  x = pre_norm(r')
           r' is kept in the residual's type, and x is the norm of what is
           kept.  train: with the backward pass, whose parameter gradients are
           sums over all tokens.
  logprob  log probabilities of given tokens under the logits, the entropy and
           the largest alternatives (ties to the lowest index).  train: with
           the gradient of the logits.
  distill  the divergence from a teacher of which each token's top logits are
           kept, and the gradient of the logits.  Form "top": the teacher's
           distribution is the softmax over its list.  Form "tail": the list
           holds log probabilities, and the rest of the vocabulary is one more
           outcome.
  head     the end of a model in block-scaled FP8, as a training step runs
           it: norm -> codes -> product with the vocabulary's weight -> log
           probabilities or distillation -> gradient of the logits as codes ->
           gradients of weight and input -> backward pass of the norm.

A padded row has no token (-1), no gradient, and zeros in the activations.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
BLOCK = 128


# ---------------------------------------------------------------- cases
def _norm(name, M, D, dtype, res, pre, post, gate, seqs, train):
    return dict(name=name, op="norm", M=M, D=D, dtype=dtype, res=res, pre=pre, post=post, gate=gate, seqs=seqs,
                train=train)


def listed():
    return [
        # one decoded token between two sublayers of the GPT-7B block
        _norm("norm token", 1, 4096, "bf16", "bf16", "layer", "none", "none", 1, False),
        # a batch of decoded tokens, a norm on either side of the sublayer
        _norm("norm 32 tokens", 32, 4096, "bf16", "f32", "rms", "rms", "channel", 1, False),
        # odd sizes, a gate for each sequence (modulation by a condition)
        _norm("norm odd", 777, 1001, "f16", "f32", "layer", "layer", "sequence", 7, True),
        # the GPT-7B block at its training batch, everything that the operator has
        _norm("norm 7b", 4096, 4096, "bf16", "f32", "rms", "rms", "channel", 1, True),
        # the GPT-175B block at its training batch, norms before the sublayers only
        _norm("norm 175b", 8192, 12288, "bf16", "bf16", "layer", "none", "none", 1, True),
        # a decoded token's log probability with the alternatives shown beside it
        dict(name="logprob token", op="logprob", M=1, V=50304, dtype="bf16", top=20, temp=1.0, ent=False, train=False),
        # a batch of decoded tokens in binary32, rows that start anywhere
        dict(name="logprob 32 tokens", op="logprob", M=32, V=50257, dtype="f32", top=5, temp=0.7, ent=True, train=False),
        # a policy's update: log probabilities and entropies, odd sizes
        dict(name="logprob odd", op="logprob", M=1003, V=32003, dtype="f16", top=0, temp=1.0, ent=True, train=True),
        # the loss of the GPT-7B model's training batch
        dict(name="logprob 7b", op="logprob", M=4096, V=50304, dtype="bf16", top=0, temp=1.0, ent=False, train=True),
        # a small odd student, binary32
        dict(name="distill odd", op="distill", M=129, V=1001, K=7, dtype="f32", form="top", temp=2.0),
        # the GPT-7B model's batch learning from a teacher's 64 largest log probabilities
        dict(name="distill 7b", op="distill", M=4096, V=50304, K=64, dtype="bf16", form="tail", temp=1.0),
        # the end of a small model
        dict(name="head", op="head", M=1024, D=2048, V=16384, dtype="bf16", loss="logprob", K=0),
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; every second one a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 16:
        v -= v % 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm", "logprob", "logprob", "logprob", "distill", "distill", "head"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "norm":
        train = rng.random() < 0.6
        seqs = rng.choice((1, 2, 3, 8, 16))
        res, D = rng.choice((dtype, "f32")), _log_int(rng, 64, 12288)
        most = 8192 * 12288 * 4 // (D * (BYTES[dtype] + BYTES[res]))
        M = _log_int(rng, 1, max(1, min(8192, most) // seqs)) * seqs
        return dict(op=op, M=M, D=D, dtype=dtype, res=res,
                    pre=rng.choice(("rms", "layer")), post=rng.choice(("none", "rms", "layer")),
                    gate="sequence" if seqs > 1 else rng.choice(("none", "channel")), seqs=seqs, train=train)
    if op == "logprob":
        train = rng.random() < 0.5
        top = 0 if train else rng.choice((0, 1, 5, 20, 32))
        V = _log_int(rng, 256, 160000)
        M = _log_int(rng, 1, max(1, min(8192 if top == 0 else 256, (4096 * 50304 // (2 if dtype == "f32" else 1)) // V)))
        return dict(op=op, M=M, V=V, dtype=dtype, top=top, temp=rng.choice((1.0, 0.7, 1.5)), ent=rng.random() < 0.5,
                    train=train)
    if op == "distill":
        V = _log_int(rng, 256, 160000)
        M = _log_int(rng, 1, max(1, min(4096, (2048 * 50304 // (2 if dtype == "f32" else 1)) // V)))
        return dict(op=op, M=M, V=V, K=_log_int(rng, 1, 200), dtype=dtype, form=rng.choice(("top", "tail")),
                    temp=rng.choice((1.0, 2.0)))
    loss = rng.choice(("logprob", "distill"))
    return dict(op=op, M=_log_int(rng, 64, 1024), D=_log_int(rng, 128, 2048), V=_log_int(rng, 512, 16384),
                dtype=rng.choice(("bf16", "f16")), loss=loss, K=16 if loss == "distill" else 0)


def work(case):
    M, op, e = case["M"], case["op"], BYTES[case["dtype"]]
    if op == "norm":
        n, er = M * case["D"], BYTES[case["res"]]
        # h and r read, r' and x written; then the gradients of x and r' read, those of h and r written
        return {"bytes": (2 if case["train"] else 1) * n * (2 * e + 2 * er), "flops": (60 if case["train"] else 16) * n}
    if op == "head":
        D, V = case["D"], case["V"]
        # h, r, and the gradient of r' read; r', the gradients of h, r and of the weight written; the weight's codes read
        return {"bytes": M * D * (2 * e + 16) + V * D * (1 + e), "flops": 6 * M * D * V + 30 * M * V}
    n = M * case["V"]
    if op == "logprob":
        # logits read, their gradient written
        return {"bytes": n * e * (2 if case["train"] else 1) + M * (24 + 8 * case["top"]), "flops": (14 if case["train"] else 5) * n}
    return {"bytes": n * e * 2 + M * (16 + 8 * case["K"]), "flops": 12 * n}


# ---------------------------------------------------------------- inputs
def _normal(shape, std, gen, dtype):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _activations(M, D, gen, dtype, std=1.0):
    """N(0, std) with a few outlier features, as activations have, around a small offset; a padded row is zero."""
    x = torch.empty((M, D), dtype=torch.float32, device="cuda").normal_(0.05 * std, std, generator=gen)
    cols = torch.randint(0, D, (max(1, D // 512),), device="cuda", generator=gen)
    x[:, cols] *= 20.0
    if M > 2:
        x[M // 2] = 0.0
    return x.to(dtype)


def _gradients(M, D, gen, dtype):
    """N(0, 1e-3), its size varying from token to token (times 2^6 in f16); none for the padded row."""
    g = torch.empty((M, D), dtype=torch.float32, device="cuda").normal_(0.0, 1e-3 * (64 if dtype == torch.float16 else 1),
                                                                        generator=gen)
    g *= torch.exp2(torch.randint(-2, 3, (M, 1), device="cuda", generator=gen).float())
    if M > 2:
        g[M // 2] = 0.0
    return g.to(dtype)


def _tokens(M, V, gen):
    t = torch.randint(0, V, (M,), device="cuda", generator=gen)
    if M > 2:
        t[M // 2] = -1
    return t


def _logits(M, V, gen, dtype, tokens):
    """Logits of a model that expects something: N(0, 2), most rows with a peak at the token; the last columns, which
    pad the vocabulary, are masked."""
    z = torch.empty((M, V), dtype=torch.float32, device="cuda").normal_(0.0, 2.0, generator=gen)
    sure = torch.rand((M,), device="cuda", generator=gen) * 12.0
    z.scatter_add_(1, tokens.clamp_min(0)[:, None], sure[:, None])
    z = z.to(dtype)
    if V >= 1000:
        z[:, V - 17:] = -math.inf
    return z


def _row_weights(M, gen, tokens):
    """The gradient of each row's loss, as a mean over the tokens gives it; none for a padded row."""
    g = (0.5 + torch.rand((M,), device="cuda", generator=gen)) / M
    return torch.where(tokens < 0, torch.zeros_like(g), g)


def _teacher(z, K, form, temp, gen):
    """A teacher near the student: its K largest logits (form "top") or log probabilities (form "tail") with their
    places, in no order."""
    t = z.float() + torch.empty(z.shape, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    values, ids = torch.topk(t, K, dim=1)
    if form == "tail":
        values = values / temp - torch.logsumexp(t / temp, dim=1, keepdim=True)
    order = torch.randperm(K, device="cuda", generator=gen)
    return values[:, order].contiguous(), ids[:, order].contiguous()


def _codes(rows, cols):
    return torch.empty((rows, -(-cols // 16) * 16), dtype=torch.uint8, device="cuda")[:, :cols]


def _scales(rows, cols):
    return torch.empty(-(-rows // 128) * -(-cols // 512) * 512, dtype=torch.uint8, device="cuda")


def _pack(e8, rows, cols):
    """Scale bytes [rows, ceil(cols / 128)] in the library's order: groups of 128 rows x 4 blocks, 512 bytes each."""
    kb = -(-cols // BLOCK)
    rb, kg = -(-rows // 128), -(-kb // 4)
    full = torch.full((rb * 128, kg * 4), 127, dtype=torch.uint8, device=e8.device)
    full[:rows, :kb] = e8
    return full.view(rb, 4, 32, kg, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _weight(V, D, gen, s):
    """The vocabulary's kept weight: E4M3 codes with the scales of their 128x128 blocks for either reduction."""
    w = torch.empty((V, D), dtype=torch.float32, device="cuda").normal_(0.0, 0.02, generator=gen).to(torch.bfloat16)
    e = _exponents(w.float(), "e4m3", BLOCK, BLOCK)
    s["wv"] = _rounded(w.float(), "e4m3", BLOCK, BLOCK)  # the values of the codes
    s["wq"] = _codes(V, D)
    s["wq"].copy_((s["wv"] * torch.exp2(_spread(e, BLOCK, BLOCK, V, D))).to(torch.float8_e4m3fn).view(torch.uint8))
    e8 = (127 - e).to(torch.uint8)
    s["ws"] = _pack(e8.repeat_interleave(BLOCK, 0)[:V], V, D)
    s["ws_t"] = _pack(e8.T.repeat_interleave(BLOCK, 0)[:D], D, V)


def _prepare_norm(s, case, gen):
    M, D, dt = case["M"], case["D"], DTYPES[case["dtype"]]
    rt = DTYPES[case["res"]]
    new = lambda t, *shape: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    s |= {"h": _activations(M, D, gen, dt), "r": _activations(M, D, gen, rt, 3.0), "res_scale": 0.9}
    s["w"] = 1.0 + _normal((D,), 0.1, gen, torch.float32)
    s["b"] = _normal((D,), 0.1, gen, torch.float32) if case["pre"] == "layer" else None
    s["post_w"] = 1.0 + _normal((D,), 0.1, gen, torch.float32) if case["post"] != "none" else None
    s["post_b"] = _normal((D,), 0.1, gen, torch.float32) if case["post"] == "layer" else None
    s["gate"] = {"none": None, "channel": _normal((D,), 0.3, gen, torch.float32),
                 "sequence": _normal((case["seqs"], D), 0.3, gen, torch.float32)}[case["gate"]]
    for k in ("w", "b", "post_w", "post_b", "gate"):
        s[k] = None if s[k] is None else s[k].to(dt)
        s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
    s |= {"r_out": new(rt, M, D), "x": new(dt, M, D), "stats": new(torch.float32, M, 4)}
    if case["train"]:
        s |= {"dx": _gradients(M, D, gen, dt), "dr_out": _gradients(M, D, gen, rt), "dh": new(dt, M, D), "dr": new(rt, M, D)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M, dt = case["op"], case["M"], DTYPES[case["dtype"]]
    s = {"case": case}
    f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device="cuda")  # noqa: E731
    if op == "norm":
        _prepare_norm(s, case, gen)
        return s
    V = case["V"]
    s["tokens"] = _tokens(M, V, gen)
    s["g"] = _row_weights(M, gen, s["tokens"])
    s |= {"loss": f32(M), "loss_stats": f32(M, 4)}
    if op == "head":
        D = case["D"]
        _prepare_norm(s, case | {"res": "f32", "pre": "rms", "post": "none", "gate": "none", "seqs": 1, "train": True}, gen)
        _weight(V, D, gen, s)
        s |= {"xq": _codes(M, D), "xs": _scales(M, D), "xq_t": _codes(M, D), "xs_t": _scales(D, M)}
        s |= {"dq": _codes(M, V), "ds": _scales(M, V), "dq_t": _codes(M, V), "ds_t": _scales(V, M)}
        s |= {"logits": f32(M, V), "dw_head": torch.empty((V, D), dtype=dt, device="cuda")}
        if case["loss"] == "distill":
            s["ids"] = torch.randint(0, V, (M, case["K"]), device="cuda", generator=gen)
            s["ids"] = (s["ids"][:, :1] + torch.arange(case["K"], device="cuda") * 31) % V  # (distinct)
            s["values"] = _normal((M, case["K"]), 2.0, gen, torch.float32)
        else:
            s["g"] = -s["g"]  # the loss is the negative log probability
    else:
        s["logits"] = _logits(M, V, gen, dt, s["tokens"])
        s["dlogits"] = torch.empty_like(s["logits"])
    if op == "distill":
        s["values"], s["ids"] = _teacher(s["logits"], case["K"], case["form"], case["temp"], gen)
    if op == "distill" or op == "head" and case["loss"] == "distill":
        s["ids"] = s["ids"].to(torch.int32)
        s["list_ids"] = torch.empty((M, case["K"]), dtype=torch.int32, device="cuda")
        s["list_q"] = f32(M, case["K"])
    if op == "logprob":
        s["entropy"] = f32(M) if case["ent"] else None
        s["g_ent"] = s["g"] * -0.01 if case["ent"] and case["train"] else None
        k = case["top"]
        s |= {"top_logp": f32(M, k) if k else None,
              "top_ids": torch.empty((M, k), dtype=torch.int32, device="cuda") if k else None}
    return s


# ---------------------------------------------------------------- plain form (32 bits)
def _centred(x, kind):
    """(x - mean for a layer norm, 1 / sqrt(mean square + eps))."""
    if kind == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    return x, torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _affine(n, w, b):
    y = n * w.float()
    return y if b is None else y + b.float()


def _norm_back(dn, n, rstd, kind):
    """Gradient of the norm's input from that of its normed value n."""
    d = dn - n * (dn * n).mean(dim=1, keepdim=True)
    if kind == "layer":
        d = d - dn.mean(dim=1, keepdim=True)
    return d * rstd


def _gate_of(s, case):
    if s["gate"] is None:
        return None
    return s["gate"].float().view(-1, case["D"]).repeat_interleave(case["M"] // case["seqs"], 0)


def _plain_norm_fwd(s, case):
    """(what the backward pass needs, r' in its type, x in 32 bits)."""
    keep = {}
    u = s["h"].float()
    if case["post"] != "none":
        c, keep["rstd1"] = _centred(u, case["post"])
        keep["n1"] = c * keep["rstd1"]
        u = _affine(keep["n1"], s["post_w"], s["post_b"])
    gate = _gate_of(s, case)
    r_out = (s["r"].float() * s["res_scale"] + (u if gate is None else u * gate)).to(s["r"].dtype)
    c, keep["rstd2"] = _centred(r_out.float(), case["pre"])
    keep |= {"u": u, "gate": gate, "n2": c * keep["rstd2"]}
    return keep, r_out, _affine(keep["n2"], s["w"], s["b"])


def _plain_norm_bwd(s, case, keep, dx, dr_out):
    """Gradients of the pass from those of x and r' (32 bits)."""
    dt, rt = s["h"].dtype, s["r"].dtype
    n2, gate = keep["n2"], keep["gate"]
    g = dr_out + _norm_back(dx * s["w"].float(), n2, keep["rstd2"], case["pre"])
    out = {"dw": (dx * n2).sum(dim=0).to(dt), "dr": (g * s["res_scale"]).to(rt)}
    if s["b"] is not None:
        out["db"] = dx.sum(dim=0).to(dt)
    if gate is not None:
        out["dgate"] = (g * keep["u"]).view(case["seqs"], -1, case["D"]).sum(dim=1).view(s["gate"].shape).to(dt)
    du = g if gate is None else g * gate
    if case["post"] != "none":
        out["dpost_w"] = (du * keep["n1"]).sum(dim=0).to(dt)
        if s["post_b"] is not None:
            out["dpost_b"] = du.sum(dim=0).to(dt)
        du = _norm_back(du * s["post_w"].float(), keep["n1"], keep["rstd1"], case["post"])
    out["dh"] = du.to(dt)
    return out


def _softmax(z, temp):
    """(scaled logits, their maximum, exp of the difference, its sum)."""
    z = z.float() / temp
    m = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - m)
    return z, m, e, e.sum(dim=1, keepdim=True)


def _plain_logprob(z, tokens, temp, ent, top, g, g_ent):
    out = {}
    s, m, e, total = _softmax(z, temp)
    log_total = torch.log(total)
    at = tokens.clamp_min(0)[:, None]
    logp = (s.gather(1, at) - m - log_total)[:, 0]
    out["logp"] = torch.where(tokens < 0, torch.zeros_like(logp), logp)
    if top:
        ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]
        out |= {"top_ids": ids.to(torch.int32), "top_logp": s.gather(1, ids) - m - log_total}
    p = e / total
    if ent:
        low = torch.where(e > 0, s - m, torch.zeros_like(s)) - log_total
        out["entropy"] = -(p * low).sum(dim=1)
    if g is None:
        return out, None
    d = p * -g[:, None]
    if g_ent is not None:
        d = d - p * (low + out["entropy"][:, None]) * g_ent[:, None]
    d.scatter_add_(1, at, g[:, None])  # (0 for a padded row)
    return out, d / temp


def _plain_distill(z, ids, values, form, temp, g):
    ids = ids.long()
    s, m, e, total = _softmax(z, temp)
    values = values.float()
    if form == "top":
        values = values / temp
        top = torch.exp(values - values.amax(dim=1, keepdim=True))
        q = top / top.sum(dim=1, keepdim=True)
    else:
        q = torch.exp(values)
    low = s.gather(1, ids) - m - torch.log(total)
    loss = torch.where(q > 0, q * (torch.log(q) - low), torch.zeros_like(q)).sum(dim=1)
    p = e / total
    if form == "top":
        d = p
    else:
        q_rest = (1.0 - q.sum(dim=1)).clamp_min(0.0)
        p_rest = p.scatter(1, ids, 0.0).sum(dim=1)
        there = (q_rest > 0) & (p_rest > 0)
        loss = loss + torch.where(there, q_rest * (torch.log(q_rest) - torch.log(p_rest)), torch.zeros_like(loss))
        q_rest, p_rest = q_rest.where(there, 0.0 * q_rest), p_rest.where(there, torch.ones_like(p_rest))
        whole = q.sum(dim=1) + q_rest
        d = p * (whole - q_rest / p_rest)[:, None]
        d.scatter_(1, ids, p.gather(1, ids) * whole[:, None])
    d = d.scatter_add(1, ids, -q) * g[:, None] / temp
    return {"loss": loss}, d


def _tiles(x, br, bc):
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, -C % bc, 0, -R % br))
    return x.view(x.shape[0] // br, br, x.shape[1] // bc, bc)


def _exponents(x, fmt, br, bc):
    """Exponents of the block scales: the largest e with amax * 2^e <= fmt_max = 0.875 * 2^k."""
    m, ex = torch.frexp(_tiles(x.abs(), br, bc).amax(dim=(1, 3)))
    k = 9 if fmt == "e4m3" else 16
    e = torch.where(m <= 0.875, k - ex, k - 1 - ex).clamp(-126, 126)
    return torch.where(m == 0, torch.zeros_like(e), e).float()


def _spread(e, br, bc, R, C):
    return e.repeat_interleave(br, 0)[:R].repeat_interleave(bc, 1)[:, :C]


def _rounded(x, fmt, br, bc):
    """The values that the codes and scales of x stand for."""
    e = _spread(_exponents(x, fmt, br, bc), br, bc, *x.shape)
    v = x * torch.exp2(e)
    bits, low = (4, -5) if fmt == "e4m3" else (3, -13)  # significand bits; frexp's exponent of the smallest normal
    unit = torch.exp2((torch.frexp(v)[1].clamp_min(low) - bits).to(x.dtype))
    return torch.round(v / unit) * unit * torch.exp2(-e)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        keep, r_out, x = _plain_norm_fwd(s, case)
        out = {"r_out": r_out, "x": x.to(s["h"].dtype)}
        if case["train"]:
            out |= _plain_norm_bwd(s, case, keep, s["dx"].float(), s["dr_out"].float())
        return out
    if op == "logprob":
        train = case["train"]
        out, d = _plain_logprob(s["logits"], s["tokens"], case["temp"], case["ent"], case["top"],
                                s["g"] if train else None, s["g_ent"])
        return out | ({"dlogits": d.to(s["logits"].dtype)} if train else {})
    if op == "distill":
        out, d = _plain_distill(s["logits"], s["ids"], s["values"], case["form"], case["temp"], s["g"])
        return out | {"dlogits": d.to(s["logits"].dtype)}
    full = case | {"pre": "rms", "post": "none", "gate": "none", "seqs": 1}
    dt = s["h"].dtype
    keep, r_out, x = _plain_norm_fwd(s, full)
    logits = _rounded(x, "e4m3", 1, BLOCK) @ s["wv"].T
    if case["loss"] == "logprob":
        out, d = _plain_logprob(logits, s["tokens"], 1.0, False, 0, s["g"], None)
    else:
        out, d = _plain_distill(logits, s["ids"], s["values"], "top", 1.0, s["g"])
    dx = (_rounded(d, "e5m2", 1, BLOCK) @ s["wv"]).to(dt)
    out["dw_head"] = (_rounded(d, "e5m2", BLOCK, 1).T @ _rounded(x, "e4m3", BLOCK, 1)).to(dt)
    return out | {"r_out": r_out} | _plain_norm_bwd(s, full, keep, dx.float(), s["dr_out"].float())


# ---------------------------------------------------------------- the library's calls
def _own_norm_fwd(s, case, fp8, **codes):
    kinds = {"none": fp8.FP8_NORM_NONE, "rms": fp8.FP8_NORM_RMS, "layer": fp8.FP8_NORM_LAYER}
    fp8.fp8_norm_fwd(s["h"], s["r"], s["r_out"], s["stats"], pre=kinds[case["pre"]], post=kinds[case["post"]],
                     w=s["w"], b=s["b"], post_w=s["post_w"], post_b=s["post_b"], gate=s["gate"],
                     res_scale=s["res_scale"], eps=EPS, **codes)
    return {"r_out": s["r_out"]}


def _own_norm_bwd(s, case, fp8, dx):
    kinds = {"none": fp8.FP8_NORM_NONE, "rms": fp8.FP8_NORM_RMS, "layer": fp8.FP8_NORM_LAYER}
    out = {k: s[k] for k in ("dh", "dr", "dw", "db", "dgate", "dpost_w", "dpost_b") if s[k] is not None}
    if "workspace" not in s:  # a program allocates it once
        need = fp8.fp8_norm_workspace_bytes(case["M"], case["D"], case["M"] // case["seqs"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    fp8.fp8_norm_bwd(dx, s["dr_out"], s["h"], s["r_out"], s["stats"], pre=kinds[case["pre"]],
                     post=kinds[case["post"]], w=s["w"], post_w=s["post_w"], post_b=s["post_b"], gate=s["gate"],
                     res_scale=s["res_scale"], workspace=s["workspace"], **out)
    return out


def _own(s):
    from fp8_mixed_precision_tensor_b200 import fp8

    case = s["case"]
    op = case["op"]
    if op == "norm":
        out = _own_norm_fwd(s, case, fp8, x=s["x"]) | {"x": s["x"]}
        return out | (_own_norm_bwd(s, case, fp8, s["dx"]) if case["train"] else {})
    if op == "logprob":
        beta = 1.0 / case["temp"]
        fp8.fp8_logprob_fwd(s["logits"], s["tokens"], s["loss"], s["loss_stats"], inv_temp=beta, entropy=s["entropy"],
                            top_logp=s["top_logp"], top_ids=s["top_ids"])
        out = {"logp": s["loss"]}
        out |= {k: s[k] for k in ("entropy", "top_logp", "top_ids") if s[k] is not None}
        if case["train"]:
            fp8.fp8_logprob_bwd(s["logits"], s["tokens"], s["loss_stats"], s["g"], inv_temp=beta, dentropy=s["g_ent"],
                                dlogits=s["dlogits"])
            out["dlogits"] = s["dlogits"]
        return out
    if op == "distill":
        form = fp8.FP8_DISTILL_TOP if case["form"] == "top" else fp8.FP8_DISTILL_TAIL
        beta = 1.0 / case["temp"]
        fp8.fp8_distill_fwd(s["logits"], s["ids"], s["values"], s["loss"], s["loss_stats"], s["list_ids"], s["list_q"],
                            form=form, inv_temp=beta)
        fp8.fp8_distill_bwd(s["logits"], s["list_ids"], s["list_q"], s["loss_stats"], s["g"], inv_temp=beta,
                            dlogits=s["dlogits"])
        return {"loss": s["loss"], "dlogits": s["dlogits"]}
    full = case | {"pre": "rms", "post": "none", "seqs": 1}
    out = _own_norm_fwd(s, full, fp8, x_q=s["xq"], x_s=s["xs"], x_q_col=s["xq_t"], x_s_col=s["xs_t"])
    fp8.fp8_block_linear_fwd(s["xq"], s["xs"], s["wq"], s["ws"], s["logits"])
    codes = dict(fmt=fp8.FP8_E5M2, d_q=s["dq"], d_s=s["ds"], d_q_col=s["dq_t"], d_s_col=s["ds_t"])
    if case["loss"] == "logprob":
        fp8.fp8_logprob_fwd(s["logits"], s["tokens"], s["loss"], s["loss_stats"])
        out["logp"] = s["loss"]
        fp8.fp8_logprob_bwd(s["logits"], s["tokens"], s["loss_stats"], s["g"], **codes)
    else:
        fp8.fp8_distill_fwd(s["logits"], s["ids"], s["values"], s["loss"], s["loss_stats"], s["list_ids"], s["list_q"])
        out["loss"] = s["loss"]
        fp8.fp8_distill_bwd(s["logits"], s["list_ids"], s["list_q"], s["loss_stats"], s["g"], **codes)
    fp8.fp8_block_linear_dgrad(s["dq"], s["ds"], fp8.FP8_E5M2, s["wq"], s["ws_t"], s["x"])
    fp8.fp8_block_linear_wgrad(s["dq_t"], s["ds_t"], fp8.FP8_E5M2, s["xq_t"], s["xs_t"], s["dw_head"])
    return out | {"dw_head": s["dw_head"]} | _own_norm_bwd(s, full, fp8, s["x"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definition
def _stored(x, like):
    """x as its type holds it, for autograd the identity."""
    return x + (x.detach().to(like.dtype).double() - x.detach())


def _exact_norm(x, kind, w, b):
    mean = x.sum(1, keepdim=True) / x.shape[1] if kind == "layer" else 0.0
    var = torch.square(x - mean).sum(1, keepdim=True) / x.shape[1]
    y = (x - mean) / torch.sqrt(var + EPS) * w
    return y if b is None else y + b


def _exact_norm_fwd(s, case):
    """(leaves by name, r', x) with the graph between them."""
    p = {k: s[k].detach().double().requires_grad_() for k in ("h", "r", "w", "b", "post_w", "post_b", "gate")
         if s[k] is not None}
    u = p["h"] if case["post"] == "none" else _exact_norm(p["h"], case["post"], p["post_w"], p.get("post_b"))
    if "gate" in p:
        u = (u.view(case["seqs"], -1, case["D"]) * p["gate"].view(case["seqs"], 1, case["D"])).view(u.shape)
    r_out = _stored(s["res_scale"] * p["r"] + u, s["r"])
    return p, r_out, _exact_norm(r_out, case["pre"], p["w"], p.get("b"))


def _exact_norm_bwd(p, r_out, x, dx, dr_out):
    grads = torch.autograd.grad([x, r_out], list(p.values()), [dx, dr_out])
    return {"d" + k: g for k, g in zip(p, grads)}


def _exact_rows(z, temp):
    """(log probabilities, probabilities), -inf and 0 where the logit is -inf."""
    lp = z.double() / temp
    lp = lp - torch.logsumexp(lp, dim=1, keepdim=True)
    return lp, torch.exp(lp)


def _exact_logprob(z, tokens, temp, ent, top, g, g_ent):
    lp, p = _exact_rows(z, temp)
    rows = torch.arange(z.shape[0], device=z.device)
    there = tokens >= 0
    out = {"logp": torch.where(there, lp[rows, tokens.clamp_min(0)], 0.0)}
    if top:
        # by (value, lowest index): numpy's lexicographic order on the candidates of torch's own top values
        kth = torch.topk(z.float(), top, dim=1)[0][:, -1:]
        ids = []
        for i in range(z.shape[0]):
            at = torch.nonzero(z[i].float() >= kth[i])[:, 0]
            ids.append(at[torch.argsort(z[i, at].double(), descending=True, stable=True)][:top])
        ids = torch.stack(ids)
        out |= {"top_ids": ids.to(torch.int32), "top_logp": lp.gather(1, ids)}
    if ent:
        out["entropy"] = torch.special.entr(p).sum(dim=1)
    if g is None:
        return out, None
    d = -p
    d[rows[there], tokens[there]] += 1.0
    d *= g.double()[:, None]
    if g_ent is not None:  # dH/ds_j = -p_j (log p_j + H)
        d += g_ent.double()[:, None] * (torch.special.entr(p) - p * out["entropy"][:, None])
    return out, d / temp


def _exact_distill(z, ids, values, form, temp, g):
    lp, p = _exact_rows(z, temp)
    v, ids = values.double(), ids.long()
    lq = torch.log_softmax(v / temp, dim=1) if form == "top" else v
    loss = (torch.exp(lq) * (lq - lp.gather(1, ids))).sum(dim=1)
    q = torch.zeros_like(p).scatter_(1, ids, torch.exp(lq))
    if form == "top":
        return {"loss": loss}, (p - q) * (g.double() / temp)[:, None]
    listed_ = torch.zeros_like(p, dtype=torch.bool).scatter_(1, ids, True)
    q_rest = (1.0 - torch.exp(lq).sum(dim=1)).clamp_min(0.0)
    p_rest = torch.where(listed_, 0.0, p).sum(dim=1)
    there = (q_rest > 0) & (p_rest > 0)
    ratio = torch.where(there, q_rest / p_rest, 0.0)
    loss = loss + torch.where(there, q_rest * torch.log(torch.where(there, q_rest / p_rest, 1.0)), 0.0)
    whole = torch.exp(lq).sum(dim=1) + torch.where(there, q_rest, 0.0)
    q = torch.where(listed_, q, p * ratio[:, None])  # the rest's share goes by the student's own proportions
    return {"loss": loss}, (p * whole[:, None] - q) * (g.double() / temp)[:, None]


def _exact_values(x, fmt, br, bc):
    """x rounded to the format at its blocks' scales, every step in binary64.

    The scale is found by trial (the guess of a logarithm, moved until
    amax * s <= fmt_max < 2 * amax * s); the format's grid at a value has the
    spacing 2^(e - digits), e the value's exponent, not below the smallest
    normal one."""
    fmax, digits, low = (448.0, 3, -6) if fmt == "e4m3" else (57344.0, 2, -14)
    R, C = x.shape
    grid = torch.zeros((-(-R // br) * br, -(-C // bc) * bc), dtype=torch.float64, device=x.device)
    grid[:R, :C] = x
    rows = grid.reshape(-1, br, grid.shape[1]).abs().amax(1)
    amax = rows.reshape(rows.shape[0], -1, bc).amax(2)
    safe = torch.where(amax > 0, amax, torch.full_like(amax, fmax))
    s = torch.exp2(torch.floor(torch.log2(fmax / safe)))
    s = torch.where(safe * s > fmax, s / 2, s)
    s = torch.where(safe * s * 2 <= fmax, s * 2, s).clamp(2.0 ** -126, 2.0 ** 126)
    s = s[:, None, :, None].expand(-1, br, -1, bc).reshape(grid.shape)[:R, :C]
    v = x * s
    mag = v.abs().clamp_min(2.0 ** low)
    e = torch.floor(torch.log2(mag))
    e = torch.where(torch.exp2(e) > mag, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= mag, e + 1, e)
    step = torch.exp2(e - digits)
    return torch.round(v / step) * step / s


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        p, r_out, x = _exact_norm_fwd(s, case)
        out = {"r_out": r_out.detach(), "x": x.detach()}
        if case["train"]:
            out |= _exact_norm_bwd(p, r_out, x, s["dx"].double(), s["dr_out"].double())
        return out
    if op == "logprob":
        out, d = _exact_logprob(s["logits"], s["tokens"], case["temp"], case["ent"], case["top"],
                                s["g"] if case["train"] else None, s["g_ent"])
        return out if d is None else out | {"dlogits": d}
    if op == "distill":
        out, d = _exact_distill(s["logits"], s["ids"], s["values"], case["form"], case["temp"], s["g"])
        return out | {"dlogits": d}
    p, r_out, x = _exact_norm_fwd(s, case | {"pre": "rms", "post": "none", "seqs": 1})
    xv = x.detach()
    logits = torch.matmul(_exact_values(xv, "e4m3", 1, BLOCK), s["wv"].double().T)
    if case["loss"] == "logprob":
        out, d = _exact_logprob(logits, s["tokens"], 1.0, False, 0, s["g"], None)
    else:
        out, d = _exact_distill(logits, s["ids"], s["values"], "top", 1.0, s["g"])
    # the gradient of x is stored in the tensors' own type
    dx = torch.matmul(_exact_values(d, "e5m2", 1, BLOCK), s["wv"].double()).to(s["h"].dtype).double()
    out["dw_head"] = torch.matmul(_exact_values(d, "e5m2", BLOCK, 1).T, _exact_values(xv, "e4m3", BLOCK, 1))
    return out | {"r_out": r_out.detach()} | _exact_norm_bwd(p, r_out, x, dx, s["dr_out"].double())
