"""Cases for the block-scaled FP8 operators: what a pass computes, in plain
torch operations and as calls of the library.

Three paths, each with its own `op`:

  linear  a linear layer on weights kept as E4M3 codes with one power-of-two
          scale per 128x128 block: the activations are cast with one scale per
          1x128 block of a token's features, multiplied, and rounded to the
          output type, with a bias.  The serving form; M is the token count.
  step    the same layer's training pass from bf16/f16/f32 tensors: casts of
          X, dY and W, forward, gradient of the input, gradient of the weight
          (blocks of 128 tokens along the reduction).
  act     an activation function whose input is kept as E4M3 codes with one
          scale per 1x128 block, and the backward pass from those codes.
  mlp     fc1 -> activation -> fc2 forward and backward on the above: only
          8-bit tensors are kept from the forward pass for the backward.

A block's scale is 2^floor(log2(fmt_max / amax)) (1 for an all-zero block);
its elements are rounded to nearest even after the scaling.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FMT_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through the QKV projection of the GPT-7B block
        dict(name="linear token qkv", op="linear", M=1, K=4096, N=12288, dtype="bf16"),
        # a batch of decoded tokens through its output projection
        dict(name="linear 16 tokens out", op="linear", M=16, K=4096, N=4096, dtype="f16"),
        # a ragged prompt through fc2 (no size a multiple of the tiles)
        dict(name="linear ragged prompt", op="linear", M=1003, K=4104, N=5000, dtype="bf16"),
        # fc1 of the GPT-7B block at its training batch
        dict(name="linear fc1 7b", op="linear", M=4096, K=4096, N=16384, dtype="bf16"),
        # the single 256x256 linear layer of the tests
        dict(name="step single linear", op="step", M=256, K=256, N=256, dtype="bf16", grad="e5m2"),
        # odd sizes in every dimension, f16 tensors
        dict(name="step odd", op="step", M=777, K=1001, N=1305, dtype="f16", grad="e4m3"),
        # output projection of the GPT-7B block
        dict(name="step out 7b", op="step", M=4096, K=4096, N=4096, dtype="bf16", grad="e5m2"),
        # output projection of the GPT-175B block
        dict(name="step out 175b", op="step", M=8192, K=12288, N=12288, dtype="bf16", grad="e5m2"),
        # a small layer's activation, f32 tensors, and the GPT-7B block's fc1 output
        dict(name="act small", op="act", M=500, N=2056, dtype="f32", act="silu"),
        dict(name="act 7b", op="act", M=4096, N=16384, dtype="bf16", act="gelu_tanh"),
        # the feed-forward half of a small odd model and of the GPT-7B block
        dict(name="mlp odd", op="mlp", M=300, K=520, N=2056, dtype="bf16", grad="e4m3", act="gelu_erf"),
        dict(name="mlp 7b", op="mlp", M=4096, K=4096, N=16384, dtype="bf16", grad="e5m2", act="gelu_tanh"),
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; every second one a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 16:
        v -= v % 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("linear", "linear", "step", "step", "act", "mlp"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    grad = rng.choice(("e5m2", "e4m3"))
    act = rng.choice(("gelu_tanh", "gelu_erf", "silu"))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 4096), K=_log_int(rng, 128, 16384), N=_log_int(rng, 128, 16384),
                    dtype=dtype)
    if op == "step":
        return dict(op=op, M=_log_int(rng, 64, 8192), K=_log_int(rng, 128, 8192), N=_log_int(rng, 128, 8192),
                    dtype=dtype, grad=grad)
    if op == "act":
        return dict(op=op, M=_log_int(rng, 16, 8192), N=_log_int(rng, 128, 16384),
                    dtype=rng.choice(("bf16", "f16", "f32")), act=act)
    return dict(op=op, M=_log_int(rng, 64, 4096), K=_log_int(rng, 128, 4096), N=_log_int(rng, 256, 16384),
                dtype=dtype, grad=grad, act=act)


def work(case):
    M, N, e = case["M"], case["N"], BYTES[case["dtype"]]
    if case["op"] == "act":
        # h and da read, a and dh written, the 8-bit copy of h written and read
        # once each; about 40 operations for the function and its derivative
        return {"bytes": M * N * (4 * e + 2) + 2 * M * -(-N // BLOCK), "flops": 40 * M * N}
    K = case["K"]
    if case["op"] == "linear":
        return {"bytes": M * K * e + N * K + -(-N // BLOCK) * -(-K // BLOCK) + N * e + M * N * e, "flops": 2 * M * N * K}
    if case["op"] == "step":
        # X, dY, W read; Y, dX, dW written
        return {"bytes": 2 * e * (M * K + M * N + N * K), "flops": 6 * M * N * K}
    # X, dY, W1, W2 read; Y, dX, dW1, dW2 written
    return {"bytes": e * (4 * M * K + 4 * N * K), "flops": 12 * M * N * K}


# ---------------------------------------------------------------- inputs
def _normal(shape, std, gen, dtype):
    t = torch.empty(shape, dtype=torch.float32, device="cuda")
    return t.normal_(0.0, std, generator=gen).to(dtype)


def _activations(M, K, gen, dtype):
    """N(0, 1) with a few outlier features, as activations have, and a padded (all-zero) token row."""
    x = torch.empty((M, K), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    cols = torch.randint(0, K, (max(1, K // 256),), device="cuda", generator=gen)
    x[:, cols] *= 20.0
    if M > 2:
        x[M // 2] = 0.0
    return x.to(dtype)


def _gradients(M, N, gen, dtype):
    """N(0, 1e-4) (loss-scaled by 2^10 in f16), the size varying from token to token; a padded row has no gradient."""
    std = 1e-4 * (1024.0 if dtype == torch.float16 else 1.0)
    g = torch.empty((M, N), dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    g *= torch.exp2(torch.randint(-3, 4, (M, 1), device="cuda", generator=gen).float())
    if M > 2:
        g[M // 2] = 0.0
    return g.to(dtype)


def _codes(rows, cols):
    """A buffer of codes: rows padded to a multiple of 16 bytes."""
    return torch.empty((rows, -(-cols // 16) * 16), dtype=torch.uint8, device="cuda")[:, :cols]


def _scales(rows, cols):
    """A buffer of scales of 1x128 blocks of a rows x cols operand."""
    return torch.empty(-(-rows // 128) * -(-cols // 512) * 512, dtype=torch.uint8, device="cuda")


def _pack(e8, rows, cols):
    """Scale bytes [rows, ceil(cols / 128)] in the library's order: groups of 128 rows x 4 blocks, 512 bytes each."""
    kb = -(-cols // BLOCK)
    rb, kg = -(-rows // 128), -(-kb // 4)
    full = torch.zeros((rb * 128, kg * 4), dtype=torch.uint8, device=e8.device)
    full[:rows, :kb] = e8
    return full.view(rb, 4, 32, kg, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _unpack(s, rows, cols):
    kb = -(-cols // BLOCK)
    rb, kg = -(-rows // 128), -(-kb // 4)
    return s.view(rb, kg, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, kg * 4)[:rows, :kb]


def _weights(N, K, gen):
    """A layer's kept weights: E4M3 codes and the scales of their 128x128 blocks, repeated for each row."""
    w = torch.empty((N, K), dtype=torch.float32, device="cuda").normal_(0.0, 0.02, generator=gen).to(torch.bfloat16)
    e = _exponents(w.float(), "e4m3", BLOCK, BLOCK)
    q = _codes(N, K)
    q.copy_((w.float() * torch.exp2(_spread(e, BLOCK, BLOCK, N, K))).to(torch.float8_e4m3fn).view(torch.uint8))
    e8 = (127 - e).to(torch.uint8).repeat_interleave(BLOCK, 0)[:N]
    return q, _pack(e8, N, K)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M, N, dt = case["op"], case["M"], case["N"], DTYPES[case["dtype"]]
    s = {"case": case}
    new = lambda *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if op == "act":
        s["h"] = _activations(M, N, gen, dt)
        s["da"] = _gradients(M, N, gen, dt)
        s |= {"cq": _codes(M, N), "cs": _scales(M, N), "a": new(M, N), "dh": new(M, N)}
        return s
    K = case["K"]
    s["x"] = _activations(M, K, gen, dt)
    if op == "linear":
        s["wq"], s["ws"] = _weights(N, K, gen)
        s["bias"] = _normal((N,), 0.1, gen, dt)
        s |= {"xq": _codes(M, K), "xs": _scales(M, K), "y": new(M, N)}
        return s
    s |= {"xq": _codes(M, K), "xs": _scales(M, K), "xq_t": _codes(M, K), "xs_t": _scales(K, M)}
    if op == "step":
        s["w"] = _normal((N, K), 0.02, gen, dt)
        s["dy"] = _gradients(M, N, gen, dt)
        s |= {"wq": _codes(N, K), "ws": _scales(N, K), "ws_t": _scales(K, N)}
        s |= {"dyq": _codes(M, N), "dys": _scales(M, N), "dyq_t": _codes(M, N), "dys_t": _scales(N, M)}
        s |= {"y": new(M, N), "dx": new(M, K), "dw": new(N, K)}
        return s
    s["w1"], s["w2"] = _normal((N, K), 0.02, gen, dt), _normal((K, N), 0.02, gen, dt)
    s["dy"] = _gradients(M, K, gen, dt)
    s |= {"w1q": _codes(N, K), "w1s": _scales(N, K), "w1s_t": _scales(K, N)}
    s |= {"w2q": _codes(K, N), "w2s": _scales(K, N), "w2s_t": _scales(N, K)}
    s |= {"h": new(M, N), "cq": _codes(M, N), "cs": _scales(M, N), "aq": _codes(M, N), "as": _scales(M, N)}
    s |= {"dyq": _codes(M, K), "dys": _scales(M, K), "dyq_t": _codes(M, K), "dys_t": _scales(K, M), "da": new(M, N)}
    s |= {"dhq": _codes(M, N), "dhs": _scales(M, N), "dhq_t": _codes(M, N), "dhs_t": _scales(N, M)}
    s |= {"aq_t": _codes(M, N), "as_t": _scales(N, M)}
    s |= {"y": new(M, K), "dx": new(M, K), "dw1": new(N, K), "dw2": new(K, N)}
    return s


# ---------------------------------------------------------------- plain form (32 bits; 64 for the activation, see _toward)
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
    """The values that the codes and scales of x stand for, in x's own precision."""
    e = _spread(_exponents(x, fmt, br, bc), br, bc, *x.shape).to(x.dtype)
    v = x * torch.exp2(e)
    bits, low = (4, -5) if fmt == "e4m3" else (3, -13)  # significand bits; frexp's exponent of the smallest normal
    unit = torch.exp2((torch.frexp(v)[1].clamp_min(low) - bits).to(x.dtype))
    return torch.round(v / unit) * unit * torch.exp2(-e)


def _toward(v, base, r):
    """v = base + base * r with |r| too small to show: one unit off base, on r's side.  What is stored in few
    bits often lies on a rounding border, and a value just beside it must not be taken for the border itself."""
    inf = torch.full_like(v, math.inf)
    return torch.where((v == base) & (r != 0) & (base != 0), torch.nextafter(base, torch.where(base * r > 0, inf, -inf)), v)


def _gate(h, kind):
    """For act(h) = h * g(h): g, 1 - g and g' in 64 bits."""
    if kind == "gelu_erf":
        z = h * math.sqrt(0.5)
        return 0.5 * torch.erfc(-z), 0.5 * torch.erfc(z), torch.exp(-z * z) / math.sqrt(2.0 * math.pi)
    u, du = h, 1.0
    if kind == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        u, du = c * (h + 0.044715 * h * h * h), c * (1.0 + 3 * 0.044715 * h * h)
    g, q = 1.0 / (1.0 + torch.exp(-u)), 1.0 / (1.0 + torch.exp(u))
    return g, q, g * q * du


def _act(h, kind):
    """act(h), in 64 bits."""
    h = h.double()
    g, q, _ = _gate(h, kind)
    return torch.where(h > 0, _toward(h - h * q, h, -q), h * g)


def _act_grad(h, da, kind):
    """da * act'(h), in 64 bits; act' = g + h g' = 1 + r."""
    h, da = h.double(), da.double()
    g, q, dg = _gate(h, kind)
    r = h * dg - q
    return torch.where(h > 0, _toward(da + da * r, da, r), da * (g + h * dg))


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "act":
        kept = _rounded(s["h"].float(), "e4m3", 1, BLOCK)
        return {"a": _act(s["h"], case["act"]).to(dt), "dh": _act_grad(kept, s["da"], case["act"]).to(dt)}
    x = s["x"].float()
    if op == "linear":
        N, K = s["wq"].shape
        ws = torch.exp2(_unpack(s["ws"], N, K).float() - 127.0).repeat_interleave(BLOCK, 1)[:, :K]
        w = s["wq"].view(torch.float8_e4m3fn).float() * ws
        return {"y": (_rounded(x, "e4m3", 1, BLOCK) @ w.T + s["bias"].float()).to(dt)}
    f = case["grad"]
    dy = s["dy"].float()
    dy_r, dy_c = _rounded(dy, f, 1, BLOCK), _rounded(dy, f, BLOCK, 1)
    if op == "step":
        w = _rounded(s["w"].float(), "e4m3", BLOCK, BLOCK)
        return {"y": (_rounded(x, "e4m3", 1, BLOCK) @ w.T).to(dt), "dx": (dy_r @ w).to(dt),
                "dw": (dy_c.T @ _rounded(x, "e4m3", BLOCK, 1)).to(dt)}
    w1, w2 = (_rounded(s[k].float(), "e4m3", BLOCK, BLOCK) for k in ("w1", "w2"))
    h = (_rounded(x, "e4m3", 1, BLOCK) @ w1.T).to(dt).float()
    y = _rounded(_act(h, case["act"]), "e4m3", 1, BLOCK).float() @ w2.T
    kept = _rounded(h, "e4m3", 1, BLOCK)
    a_c = _rounded(_act(kept, case["act"]), "e4m3", BLOCK, 1).float()
    dh = _act_grad(kept, (dy_r @ w2).to(dt), case["act"])
    return {"y": y.to(dt), "dw2": (dy_c.T @ a_c).to(dt), "dx": (_rounded(dh, f, 1, BLOCK).float() @ w1).to(dt),
            "dw1": (_rounded(dh, f, BLOCK, 1).float().T @ _rounded(x, "e4m3", BLOCK, 1)).to(dt)}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from fp8_mixed_precision_tensor_b200 import fp8

    case = s["case"]
    op, E4M3 = case["op"], fp8.FP8_E4M3
    if op == "linear":
        if case["M"] <= fp8.FP8_BLOCK_TOKENS_MAX:
            fp8.fp8_block_linear_tokens(s["x"], s["wq"], s["ws"], s["y"], bias=s["bias"])
        else:
            fp8.fp8_block_cast(s["x"], E4M3, 0, s["xq"], s["xs"])
            fp8.fp8_block_linear_fwd(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], bias=s["bias"])
        return {"y": s["y"]}
    if op == "act":
        act = getattr(fp8, "FP8_ACT_" + case["act"].upper())
        fp8.fp8_act_fwd(s["h"], act, 0, s["cq"], s["cs"], a=s["a"])
        fp8.fp8_act_bwd(s["cq"], s["cs"], s["da"], act, dh=s["dh"])
        return {"a": s["a"], "dh": s["dh"]}
    fmt = fp8.FP8_E5M2 if case["grad"] == "e5m2" else E4M3
    if op == "step":
        fp8.fp8_block_cast(s["x"], E4M3, 0, s["xq"], s["xs"], s["xq_t"], s["xs_t"])
        fp8.fp8_block_cast(s["dy"], fmt, 0, s["dyq"], s["dys"], s["dyq_t"], s["dys_t"])
        fp8.fp8_block_cast_square(s["w"], E4M3, 0, s["wq"], s["ws"], s["ws_t"])
        fp8.fp8_block_linear_fwd(s["xq"], s["xs"], s["wq"], s["ws"], s["y"])
        fp8.fp8_block_linear_dgrad(s["dyq"], s["dys"], fmt, s["wq"], s["ws_t"], s["dx"])
        fp8.fp8_block_linear_wgrad(s["dyq_t"], s["dys_t"], fmt, s["xq_t"], s["xs_t"], s["dw"])
        return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    act = getattr(fp8, "FP8_ACT_" + case["act"].upper())
    fp8.fp8_block_cast_square(s["w1"], E4M3, 0, s["w1q"], s["w1s"], s["w1s_t"])
    fp8.fp8_block_cast_square(s["w2"], E4M3, 0, s["w2q"], s["w2s"], s["w2s_t"])
    fp8.fp8_block_cast(s["x"], E4M3, 0, s["xq"], s["xs"], s["xq_t"], s["xs_t"])
    fp8.fp8_block_linear_fwd(s["xq"], s["xs"], s["w1q"], s["w1s"], s["h"])
    fp8.fp8_act_fwd(s["h"], act, 0, s["cq"], s["cs"], s["aq"], s["as"])
    fp8.fp8_block_linear_fwd(s["aq"], s["as"], s["w2q"], s["w2s"], s["y"])
    fp8.fp8_block_cast(s["dy"], fmt, 0, s["dyq"], s["dys"], s["dyq_t"], s["dys_t"])
    fp8.fp8_block_linear_dgrad(s["dyq"], s["dys"], fmt, s["w2q"], s["w2s_t"], s["da"])
    fp8.fp8_act_bwd(s["cq"], s["cs"], s["da"], act, fmt, 0, s["dhq"], s["dhs"], s["dhq_t"], s["dhs_t"],
                    s["aq_t"], s["as_t"])
    fp8.fp8_block_linear_wgrad(s["dyq_t"], s["dys_t"], fmt, s["aq_t"], s["as_t"], s["dw2"])
    fp8.fp8_block_linear_dgrad(s["dhq"], s["dhs"], fmt, s["w1q"], s["w1s_t"], s["dx"])
    fp8.fp8_block_linear_wgrad(s["dhq_t"], s["dhs_t"], fmt, s["xq_t"], s["xs_t"], s["dw1"])
    return {"y": s["y"], "dx": s["dx"], "dw1": s["dw1"], "dw2": s["dw2"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definition
def _exact_values(x, fmt, br, bc):
    """x rounded to the format at its blocks' scales, every step in binary64.

    The scale is found by trial (the guess of a logarithm, moved until
    amax * s <= fmt_max < 2 * amax * s); the format's grid at a value has the
    spacing 2^(e - digits), e the value's exponent, not below the smallest
    normal one."""
    fmax = FMT_MAX[fmt]
    digits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    R, C = x.shape
    out = torch.zeros_like(x)
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
    torch.div(torch.round(v / step) * step, s, out=out)
    return out


def _exact_act(h, kind):
    """act(h), and act'(h) as a pair (d, d - 1): near 1 the second still tells the side."""
    if kind == "gelu_erf":
        upper = 0.5 * torch.special.erfc(h / math.sqrt(2.0))
        lower = 0.5 * torch.special.erfc(-h / math.sqrt(2.0))
        slope = torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)
    else:
        k = 2 * math.sqrt(2 / math.pi) if kind == "gelu_tanh" else 1.0
        c3 = 0.044715 if kind == "gelu_tanh" else 0.0
        u = k * (h + c3 * h ** 3)           # gelu_tanh: (1 + tanh(u / 2)) / 2 = sigmoid(u)
        lower, upper = torch.sigmoid(u), torch.sigmoid(-u)
        slope = lower * upper * k * (1 + 3 * c3 * h ** 2)
    a = h * lower
    # the true value is below h: never let it round up to h itself
    a = torch.where((h > 0) & (a >= h) & (upper > 0), torch.nextafter(h, torch.zeros_like(h)), a)
    return a, (lower + h * slope, h * slope - upper)


def _exact_product(da, d):
    """da * d, one unit off da where d is not 1 but rounds to it."""
    d, less1 = d
    p = da * d
    beside = torch.nextafter(da, torch.sign(less1) * torch.sign(da) * math.inf)
    return torch.where((d == 1) & (less1 != 0) & (da != 0), beside, p)


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "act":
        h = s["h"].double()
        d = _exact_act(_exact_values(h, "e4m3", 1, BLOCK), case["act"])[1]
        return {"a": _exact_act(h, case["act"])[0], "dh": _exact_product(s["da"].double(), d)}
    x = s["x"].double()
    if op == "linear":
        N, K = s["wq"].shape
        w = s["wq"].view(torch.float8_e4m3fn).double()
        for b in range(-(-K // BLOCK)):  # the scale byte of (row r, block b) by its address
            r = torch.arange(N, device="cuda")
            at = ((r // 128) * -(-K // 512) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
            w[:, b * BLOCK:(b + 1) * BLOCK] *= torch.exp2(s["ws"][at].double() - 127)[:, None]
        return {"y": torch.matmul(_exact_values(x, "e4m3", 1, BLOCK), w.T) + s["bias"].double()}
    f = case["grad"]
    dy = s["dy"].double()
    x_c = _exact_values(x, "e4m3", BLOCK, 1)
    if op == "step":
        w = _exact_values(s["w"].double(), "e4m3", BLOCK, BLOCK)
        return {"y": torch.matmul(_exact_values(x, "e4m3", 1, BLOCK), w.T),
                "dx": torch.matmul(_exact_values(dy, f, 1, BLOCK), w),
                "dw": torch.matmul(_exact_values(dy, f, BLOCK, 1).T, x_c)}
    w1 = _exact_values(s["w1"].double(), "e4m3", BLOCK, BLOCK)
    w2 = _exact_values(s["w2"].double(), "e4m3", BLOCK, BLOCK)
    # the layer outputs h and da are stored in the tensors' own type
    h = torch.matmul(_exact_values(x, "e4m3", 1, BLOCK), w1.T).to(dt).double()
    y = torch.matmul(_exact_values(_exact_act(h, case["act"])[0], "e4m3", 1, BLOCK), w2.T)
    a, d = _exact_act(_exact_values(h, "e4m3", 1, BLOCK), case["act"])
    dh = _exact_product(torch.matmul(_exact_values(dy, f, 1, BLOCK), w2).to(dt).double(), d)
    return {"y": y, "dw2": torch.matmul(_exact_values(dy, f, BLOCK, 1).T, _exact_values(a, "e4m3", BLOCK, 1)),
            "dx": torch.matmul(_exact_values(dh, f, 1, BLOCK), w1),
            "dw1": torch.matmul(_exact_values(dh, f, BLOCK, 1).T, x_c)}
