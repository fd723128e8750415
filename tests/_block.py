"""References of the block-scaled operators in binary64 (numpy and torch on the
CPU), written from the definitions: block scales, FP8 rounding, the scale
bytes' addresses, products and activation functions."""
import math

import numpy as np
import torch

import oracle

FMT = {"e4m3": (oracle.E4M3, 448.0, 3, -6), "e5m2": (oracle.E5M2, 57344.0, 2, -14)}


def blocks_of(x: np.ndarray, br: int, bc: int) -> np.ndarray:
    """amax of every br x bc block of x (NaN wins, then inf)."""
    R, C = x.shape
    out = np.zeros((-(-R // br), -(-C // bc)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.max(np.abs(x[i * br:(i + 1) * br, j * bc:(j + 1) * bc]))
    return out


def exponents(amax: np.ndarray, fmt: str, margin: int = 0) -> np.ndarray:
    """k of the scales 2^k, by exact comparison of amax * 2^e with fmt_max."""
    fmax = FMT[fmt][1]
    k = np.zeros(amax.shape, dtype=np.int64)
    for i, a in np.ndenumerate(amax):
        if a == 0 or not np.isfinite(a):
            continue
        e = int(math.floor(math.log2(fmax) - math.log2(a)))
        while math.ldexp(a, e) > fmax:
            e -= 1
        while math.ldexp(a, e + 1) <= fmax:
            e += 1
        k[i] = min(126, max(-126, e - margin))
    return k


def spread(k: np.ndarray, br: int, bc: int, shape) -> np.ndarray:
    return np.repeat(np.repeat(k, br, 0), bc, 1)[:shape[0], :shape[1]]


def round_fp8(v: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest value of the format (ties to even, saturating); v in binary64."""
    _, fmax, digits, low = FMT[fmt]
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** (low - 1)))), low)
    step = np.exp2(e - digits)
    return np.copysign(np.minimum(np.round(a / step) * step, fmax), v)


def cast_values(x: np.ndarray, fmt: str, br: int, bc: int, margin: int = 0):
    """(values that the codes stand for, exponents k per block), finite x."""
    x = x.astype(np.float64)
    k = exponents(blocks_of(x, br, bc), fmt, margin)
    s = np.exp2(spread(k, br, bc, x.shape).astype(np.float64))
    return round_fp8(x * s, fmt) / s, k


def scale_address(r, b, red: int):
    return ((r // 128) * (-(-(-(-red // 128)) // 4)) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def packed(k_rows: np.ndarray, outer: int, red: int) -> np.ndarray:
    """Scale bytes of exponents k_rows [outer, ceil(red / 128)] at their addresses; padding 127."""
    kb = -(-red // 128)
    out = np.full(-(-outer // 128) * -(-kb // 4) * 512, 127, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(outer), np.arange(kb), indexing="ij")
    out[scale_address(r, b, red)] = (127 - k_rows).astype(np.uint8)
    return out


def codes_of(values: np.ndarray, k_spread: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of already representable values."""
    table = oracle.decode_table(FMT[fmt][0])
    back = {}
    for c in range(256):
        if np.isfinite(table[c]) and abs(table[c]) <= FMT[fmt][1]:
            back.setdefault((float(table[c]), bool(np.signbit(table[c]))), c)
    v = values * np.exp2(k_spread.astype(np.float64))
    return np.array([back[(float(t), bool(np.signbit(t)))] for t in v.reshape(-1)], dtype=np.uint8).reshape(v.shape)


# ---------------------------------------------------------------- activations
def act_parts(h: np.ndarray, kind: str):
    """act(h), act'(h) in binary64."""
    t = torch.from_numpy(np.ascontiguousarray(h, dtype=np.float64))
    if kind == "silu":
        g = torch.sigmoid(t)
        a, d = t * g, g + t * g * torch.sigmoid(-t)
    elif kind == "gelu_erf":
        g = 0.5 * torch.special.erfc(-t / math.sqrt(2.0))
        a, d = t * g, g + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    else:
        c = math.sqrt(2 / math.pi)
        u = 2 * c * (t + 0.044715 * t ** 3)
        g = torch.sigmoid(u)
        a, d = t * g, g + t * g * torch.sigmoid(-u) * 2 * c * (1 + 3 * 0.044715 * t * t)
    return a.numpy(), d.numpy()


def act_strict(h: np.ndarray, kind: str) -> np.ndarray:
    """act(h) in binary64, below h for every h > 0 as the function is (also
    where the difference is less than binary64 shows): what decides a tie."""
    a = act_parts(h, kind)[0]
    return np.where((h > 0) & (a >= h), np.nextafter(h, 0), a)


def act_grad_strict(h: np.ndarray, da: np.ndarray, kind: str) -> np.ndarray:
    """da * act'(h) in binary64, beside da (act' is above 1 for every large h) where act' rounds to 1."""
    d = act_parts(h, kind)[1]
    return np.where((h > 4) & (d == 1), np.nextafter(da, np.copysign(np.inf, da)) * (da != 0), da * d)
