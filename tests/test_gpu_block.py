"""Block-scaled FP8 casts, products and activation checkpoints on the GPU
against binary64 references (tests/_block.py).

Tolerances.  Codes and scales of a cast are exact.  A product: the tensor core
multiplies FP8 values exactly, scales by powers of two exactly and adds in
binary32; `red + 32` additions, each off by at most one unit (2^-23, as it may
truncate) of a partial sum that is at most sum |a b|, then the bias add and the
rounding to the output type.  Activations: stated at `_act_tolerance`.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from fp8_mixed_precision_tensor_b200 import fp8, synth
from fp8_mixed_precision_tensor_b200.block_linear import BlockLinear, BlockMLP
from _block import act_grad_strict, act_parts, act_strict, blocks_of, cast_values, codes_of, exponents, packed, round_fp8, spread
from _util import half_ulp_out

pytestmark = pytest.mark.gpu

FMTS = {"e4m3": fp8.FP8_E4M3, "e5m2": fp8.FP8_E5M2}
ACTS = {"gelu_tanh": fp8.FP8_ACT_GELU_TANH, "gelu_erf": fp8.FP8_ACT_GELU_ERF, "silu": fp8.FP8_ACT_SILU}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
GUARD = 0xA5


def data(rows, cols, *key, std=1.0, zeros=True):
    """Normal values over many magnitudes, an outlier column and all-zero rows (float32)."""
    g = synth.rng("block", rows, cols, *key)
    x = g.standard_normal((rows, cols)).astype(np.float32) * np.exp2(g.integers(-6, 7, (rows, cols))).astype(np.float32)
    x[:, g.integers(0, cols)] *= 256.0
    if zeros and rows > 2:
        x[rows // 2] = 0.0
    return (x * np.float32(std)).astype(np.float32)


def dev(x, dtype, ld=None, offset=0):
    """x on the device in dtype, rows ld elements apart, the first one `offset` elements into the buffer."""
    rows, cols = x.shape
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 8,), float("nan"), dtype=dtype, device="cuda")
    t = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    t.copy_(torch.from_numpy(x))
    return t


def f64(t):
    return t.double().cpu().numpy()


class Guarded:
    """A code matrix [rows, cols] with rows `ld` bytes apart, and its scales, every other byte a pattern."""

    def __init__(self, rows, cols, outer, red, ld=None):
        self.rows, self.cols = rows, cols
        self.ld = -(-cols // 16) * 16 if ld is None else ld
        self.raw = torch.full((64 + rows * self.ld + 64,), GUARD, dtype=torch.uint8, device="cuda")
        self.q = self.raw[64:64 + rows * self.ld].view(rows, self.ld)[:, :cols]
        n = fp8.fp8_block_scale_bytes(outer, red)
        self.sraw = torch.full((64 + n + 64,), GUARD, dtype=torch.uint8, device="cuda")
        self.s = self.sraw[64:64 + n]

    def intact(self):
        body = self.raw[64:64 + self.rows * self.ld].view(self.rows, self.ld)
        edge = torch.cat([self.raw[:64], self.raw[64 + self.rows * self.ld:], body[:, self.cols:].reshape(-1),
                          self.sraw[:64], self.sraw[-64:]])
        return bool((edge == GUARD).all())


def row_blocks(rows, cols, ld=None):
    return Guarded(rows, cols, rows, cols, ld)


def col_blocks(rows, cols, ld=None):
    return Guarded(rows, cols, cols, rows, ld)


def check_codes(b, x, fmt, br, bc, margin=0, what=""):
    """b's codes and scale bytes are exactly those of x's br x bc blocks; returns their values."""
    v, k = cast_values(x, fmt, br, bc, margin)
    ks = spread(k, br, bc, x.shape)
    assert np.array_equal(b.q.cpu().numpy(), codes_of(v, ks, fmt)), what
    rows, cols = x.shape
    if bc == 1:
        want = packed(k.T, cols, rows)
    else:
        want = packed(np.repeat(k, br, 0)[:rows], rows, cols)
    assert np.array_equal(b.s.cpu().numpy(), want), what
    assert b.intact(), what
    return v


# ---------------------------------------------------------------- casts
SHAPES = [(1, 1), (1, 128), (3, 300), (128, 128), (129, 257), (260, 1040), (513, 130)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_cast_is_exact_and_writes_only_its_outputs(shape, dtype, fmt):
    R, C = shape
    x = dev(data(R, C, "cast"), dtype)
    xs = f64(x)
    r, c = row_blocks(R, C), col_blocks(R, C)
    fp8.fp8_block_cast(x, FMTS[fmt], 0, r.q, r.s, c.q, c.s)
    check_codes(r, xs, fmt, 1, 128, what="rows")
    check_codes(c, xs, fmt, 128, 1, what="columns")
    r1, c1 = row_blocks(R, C), col_blocks(R, C)  # one side at a time, with a margin
    fp8.fp8_block_cast(x, FMTS[fmt], 3, r1.q, r1.s)
    fp8.fp8_block_cast(x, FMTS[fmt], 3, q_col=c1.q, s_col=c1.s)
    check_codes(r1, xs, fmt, 1, 128, 3)
    check_codes(c1, xs, fmt, 128, 1, 3)
    s, s_col = row_blocks(R, C), col_blocks(R, C)
    fp8.fp8_block_cast_square(x, FMTS[fmt], 0, s.q, s.s, s_col.s)
    check_codes(s, xs, fmt, 128, 128)
    k = exponents(blocks_of(xs, 128, 128), fmt)
    assert np.array_equal(s_col.s.cpu().numpy(), packed(np.repeat(k.T, 128, 0)[:C], C, R)) and s_col.intact()
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ld,offset", [(208, 0), (208, 8), (203, 0), (201, 3)])
def test_cast_of_strided_and_unaligned_rows(ld, offset, dtype):
    x = dev(data(150, 200, "strided", ld), dtype, ld, offset)
    r, c = row_blocks(150, 200, 256), col_blocks(150, 200, 224)
    fp8.fp8_block_cast(x, fp8.FP8_E4M3, 0, r.q, r.s, c.q, c.s)
    check_codes(r, f64(x), "e4m3", 1, 128)
    check_codes(c, f64(x), "e4m3", 128, 1)


def test_cast_at_the_ends_of_the_range_and_on_thresholds():
    x = np.zeros((8, 256), dtype=np.float32)
    x[0, 0] = 448.0                                  # exactly on a threshold
    x[0, 128] = np.nextafter(np.float32(448), np.float32(1e9))
    x[1, :128] = np.float32(2.0 ** -149)             # the clamp of the exponent
    x[2, :128] = np.linspace(1, 3.3e38, 128, dtype=np.float32)
    x[3, :] = np.linspace(-1, 1, 256, dtype=np.float32)
    x[4, :128] = -0.0
    x[5, :] = np.float32(1.0625) * np.exp2(np.arange(256) % 20 - 10).astype(np.float32)  # ties
    for fmt in ("e4m3", "e5m2"):
        r, c = row_blocks(8, 256), col_blocks(8, 256)
        t = dev(x, F32)
        fp8.fp8_block_cast(t, FMTS[fmt], 0, r.q, r.s, c.q, c.s)
        check_codes(r, x.astype(np.float64), fmt, 1, 128)
        check_codes(c, x.astype(np.float64), fmt, 128, 1)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_non_finite_value_stays_in_its_block(bad):
    clean = data(140, 300, "nonfinite")
    x = clean.copy()
    x[70, 200] = bad
    r0, c0, r, c = row_blocks(140, 300), col_blocks(140, 300), row_blocks(140, 300), col_blocks(140, 300)
    fp8.fp8_block_cast(dev(clean, F32), fp8.FP8_E4M3, 0, r0.q, r0.s, c0.q, c0.s)
    assert fp8.fp8_get_status() == 0
    fp8.fp8_block_cast(dev(x, F32), fp8.FP8_E4M3, 0, r.q, r.s, c.q, c.s)
    assert fp8.fp8_get_status() == fp8.FP8_STATUS_NONFINITE
    code = 0x7F if np.isnan(bad) else (0x7E if bad > 0 else 0xFE)
    for got, ref, rows, cols in ((r, r0, slice(70, 71), slice(128, 256)), (c, c0, slice(0, 128), slice(200, 201))):
        q, q0 = got.q.cpu().numpy(), ref.q.cpu().numpy()
        assert q[70, 200] == code
        own = np.zeros(q.shape, dtype=bool)
        own[rows, cols] = True
        assert np.array_equal(q[~own], q0[~own])
        blk = x[rows, cols].astype(np.float64)
        fin = np.isfinite(blk)
        assert np.array_equal(codes_of(round_fp8(blk[fin], "e4m3"), np.zeros(fin.sum()), "e4m3"), q[rows, cols][fin])
        assert np.count_nonzero(got.s.cpu().numpy() != ref.s.cpu().numpy()) <= 1


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_decode_gives_the_codes_values(fmt, dtype):
    for R, C in SHAPES:
        x = dev(data(R, C, "decode", std=1e-3), F32)
        r, c = row_blocks(R, C), col_blocks(R, C)
        fp8.fp8_block_cast(x, FMTS[fmt], 0, r.q, r.s, c.q, c.s)
        for b, axis, br, bc in ((r, 1, 1, 128), (c, 0, 128, 1)):
            out = dev(np.zeros((R, C), dtype=np.float32), dtype, C + 5, 1)
            fp8.fp8_block_decode(b.q, b.s, FMTS[fmt], axis, out)
            want = torch.from_numpy(cast_values(f64(x), fmt, br, bc)[0]).to(dtype)
            assert torch.equal(out.cpu(), want), (R, C, axis)


def test_offsets_past_32_bits():
    """Casts and products whose last rows lie beyond 2^31 elements give what those rows give alone."""
    R, C = 70016, 32768
    x = torch.zeros((R, C), dtype=BF16, device="cuda")
    x[-300:] = torch.from_numpy(data(300, C, "far")).to(BF16).cuda()
    q, s, qc, sc = (fp8.block_codes(R, C), fp8.block_scales(R, C), fp8.block_codes(R, C), fp8.block_scales(C, R))
    fp8.fp8_block_cast(x, fp8.FP8_E4M3, 0, q, s, qc, sc)
    r = row_blocks(300, C)
    fp8.fp8_block_cast(x[-300:].contiguous(), fp8.FP8_E4M3, 0, r.q, r.s)
    assert torch.equal(q[-300:], r.q) and int(q[:-300].max()) == 0
    tail = x[R // 128 * 128 - 128:].float()
    out = torch.empty((R, C), dtype=BF16, device="cuda")
    fp8.fp8_block_decode(qc, sc, fp8.FP8_E4M3, 0, out)
    ref = cast_values(f64(tail[:, :64]), "e4m3", 128, 1)[0]
    assert np.array_equal(f64(out[R // 128 * 128 - 128:, :64]), ref)
    del x, qc, sc, out
    wq, ws, ws_col = fp8.block_codes(C, 128), fp8.block_scales(C, 128), fp8.block_scales(128, C)
    fp8.fp8_block_cast_square(torch.from_numpy(data(C, 128, "farw")).cuda(), fp8.FP8_E4M3, 0, wq, ws, ws_col)
    xq, xs = q[:, :128], fp8.block_scales(R, 128)
    fp8.fp8_block_cast(torch.randn(R, 128, device="cuda"), fp8.FP8_E4M3, 0, xq, xs)
    y = torch.empty((R, C), dtype=BF16, device="cuda")
    fp8.fp8_block_linear_fwd(xq, xs, wq, ws, y)
    at = R // 128 * 128 - 128
    ya = torch.empty((R - at, C), dtype=BF16, device="cuda")
    fp8.fp8_block_linear_fwd(xq[at:], xs[at // 128 * 512:], wq, ws, ya)
    assert torch.equal(y[at:], ya) and fp8.fp8_get_status() == 0


# ---------------------------------------------------------------- products
class Layer:
    """Operands of one layer (float32 sources), their codes, and the values these stand for."""

    def __init__(self, M, N, K, grad="e5m2", key=()):
        self.M, self.N, self.K, self.grad = M, N, K, FMTS[grad]
        x, w, dy = data(M, K, "x", *key), data(N, K, "w", *key, std=0.02), data(M, N, "dy", *key, std=1e-4)
        C, S = fp8.block_codes, fp8.block_scales
        self.xq, self.xs, self.xqc, self.xsc = C(M, K), S(M, K), C(M, K), S(K, M)
        self.gq, self.gs, self.gqc, self.gsc = C(M, N), S(M, N), C(M, N), S(N, M)
        self.wq, self.ws, self.wsc = C(N, K), S(N, K), S(K, N)
        self.x = dev(x, F32)
        fp8.fp8_block_cast(self.x, fp8.FP8_E4M3, 0, self.xq, self.xs, self.xqc, self.xsc)
        fp8.fp8_block_cast(dev(dy, F32), self.grad, 0, self.gq, self.gs, self.gqc, self.gsc)
        fp8.fp8_block_cast_square(dev(w, F32), fp8.FP8_E4M3, 0, self.wq, self.ws, self.wsc)
        val = lambda q, s, f, ax, shape: self._values(q, s, f, ax, shape)  # noqa: E731
        self.X, self.Xc = val(self.xq, self.xs, 0, 1, (M, K)), val(self.xqc, self.xsc, 0, 0, (M, K))
        self.G, self.Gc = val(self.gq, self.gs, self.grad, 1, (M, N)), val(self.gqc, self.gsc, self.grad, 0, (M, N))
        self.W = val(self.wq, self.ws, 0, 1, (N, K))

    @staticmethod
    def _values(q, s, fmt, axis, shape):
        out = torch.empty(shape, dtype=F32, device="cuda")
        fp8.fp8_block_decode(q, s, fmt, axis, out)
        return out.double()

    def references(self, bias=None):
        b = 0 if bias is None else bias.double()
        return {"y": (self.X @ self.W.T + b, self.X.abs() @ self.W.abs().T + (0 if bias is None else b.abs()), self.K),
                "dx": (self.G @ self.W, self.G.abs() @ self.W.abs(), self.N),
                "dw": (self.Gc.T @ self.Xc, self.Gc.abs().T @ self.Xc.abs(), self.M)}


def assert_product(out, ref, what=""):
    exact, mag, red = ref
    bound = (red + 32) * 2.0 ** -23 * mag
    got = out.double()
    if out.dtype == F32:
        bound = bound + 2.0 ** -24 * exact.abs()
    else:
        bound = bound + torch.from_numpy(half_ulp_out(exact.abs().cpu().numpy() + bound.cpu().numpy(), out.dtype)).cuda()
    if out.dtype == F16:  # values from 65520 on round to infinity
        must, may = exact.abs() - bound >= 65520, exact.abs() + bound >= 65520
        over = got.isinf()
        assert bool((over | ~must).all()) and bool((may | ~over).all()), what
        got = torch.where(over & (got.sign() == exact.sign()), exact, got)
    off = (got - exact).abs() - bound
    assert torch.isfinite(got).all() and float(off.max()) <= 0, (what, float(off.max()), exact.shape)


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 300, 1000), (7, 129, 65), (33, 512, 256), (128, 256, 512), (129, 257, 385),
            (300, 520, 2056), (513, 1305, 1001), (1024, 640, 4112), (2560, 2560, 384), (2309, 4871, 700)]


@pytest.mark.parametrize("grad", ["e5m2", "e4m3"])
@pytest.mark.parametrize("shape", PRODUCTS)
def test_products_against_binary64(shape, grad):
    M, N, K = shape
    L = Layer(M, N, K, grad)
    bias = torch.randn(N, device="cuda").to(BF16)
    ref = L.references(bias)
    for dtype in (F32, BF16):
        y, dx, dw = (dev(np.full(s, 7.0, np.float32), dtype) for s in ((M, N), (M, K), (N, K)))
        fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y, bias=bias)
        fp8.fp8_block_linear_dgrad(L.gq, L.gs, L.grad, L.wq, L.wsc, dx)
        fp8.fp8_block_linear_wgrad(L.gqc, L.gsc, L.grad, L.xqc, L.xsc, dw)
        for name, out in (("y", y), ("dx", dx), ("dw", dw)):
            assert_product(out, ref[name], (name, dtype))
        again = torch.empty_like(dw)
        fp8.fp8_block_linear_wgrad(L.gqc, L.gsc, L.grad, L.xqc, L.xsc, again)
        assert torch.equal(again, dw)  # the same bits each time
    assert fp8.fp8_get_status() == 0


# A long reduction behind few output tiles, in turn in y, dx and dw: one to
# eight CTAs share a tile, with the last tiles and blocks cut short.
FEW_TILES = [(65, 100, 1100), (130, 260, 9000), (200, 9000, 136), (8200, 130, 257), (65, 7000, 12300), (777, 1305, 4100),
             (1024, 1024, 4096), (1500, 1100, 8200), (129, 12000, 300)]


@pytest.mark.parametrize("shape", FEW_TILES)
def test_long_reductions_of_few_tiles(shape):
    M, N, K = shape
    L = Layer(M, N, K)
    bias = torch.randn(N, device="cuda")
    ref = L.references(bias)
    for dtype, pad in ((BF16, 0), (F16, 3), (F32, 1)):
        y, dx, dw = (torch.full((r, c + pad), 7.0, dtype=dtype, device="cuda") for r, c in ((M, N), (M, K), (N, K)))
        for _ in range(2):
            fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y[:, :N], bias=bias)
            fp8.fp8_block_linear_dgrad(L.gq, L.gs, L.grad, L.wq, L.wsc, dx[:, :K])
            fp8.fp8_block_linear_wgrad(L.gqc, L.gsc, L.grad, L.xqc, L.xsc, dw[:, :K])
        for name, out, n in (("y", y, N), ("dx", dx, K), ("dw", dw, K)):
            assert_product(out[:, :n], ref[name], (name, dtype))
            assert bool((out[:, n:] == 7.0).all()), name
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("shape", [(5, 260, 200), (200, 260, 200), (2309, 4871, 256)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16, "rto"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 0), (0, 1)])
def test_output_types_and_pitches(shape, dtype, pad, offset):
    M, N, K = shape
    L = Layer(M, N, K)
    rto, dt = dtype == "rto", BF16 if dtype == "rto" else dtype
    ref = L.references()["y"]
    buf = torch.full((offset + M * (N + pad) + 16,), 3.0, dtype=dt, device="cuda")
    y = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y, rto=rto)
    if rto:  # the round-to-odd image of the float32 output
        y32 = torch.empty((M, N), dtype=F32, device="cuda")
        fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y32)
        bits = y32.view(torch.int32)
        want = ((bits >> 16) | ((bits & 0xffff) != 0)).to(torch.int16)
        assert torch.equal(y.contiguous().view(torch.int16), want)
    else:
        assert_product(y, ref)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N] = False
    assert bool((buf[rest] == 3.0).all())


@pytest.mark.parametrize("bias_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(20, 300, 200), (300, 700, 520), (2309, 4871, 200)])
def test_bias_types(shape, bias_dtype):
    M, N, K = shape
    L = Layer(M, N, K)
    bias = torch.randn(N + 1, device="cuda").to(bias_dtype)[1:]  # (at any element's alignment)
    ref = L.references(bias)["y"]
    for dtype in (F32, BF16):
        y = torch.empty((M, N), device="cuda", dtype=dtype)
        fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y, bias=bias)
        assert_product(y, ref, (dtype, bias_dtype))


def test_products_with_empty_sides():
    bias = torch.randn(40, device="cuda")
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    z = lambda r, c: fp8.block_codes(r, c)  # noqa: E731
    y = torch.full((3, 40), 5.0, device="cuda")
    fp8.fp8_block_linear_fwd(z(3, 0), e, z(40, 0), e, y, bias=bias)
    assert torch.equal(y, bias.expand(3, 40))
    dw = torch.full((40, 20), 5.0, device="cuda", dtype=BF16)
    fp8.fp8_block_linear_wgrad(z(0, 40), e, fp8.FP8_E5M2, z(0, 20), e, dw)
    assert int(dw.count_nonzero()) == 0
    x0 = torch.empty((0, 20), device="cuda", dtype=BF16)
    w, ws = z(40, 20), fp8.block_scales(40, 20)
    fp8.fp8_block_linear_tokens(x0, w, ws, torch.empty((0, 40), device="cuda"))
    fp8.fp8_block_linear_tokens(torch.empty((2, 0), device="cuda"), z(40, 0), e, y[:2], bias=bias)
    assert torch.equal(y[:2], bias.expand(2, 40))
    fp8.fp8_block_cast(x0, fp8.FP8_E4M3, 0, z(0, 20), e)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M", [1, 2, 9, 16, 31, 32])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (300, 1000), (1024, 4096), (4100, 520)])
def test_tokens_form_against_binary64(M, N, K, dtype):
    L = Layer(M, N, K)
    x = dev(data(M, K, "tok"), dtype, K + (8 if K % 8 == 0 else 3))
    X = torch.from_numpy(cast_values(f64(x), "e4m3", 1, 128)[0]).cuda()
    bias = torch.randn(N, device="cuda")
    exact, mag = X @ L.W.T + bias.double(), X.abs() @ L.W.abs().T + bias.double().abs()
    for out in (dtype, F32):
        y = dev(np.full((M, N), 9.0, np.float32), out, N + 1)
        fp8.fp8_block_linear_tokens(x, L.wq, L.ws, y, bias=bias)
        assert_product(y, (exact, mag, K))
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("M", [1, 8, 9, 17, 32])
@pytest.mark.parametrize("N,K", [(19000, 3000), (12288, 4096), (300, 33000), (128, 70000)])
def test_tokens_form_runs_its_ring_many_times(M, N, K):
    """Reductions much longer than the kernel's ring of operand stages, on one CTA per tile and split."""
    L = Layer(M, N, K, key=("ring",))
    y = torch.empty((M, N), device="cuda")
    for _ in range(5):
        y.fill_(float("nan"))
        fp8.fp8_block_linear_tokens(L.x, L.wq, L.ws, y)
        assert_product(y, (L.X @ L.W.T, L.X.abs() @ L.W.abs().T, K))
    assert fp8.fp8_get_status() == 0


def test_tokens_form_reports_a_non_finite_token():
    L = Layer(4, 256, 256)
    x = torch.randn(4, 256, device="cuda")
    y0, y = torch.empty((4, 256), device="cuda"), torch.empty((4, 256), device="cuda")
    fp8.fp8_block_linear_tokens(x, L.wq, L.ws, y0)
    x[2, 5] = float("nan")
    fp8.fp8_block_linear_tokens(x, L.wq, L.ws, y)
    assert fp8.fp8_get_status() == fp8.FP8_STATUS_NONFINITE
    assert bool(y[2].isnan().all()) and torch.equal(y[[0, 1, 3]], y0[[0, 1, 3]])


def test_extreme_scales_multiply_exactly():
    """One value per block at both ends of the exponents: the descale is applied, not lost."""
    x = torch.zeros((2, 256), device="cuda")
    w = torch.zeros((16, 256), device="cuda")
    x[0, 0], x[0, 128], x[1, 0] = 2.0 ** 100, 2.0 ** -100, 2.0 ** -60
    w[:, 0], w[:, 128] = 2.0 ** -90, 2.0 ** 110
    C, S = fp8.block_codes, fp8.block_scales
    xq, xs, wq, ws = C(2, 256), S(2, 256), C(16, 256), S(16, 256)
    fp8.fp8_block_cast(x, 0, 0, xq, xs)
    fp8.fp8_block_cast(w, 0, 0, wq, ws)
    y = torch.empty((2, 16), device="cuda")
    fp8.fp8_block_linear_fwd(xq, xs, wq, ws, y)
    assert bool((y[0] == 2.0 ** 10 + 2.0 ** 10).all()) and bool((y[1] == 2.0 ** -150 * 2 ** 1 / 2).all())


# ---------------------------------------------------------------- activations
def _act_tolerance(h, kind):
    """Bound of |act - exact| and of |act' - exact| in binary32.  The gate's
    argument u carries a few roundings, relative 2^-22 of |u|; exp and the
    reciprocal add 4 + 1.2 |u| units of 2^-24; the gate (or 1 - gate, the
    small one) is therefore off by a factor within (2 |u| + 8) 2^-22 with |u|
    at most 100 where it has not underflowed, and by 2^-126 where it has; erfc
    is within 4 units and its argument's rounding is another |h|^2 units.
    Products with h and g' add two more."""
    u = np.abs(h) * (1 if kind == "silu" else 1.6 * (1 + 0.045 * h * h)) if kind != "gelu_erf" else h * h
    return (2 * np.minimum(u, 100) + 12) * 2.0 ** -22


def act_bounds(h, kind):
    a, d = act_parts(h, kind)
    t = _act_tolerance(h, kind)
    q = np.abs(1 - act_parts(h, kind)[0] / np.where(h == 0, 1, h))     # 1 - g
    g = 1 - q
    small = np.minimum(np.abs(q), np.abs(g)) + 2.0 ** -30
    # an underflowed gate is off by at most 2^-126, its factor |h| limited to 110
    flush = 110 * 2.0 ** -126
    e = 1e-4
    dg = np.abs(act_parts(h + e, kind)[0] / np.where(h + e == 0, 1, h + e) - a / np.where(h == 0, 1, h)) / e + 1e-3
    # act: g is off by `t` of the smaller of g, 1 - g; act' also by h g' and its error
    return a, d, np.abs(h) * small * t + np.abs(a) * 2.0 ** -22 + flush, (small + np.abs(h) * dg) * t + np.abs(d) * 2.0 ** -22 + 1e-37


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(1, 1), (3, 300), (130, 257), (257, 1024)])
def test_activation_forward(shape, dtype, kind):
    R, C = shape
    x = data(R, C, "act", std=0.25)
    x[0, :: 7] = np.linspace(-30, 30, len(x[0, :: 7]))
    h = dev(x, dtype, C + 3 if C % 2 else None)
    hs = f64(h)
    ck, aq, a = row_blocks(R, C), row_blocks(R, C), dev(np.zeros((R, C), np.float32), dtype)
    fp8.fp8_act_fwd(h, ACTS[kind], 0, ck.q, ck.s, aq.q, aq.s, a)
    check_codes(ck, hs, "e4m3", 1, 128)
    want, _, tol, _ = act_bounds(hs, kind)
    extra = half_ulp_out(np.abs(want) + tol, dtype) if dtype != F32 else 0
    assert np.all(np.abs(f64(a) - want) <= tol + extra)
    check_near_codes(aq, want, tol, "e4m3", 1, 128)
    ck2 = row_blocks(R, C)  # the checkpoint alone is the same
    fp8.fp8_act_fwd(h, ACTS[kind], 0, ck2.q, ck2.s)
    assert torch.equal(ck2.q, ck.q) and torch.equal(ck2.s, ck.s)
    assert fp8.fp8_get_status() == 0


def check_near_codes(b, want, tol, fmt, br, bc):
    """Codes of values known to within tol: each block's scale that of an amax
    within tol of the exact one, each code that of a value within tol."""
    R, C = want.shape
    axis = 0 if bc == 1 else 1
    out = torch.empty((R, C), dtype=F32, device="cuda")
    fp8.fp8_block_decode(b.q, b.s, FMTS[fmt], axis, out)
    lo_k = exponents(blocks_of(np.abs(want) + tol, br, bc), fmt)
    hi_k = exponents(blocks_of(np.maximum(np.abs(want) - tol, 0), br, bc), fmt)
    outer = C if bc == 1 else R
    red = R if bc == 1 else C
    got = b.s.cpu().numpy()
    r, j = np.meshgrid(np.arange(outer), np.arange(-(-red // 128)), indexing="ij")
    from _block import scale_address
    k = 127 - got[scale_address(r, j, red)].astype(np.int64)
    k = k.T if bc == 1 else k
    if br > 1 and bc > 1:
        raise AssertionError("square blocks are exact casts")
    # an amax that may be zero either way leaves the scale open
    open_ = blocks_of(np.maximum(np.abs(want) - tol, 0), br, bc) == 0
    assert np.all(open_ | ((k >= np.minimum(lo_k, hi_k)) & (k <= np.maximum(lo_k, hi_k))))
    s = np.exp2(spread(k, br, bc, want.shape).astype(np.float64))
    lo, hi = round_fp8((want - tol) * s, fmt) / s, round_fp8((want + tol) * s, fmt) / s
    v = f64(out)
    assert np.all((v >= lo) & (v <= hi))
    assert b.intact()


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("dtype,fmt", [(F32, "e5m2"), (BF16, "e5m2"), (BF16, "e4m3"), (F16, "e4m3")])
@pytest.mark.parametrize("shape", [(1, 1), (3, 300), (130, 257), (300, 640)])
def test_activation_backward(shape, dtype, fmt, kind):
    R, C = shape
    x = data(R, C, "actb", std=0.25)
    x[0, :: 7] = np.linspace(-30, 30, len(x[0, :: 7]))
    h = dev(x, F32)
    ck = row_blocks(R, C)
    fp8.fp8_act_fwd(h, ACTS[kind], 0, ck.q, ck.s)
    kept = cast_values(f64(h), "e4m3", 1, 128)[0]
    da = dev(data(R, C, "da", std=0.01), dtype, C + 3 if C % 2 else None)
    das = f64(da)
    dh, r, c, ac = dev(np.zeros((R, C), np.float32), dtype), row_blocks(R, C), col_blocks(R, C), col_blocks(R, C)
    fp8.fp8_act_bwd(ck.q, ck.s, da, ACTS[kind], FMTS[fmt], 0, r.q, r.s, c.q, c.s, ac.q, ac.s, dh)
    a, d, tol_a, tol_d = act_bounds(kept, kind)
    want, tol = das * d, np.abs(das) * tol_d + 1e-40
    extra = half_ulp_out(np.abs(want) + tol, dtype) if dtype != F32 else 0
    assert np.all(np.abs(f64(dh) - want) <= tol + extra)
    check_near_codes(r, want, tol, fmt, 1, 128)
    check_near_codes(c, want, tol, fmt, 128, 1)
    check_near_codes(ac, a, tol_a, "e4m3", 128, 1)
    # each output alone is the same
    dh1, r1, c1, a1 = torch.empty_like(dh), row_blocks(R, C), col_blocks(R, C), col_blocks(R, C)
    fp8.fp8_act_bwd(ck.q, ck.s, da, ACTS[kind], dh=dh1)
    fp8.fp8_act_bwd(ck.q, ck.s, da, ACTS[kind], FMTS[fmt], 0, r1.q, r1.s)
    fp8.fp8_act_bwd(ck.q, ck.s, da, ACTS[kind], FMTS[fmt], 0, dh_q_col=c1.q, dh_s_col=c1.s)
    fp8.fp8_act_bwd(ck.q, ck.s, da, ACTS[kind], a_q_col=a1.q, a_s_col=a1.s)
    assert torch.equal(dh1, dh)
    for p, q in ((r1, r), (c1, c), (a1, ac)):
        assert torch.equal(p.q, q.q) and torch.equal(p.s, q.s)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("kind", list(ACTS))
def test_activation_gradient_against_differences(kind):
    """act' of the backward pass against a central difference of the forward pass (float32 outputs)."""
    h = torch.linspace(-6, 6, 1024, device="cuda").view(8, 128)
    q, s = fp8.block_codes(8, 128), fp8.block_scales(8, 128)
    fp8.fp8_act_fwd(h, ACTS[kind], 0, q, s)
    kept = torch.empty_like(h)
    fp8.fp8_block_decode(q, s, fp8.FP8_E4M3, 1, kept)
    one, dh = torch.ones_like(h), torch.empty_like(h)
    fp8.fp8_act_bwd(q, s, one, ACTS[kind], dh=dh)
    e = 2.0 ** -7
    up, dn = torch.empty_like(h), torch.empty_like(h)
    spare_q, spare_s = torch.empty_like(q), torch.empty_like(s)
    fp8.fp8_act_fwd(kept + e, ACTS[kind], 0, spare_q, spare_s, a=up)
    fp8.fp8_act_fwd(kept - e, ACTS[kind], 0, spare_q, spare_s, a=dn)
    # third derivative below 3, rounding of values up to 7 by 2^-20 of them
    assert float(((up - dn) / (2 * e) - dh).abs().max()) < 3 * e * e / 6 + 7 * 2.0 ** -20 / e


@pytest.mark.parametrize("kind", list(ACTS))
def test_values_just_off_a_tie_keep_their_side(kind):
    """For large h, act(h) is h less something far below binary32's reach, and
    h may be exactly halfway between two codes: the code is the lower one.
    Likewise dh = da * act'(h) beside a halfway da."""
    h = torch.zeros((1, 128), device="cuda")
    h[0, 0] = 24.0                                     # the block's amax: scale 16, unit 1 above 8
    ties = torch.tensor([10.5, 11.5, 12.5, 13.5], device="cuda")  # halfway at unit 1; ties would go to 10, 12, 12, 14
    h[0, 1:5] = ties
    q, s = fp8.block_codes(1, 128), fp8.block_scales(1, 128)
    aq, a_s = fp8.block_codes(1, 128), fp8.block_scales(1, 128)
    fp8.fp8_act_fwd(h, ACTS[kind], 0, q, s, aq, a_s)
    out = torch.empty_like(h)
    fp8.fp8_block_decode(aq, a_s, fp8.FP8_E4M3, 1, out)
    assert out[0, 1:5].tolist() == [10.0, 11.0, 12.0, 13.0]


def test_activation_of_non_finite_values():
    h = torch.zeros((2, 256), device="cuda")
    h[0, 3], h[0, 4], h[1, 200] = float("inf"), -float("inf"), float("nan")
    for act in ACTS.values():
        q, s, a = fp8.block_codes(2, 256), fp8.block_scales(2, 256), torch.empty_like(h)
        fp8.fp8_act_fwd(h, act, 0, q, s, a=a)
        assert fp8.fp8_get_status() == fp8.FP8_STATUS_NONFINITE
        # act(-inf) is 0 less the smallest subnormal gate times 110
        assert a[0, 3] == float("inf") and -110 * 2.0 ** -149 <= a[0, 4] <= 0 and a[1, 200].isnan()
        assert int(a.isfinite().sum()) == 2 * 256 - 2


# ---------------------------------------------------------------- streams, graphs, runs together
def _step(b):
    fp8.fp8_block_cast(b["x"], fp8.FP8_E4M3, 0, b["xq"], b["xs"], b["xqc"], b["xsc"])
    fp8.fp8_block_cast(b["dy"], fp8.FP8_E5M2, 0, b["gq"], b["gs"], b["gqc"], b["gsc"])
    fp8.fp8_block_cast_square(b["w"], fp8.FP8_E4M3, 0, b["wq"], b["ws"], b["wsc"])
    fp8.fp8_block_linear_fwd(b["xq"], b["xs"], b["wq"], b["ws"], b["y"])
    fp8.fp8_block_linear_dgrad(b["gq"], b["gs"], fp8.FP8_E5M2, b["wq"], b["wsc"], b["dx"])
    fp8.fp8_block_linear_wgrad(b["gqc"], b["gsc"], fp8.FP8_E5M2, b["xqc"], b["xsc"], b["dw"])
    fp8.fp8_act_fwd(b["y"], fp8.FP8_ACT_SILU, 0, b["cq"], b["cs"], a=b["a"])
    fp8.fp8_act_bwd(b["cq"], b["cs"], b["dy"], fp8.FP8_ACT_SILU, dh=b["dh"])
    fp8.fp8_block_linear_tokens(b["x"][:20], b["wq"], b["ws"], b["yt"])


def _buffers(M, N, K, seed):
    C, S = fp8.block_codes, fp8.block_scales
    b = dict(x=synth.device_normal((M, K), 1.0, seed, BF16, "cuda"), w=synth.device_normal((N, K), 0.02, seed + 1, BF16, "cuda"),
             dy=synth.device_normal((M, N), 1e-4, seed + 2, BF16, "cuda"))
    b |= dict(xq=C(M, K), xs=S(M, K), xqc=C(M, K), xsc=S(K, M), gq=C(M, N), gs=S(M, N), gqc=C(M, N), gsc=S(N, M),
              wq=C(N, K), ws=S(N, K), wsc=S(K, N), cq=C(M, N), cs=S(M, N))
    b |= {k: torch.empty(s, dtype=BF16, device="cuda") for k, s in
          dict(y=(M, N), dx=(M, K), dw=(N, K), a=(M, N), dh=(M, N), yt=(20, N)).items()}
    return b


OUTS = ("y", "dx", "dw", "a", "dh", "yt", "xs", "gsc", "wsc", "cs")


@pytest.mark.parametrize("shape", [(200, 264, 520), (2304, 4864, 512)])
def test_graph_replay_equals_eager_calls(shape):
    eager, graphed = _buffers(*shape, 5), _buffers(*shape, 5)
    _step(eager)
    _step(graphed)
    for k in OUTS:
        graphed[k].zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _step(graphed)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(eager[k], graphed[k]), k
    assert fp8.fp8_get_status() == 0


def test_two_streams_at_once_give_the_same_results():
    ref, a, b = _buffers(520, 1032, 1040, 9), _buffers(520, 1032, 1040, 9), _buffers(520, 1032, 1040, 9)
    _step(ref)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(8):
        with torch.cuda.stream(s1):
            _step(a)
        with torch.cuda.stream(s2):
            _step(b)
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(ref[k], a[k]) and torch.equal(ref[k], b[k]), k
    assert fp8.fp8_get_status() == 0


class _Routed:
    """fp8._calls with its answers noted, or refusing every call."""

    def __init__(self, calls, refuse):
        self.calls, self.refuse, self.answers = calls, refuse, []

    def __getattr__(self, name):
        def call(*a):
            ok = False if self.refuse else getattr(self.calls, name)(*a)
            self.answers.append((name, ok))
            return ok
        return call


def test_both_routes_of_a_call_give_the_same_results(monkeypatch):
    a, b = _buffers(200, 264, 520, 5), _buffers(200, 264, 520, 5)
    short, long = _Routed(fp8._calls, False), _Routed(fp8._calls, True)
    for calls, buffers in ((short, a), (long, b)):
        monkeypatch.setattr(fp8, "_calls", calls)
        _step(buffers)
    torch.cuda.synchronize()
    assert all(ok for _, ok in short.answers) and len({n for n, _ in short.answers}) == 8
    for k in OUTS:
        assert torch.equal(a[k], b[k]), k


def test_the_short_route_leaves_what_is_not_plain():
    L, calls = Layer(32, 64, 128), fp8._calls
    y, st = torch.full((32, 64), 5.0, device="cuda"), torch.cuda.Stream()
    fwd = dict(xq=L.xq, xs=L.xs, wq=L.wq, ws=L.ws, y=y, bias=None, stream=None, rto=False)
    for name, bad in (("xq", L.xq[:, :100]), ("xq", L.xq[None]), ("xq", L.xq.cpu()), ("xq", None), ("xs", L.xs[:100]),
                      ("xs", L.xs.float()), ("xs", L.xs.cpu()), ("wq", L.wq.view(torch.int8)), ("wq", 3), ("y", y[:, :63]),
                      ("y", y.double()), ("y", y.t().contiguous().t()), ("bias", torch.ones(63, device="cuda")),
                      ("bias", torch.ones(64)), ("stream", st), ("stream", 0), ("rto", 1), ("rto", True)):
        assert calls.linear_fwd(*(fwd | {name: bad}).values()) is False, (name, bad)
    cast = dict(x=L.x, fmt=0, margin=0, q=L.xq.clone(), s=L.xs.clone(), qc=None, sc=None, stream=None)
    for name, bad in (("x", L.x.double()), ("x", L.x[:1].expand(32, 128)), ("x", L.x[:, ::2]), ("fmt", 0.0), ("fmt", 2 ** 40),
                      ("fmt", 7), ("margin", None), ("margin", -1), ("s", None), ("q", None), ("qc", L.xq), ("stream", st)):
        assert calls.block_cast(*(cast | {name: bad}).values()) is False, (name, bad)
    torch.cuda.synchronize()
    assert bool((y == 5.0).all()) and calls.block_cast(*cast.values()) is True
    assert torch.equal(cast["q"], L.xq)
    assert fp8.fp8_get_status() == 0


def test_calls_take_an_explicit_stream():
    L = Layer(64, 128, 256)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y, y0 = torch.empty((64, 128), device="cuda"), torch.empty((64, 128), device="cuda")
    fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y0)
    fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y, y0)


@pytest.mark.parametrize("M", [5, 200])
def test_block_linear_layer(M):
    """The layer module against its products in binary64, with and without kept activations."""
    N, K = 264, 520
    x, w, dy = dev(data(M, K, "lx"), BF16), dev(data(N, K, "lw", std=0.02), BF16), dev(data(M, N, "ldy", std=1e-3), BF16)
    bias = torch.randn(N, device="cuda").to(BF16)
    layer = BlockLinear(w, bias)
    X, Xc = (torch.from_numpy(cast_values(f64(x), "e4m3", *b)[0]).cuda() for b in ((1, 128), (128, 1)))
    G, Gc = (torch.from_numpy(cast_values(f64(dy), "e5m2", *b)[0]).cuda() for b in ((1, 128), (128, 1)))
    W = torch.from_numpy(cast_values(f64(w), "e4m3", 128, 128)[0]).cuda()
    ref = (X @ W.T + bias.double(), X.abs() @ W.abs().T + bias.double().abs(), K)
    assert_product(layer.forward(x), ref)
    with pytest.raises(RuntimeError):
        layer.backward(dy)
    assert_product(layer.forward(x, keep=True), ref)
    dx, dw = layer.backward(dy)
    assert_product(dx, (G @ W, G.abs() @ W.abs(), N))
    assert_product(dw, (Gc.T @ Xc, Gc.abs().T @ Xc.abs(), M))
    layer.weight.update(w * 2)
    assert torch.equal(layer.forward(x), BlockLinear(w * 2, bias).forward(x))


@pytest.mark.parametrize("kind", list(ACTS))
def test_block_mlp_gradients(kind):
    """The feed-forward block: every product against binary64 from the tensors
    it really multiplied (recomputed with the library's casts, each tested
    above), and the whole against the plain layer in binary64 to the size of
    FP8's rounding."""
    M, K, F, N = 150, 264, 520, 200
    x, dy = dev(data(M, K, "mx", std=0.02), BF16), dev(data(M, N, "mdy", std=1e-3), BF16)
    w1, w2 = dev(data(F, K, "mw1", std=0.02), BF16), dev(data(N, F, "mw2", std=0.02), BF16)
    mlp = BlockMLP(w1, w2, ACTS[kind])
    y = mlp.forward(x)
    assert mlp.kept_bytes() <= M * (K + F) + 16 * M + (K + 128) * 1024 // 128 * 8 + M * F // 64 + 65536
    dx, dw1, dw2 = mlp.backward(dy)
    assert fp8.fp8_get_status() == 0
    c = lambda t, f, *b: cast_values(t, f, *b)[0]  # noqa: E731
    X, W1, W2, DY = f64(x), c(f64(w1), "e4m3", 128, 128), c(f64(w2), "e4m3", 128, 128), f64(dy)
    bf = lambda t: torch.from_numpy(t).to(BF16).double().numpy()  # noqa: E731
    h = bf(c(X, "e4m3", 1, 128) @ W1.T)
    kept = c(h, "e4m3", 1, 128)
    da = bf(c(DY, "e5m2", 1, 128) @ W2)
    dh = act_grad_strict(kept, da, kind)
    want = dict(y=c(act_strict(h, kind), "e4m3", 1, 128) @ W2.T, dx=c(dh, "e5m2", 1, 128) @ W1,
                dw1=c(dh, "e5m2", 128, 1).T @ c(X, "e4m3", 128, 1),
                dw2=c(DY, "e5m2", 128, 1).T @ c(act_strict(kept, kind), "e4m3", 128, 1))
    for name, got in (("y", y), ("dx", dx), ("dw1", dw1), ("dw2", dw2)):
        ref = want[name]
        # bf16 rounding (2^-9 rms of a half-unit error) and the few elements of h, da that bf16 or FP8 rounds
        # to the neighbour where binary32 sums differ from binary64's in the last place
        assert np.linalg.norm(f64(got) - ref) <= 0.005 * np.linalg.norm(ref), name
    with pytest.raises(RuntimeError):
        mlp.backward(dy)


@pytest.mark.parametrize("given", [True, False])
def test_modules_on_another_stream(given):
    """A pass on a busy side stream while the current one reuses whatever
    memory its temporaries and kept tensors would have given back to it."""
    M, K, F = 200, 264, 520
    x, dy = (synth.device_normal((M, n), 1.0, 40 + n, BF16, "cuda") for n in (K, F))
    w1, w2 = (synth.device_normal(s, 0.02, 50 + s[0], BF16, "cuda") for s in ((F, K), (K, F)))
    lin, mlp = BlockLinear(w1), BlockMLP(w1, w2, fp8.FP8_ACT_SILU)
    dz = synth.device_normal((M, K), 1.0, 60, BF16, "cuda")

    def passes(side=None):
        out = []

        def there(f, *a, **k):  # f on the side stream, behind a wait there; then memory is taken and filled here
            if side is None:
                return f(*a, **k)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            if given:
                r = f(*a, **k, stream=side)
            else:
                with torch.cuda.stream(side):
                    r = f(*a, **k)
            for n in (M * K, M * F, M * 384, M * 640, 2 * M * F, 4096, 5120):
                for _ in range(4):
                    torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55)
            return r

        out.append(there(lin.forward, x, keep=True))
        out += there(lin.backward, dy)
        out.append(there(lin.forward, x[:9]))
        out.append(there(mlp.forward, x))
        out += there(mlp.backward, dz)
        out.append(mlp.forward(x))  # kept here, used there
        out += there(mlp.backward, dz)
        torch.cuda.synchronize()
        return out

    for got, want in zip(passes(torch.cuda.Stream()), passes(), strict=True):
        assert torch.equal(got, want)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(500, 2056), (129, 257), (2100, 4100)])
def test_activation_in_place(shape, dtype):
    R, C = shape
    h, da = (synth.device_normal(shape, s, 70 + i, dtype, "cuda") for i, s in enumerate((2.0, 1.0)))
    q, s = fp8.block_codes(R, C), fp8.block_scales(R, C)
    q2, s2 = fp8.block_codes(R, C), fp8.block_scales(R, C)
    a, dh = torch.empty_like(h), torch.empty_like(da)
    fp8.fp8_act_fwd(h, fp8.FP8_ACT_GELU_TANH, 0, q, s, a=a)
    fp8.fp8_act_bwd(q, s, da, fp8.FP8_ACT_GELU_TANH, dh=dh)
    fp8.fp8_act_fwd(h, fp8.FP8_ACT_GELU_TANH, 0, q2, s2, a=h)
    fp8.fp8_act_bwd(q2, s2, da, fp8.FP8_ACT_GELU_TANH, dh=da)
    assert torch.equal(h, a) and torch.equal(da, dh) and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("cols", [2304, 2300, 2297])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_many_tiles_as_their_rows_of_tiles(dtype, cols):
    """The elementwise kernels' forms for many tiles against those for few,
    which the binary64 tests cover: 128 rows at a time, the same bits."""
    R, C, S = 1500, fp8.block_codes, fp8.block_scales
    h, da = (dev(data(R, cols, "tiles", i), dtype) for i in range(2))

    def run(h, da):
        r = h.shape[0]
        o = {k: C(r, cols) for k in ("row", "row2", "col", "square", "ck", "aq", "dq", "dqc", "aqc")}
        o |= {k: S(r, cols) for k in ("row_s", "row2_s", "square_s", "ck_s", "aq_s", "dq_s")}
        cs = [S(cols, r) for _ in range(4)]
        o |= {k: torch.empty_like(h) for k in ("a", "dh", "dh2")}
        fp8.fp8_block_cast(h, fp8.FP8_E4M3, 0, o["row"], o["row_s"])
        fp8.fp8_block_cast(h, fp8.FP8_E5M2, 0, o["row2"], o["row2_s"], o["col"], cs[0])
        fp8.fp8_block_cast_square(h, fp8.FP8_E4M3, 0, o["square"], o["square_s"], cs[1])
        fp8.fp8_act_fwd(h, fp8.FP8_ACT_GELU_TANH, 0, o["ck"], o["ck_s"], o["aq"], o["aq_s"], o["a"])
        fp8.fp8_act_bwd(o["ck"], o["ck_s"], da, fp8.FP8_ACT_GELU_TANH, dh=o["dh"])
        fp8.fp8_act_bwd(o["ck"], o["ck_s"], da, fp8.FP8_ACT_GELU_TANH, fp8.FP8_E5M2, 0, o["dq"], o["dq_s"], o["dqc"],
                        cs[2], o["aqc"], cs[3], o["dh2"])
        return o

    whole = run(h, da)
    for r0 in range(0, R, 128):
        part = run(h[r0:r0 + 128], da[r0:r0 + 128])
        for k, v in part.items():
            w = whole[k][r0:r0 + 128] if v.dim() == 2 else whole[k][r0 // 128 * v.numel():][:v.numel()]
            bits = torch.int32 if v.dtype == F32 else torch.int16 if v.dtype in (BF16, F16) else torch.uint8
            assert torch.equal(w.view(bits) if v.dim() == 1 else w.contiguous().view(bits), v.contiguous().view(bits)), (k, r0)
    assert fp8.fp8_get_status() == 0


def test_first_calls_of_a_process_captured():
    """No call of the library before the capture: what it sets up once per
    device is set up then."""
    code = """
import torch
from fp8_mixed_precision_tensor_b200 import fp8
C, S = fp8.block_codes, fp8.block_scales
x = torch.randn(200, 300, device="cuda").to(torch.bfloat16)
w = torch.randn(260, 300, device="cuda").to(torch.bfloat16)
b = [C(200, 300), S(200, 300), C(260, 300), S(260, 300), S(300, 260)]
y = torch.zeros(200, 260, device="cuda", dtype=torch.bfloat16)
t, z = torch.zeros_like(y), torch.zeros_like(y)
ck, cs = C(200, 260), S(200, 260)
def work():
    fp8.fp8_block_cast(x, 0, 0, b[0], b[1])
    fp8.fp8_block_cast_square(w, 0, 0, b[2], b[3], b[4])
    fp8.fp8_block_linear_fwd(b[0], b[1], b[2], b[3], y)
    fp8.fp8_block_linear_tokens(x[:7], b[2], b[3], t[:7])
    fp8.fp8_act_fwd(y, 2, 0, ck, cs)
    fp8.fp8_act_bwd(ck, cs, y, 2, dh=z)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    work()
g.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (y, t, z)]
work()
torch.cuda.synchronize()
assert all(torch.equal(u, v) for u, v in zip(got, (y, t, z))) and float(y.abs().sum()) > 0
assert fp8.fp8_get_status() == 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_block_wgrad_feeds_the_adam_step():
    """dW as round-to-odd bf16 into the per-tensor FP8 gradient cast and Adam, as the other wgrad does."""
    from fp8_mixed_precision_tensor_b200.adam_state import AdamTensorState, FP8Adam

    w = synth.device_normal((256, 256), 0.02, 31, BF16, "cuda")
    x, dy = synth.device_normal((256, 256), 1.0, 32, BF16, "cuda"), synth.device_normal((256, 256), 1e-4, 33, BF16, "cuda")
    states, layers = [AdamTensorState(w) for _ in range(2)], [BlockLinear(w) for _ in range(2)]
    for st, layer, rto in zip(states, layers, (True, False)):
        layer.forward(x, keep=True)
        _, dw = layer.backward(dy if rto else dy.float(), rto=rto)
        assert dw.dtype == (BF16 if rto else F32)
        st.set_gradient(dw, mu=1.0)
        FP8Adam([st], lr=1e-3).step()
    assert torch.equal(states[0].g, states[1].g) and torch.equal(states[0].w, states[1].w)
    assert fp8.fp8_get_status() == 0


def test_binding_refuses_wrong_shapes_and_layouts():
    L = Layer(32, 64, 128)
    y = torch.empty((32, 64), device="cuda")
    for bad in (lambda: fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y[:, :63]),
                lambda: fp8.fp8_block_linear_fwd(L.xq, L.xs[:100], L.wq, L.ws, y),
                lambda: fp8.fp8_block_linear_fwd(L.xq[:, :100], L.xs, L.wq, L.ws, y),
                lambda: fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y.t().contiguous().t()),
                lambda: fp8.fp8_block_linear_fwd(L.xq, L.xs, L.wq, L.ws, y, bias=torch.ones(63, device="cuda")),
                lambda: fp8.fp8_block_cast(L.x, 0, 0, L.xq),
                lambda: fp8.fp8_block_cast(L.x[:1].expand(32, 128), 0, 0, L.xq, L.xs),
                lambda: fp8.fp8_act_bwd(L.gq, L.gs, y[:8], fp8.FP8_ACT_SILU, dh=y)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fp8.fp8_block_cast(L.x, 0, 0, L.xq.view(torch.int8), L.xs)
    with pytest.raises(fp8.FP8Error):
        fp8.fp8_block_linear_tokens(L.x.repeat(2, 1), L.wq, L.ws, torch.empty((64, 64), device="cuda"))


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(5, 300), (1500, 2304), (1500, 2297)])
def test_activation_backward_of_non_finite_gradients(shape, dtype, kind):
    """An infinite da stays infinite, of the sign of da * act'(h'), for h' of
    either sign and 0; a NaN stays NaN; codes saturate; nothing else changes.
    Fewer tiles than SMs, and more, of aligned rows and of odd ones."""
    R, C = shape
    h = torch.tensor([-2.0, -0.5, 0.0, 0.25, 0.5, 1.0, 1.5, 2.0], device="cuda").repeat(-(-C // 8))[:C].repeat(R, 1)  # exact in E4M3
    ck = row_blocks(R, C)
    fp8.fp8_act_fwd(h, ACTS[kind], 0, ck.q, ck.s)
    fine = dev(data(R, C, "nfda", zeros=False), dtype)
    da = fine.clone()
    bad = [(1, 0, float("inf")), (2, 8, -float("inf")), (3, 16, float("nan")), (R - 1, C - 12, float("inf"))]
    for r, c, v in bad:
        da[r, c:c + 8] = v
    hit = da != fine
    named = lambda t: t.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0)  # noqa: E731  (comparable)
    out = {}
    for fmt in FMTS:
        for name, g in (("fine", fine), ("da", da)):
            o = dict(dh=torch.empty_like(g), r=row_blocks(R, C), c=col_blocks(R, C), a=col_blocks(R, C))
            fp8.fp8_act_bwd(ck.q, ck.s, g, ACTS[kind], FMTS[fmt], 0, o["r"].q, o["r"].s, o["c"].q, o["c"].s, o["a"].q,
                            o["a"].s, o["dh"])
            assert fp8.fp8_get_status() == (0 if name == "fine" else fp8.FP8_STATUS_NONFINITE)
            alone, placed, spare = torch.empty_like(g), g.clone(), row_blocks(R, C)
            fp8.fp8_act_bwd(ck.q, ck.s, g, ACTS[kind], dh=alone)
            assert fp8.fp8_get_status() == 0
            fp8.fp8_act_bwd(ck.q, ck.s, placed, ACTS[kind], FMTS[fmt], 0, spare.q, spare.s, dh=placed)
            fp8.fp8_get_status()
            for t in (alone, placed):
                assert torch.equal(named(t), named(o["dh"]))
            out[name] = o
        _, d, _, tol_d = (torch.from_numpy(t).cuda() for t in act_bounds(f64(h), kind))
        want = d * da.double()
        got = out["da"]["dh"]
        assert bool(want[hit].isnan().any()) and bool((want[hit] == float("inf")).any()) and bool((want[hit] == -float("inf")).any())
        assert torch.equal(named(got[hit].double()), named(want[hit]))
        assert torch.equal(got[~hit], out["fine"]["dh"][~hit])
        assert torch.equal(out["da"]["a"].q, out["fine"]["a"].q) and torch.equal(out["da"]["a"].s, out["fine"]["a"].s)
        fmax = {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
        for axis, key in ((1, "r"), (0, "c")):
            v = {n: torch.empty((R, C), device="cuda") for n in out}
            for n in v:
                fp8.fp8_block_decode(out[n][key].q, out[n][key].s, FMTS[fmt], axis, v[n])
                assert out[n][key].intact()
            sat = want[hit].clamp(-fmax, fmax).nan_to_num(nan=7.0)
            assert torch.equal(v["da"][hit].double().nan_to_num(nan=7.0), sat)
            # a block with such a value has scale 1; the others are as without
            blocks = {(r, c0 // 128 * 128) if axis else (r // 128 * 128, c0) for r, c, _ in bad for c0 in range(c, c + 8)}
            for r0, c0 in blocks:
                b = (slice(r0, r0 + 1), slice(c0, c0 + 128)) if axis else (slice(r0, r0 + 128), slice(c0, c0 + 1))
                keep = ~hit[b]
                x, tol = f64(want[b][keep]), f64(da[b][keep].abs().double() * tol_d[b][keep] + 1e-40)
                w = f64(v["da"][b][keep])
                assert np.all((w >= round_fp8(x - tol, fmt)) & (w <= round_fp8(x + tol, fmt)))
                v["da"][b] = v["fine"][b] = 0.0
            assert torch.equal(v["da"], v["fine"])


def _behind_a_wait(side):
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)


def _take_memory(*sizes):
    """Whatever memory of these sizes was given back to the current stream, overwritten on it."""
    for n in sizes:
        for _ in range(4):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55)


def test_weight_update_from_a_temporary_on_another_stream():
    N, K = 520, 264
    w = synth.device_normal((N, K), 0.02, 81, BF16, "cuda")
    want, layer, side = BlockLinear(w * 2), BlockLinear(w), torch.cuda.Stream()
    _behind_a_wait(side)
    layer.weight.update(w * 2, stream=side)
    _take_memory(2 * N * K)
    torch.cuda.synchronize()
    for k in ("q", "s", "s_col"):
        assert torch.equal(getattr(layer.weight, k), getattr(want.weight, k)), k


@pytest.mark.parametrize("given", [True, False])
def test_a_layer_dropped_while_its_pass_runs_on_another_stream(given):
    M, N, K = 200, 520, 264
    x, w1, w2 = (synth.device_normal(s, 0.5, 90 + i, BF16, "cuda") for i, s in enumerate(((M, K), (N, K), (K, N))))
    make = {"linear": lambda: BlockLinear(w1, w1[:, 0] * 4), "tokens": lambda: BlockLinear(w1, w1[:, 0] * 4),
            "mlp": lambda: BlockMLP(w1, w2)}
    side = torch.cuda.Stream()
    for kind, new in make.items():
        a = x[:9] if kind == "tokens" else x
        want, layer = new().forward(a), new()
        _behind_a_wait(side)
        if given:
            got = layer.forward(a, stream=side)
        else:
            with torch.cuda.stream(side):
                got = layer.forward(a)
        del layer
        _take_memory(N * 384, N * 640, K * 640, 2 * N, 4096, 5120, 512 * 5, 512 * 15, 512 * 10)
        torch.cuda.synchronize()
        assert torch.equal(got, want), kind


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("R", [1, 1500])
def test_gradients_just_off_a_tie_keep_their_side(kind, R):
    """For large h', act'(h') is above 1 by something far below binary32's
    reach.  A da exactly halfway between two codes gives the one farther from
    0, in blocks along either axis."""
    C = 2048 if R > 1 else 128  # more tiles than SMs, or one
    ck, cs = fp8.block_codes(R, C), fp8.block_scales(R, C)
    fp8.fp8_act_fwd(torch.full((R, C), 24.0, device="cuda"), ACTS[kind], 0, ck, cs)  # kept as it is
    # Every block along the rows and the columns has amax 24, scale 16: units of 1 above 8, 0.5 below.
    # Ties to even would give 10, 12, 12, 14, 4 and 5.
    da = torch.full((R, C), 24.0, device="cuda")
    ties = torch.tensor([10.5, 11.5, 12.5, 13.5, 4.25, 5.25], device="cuda")
    want = torch.tensor([11.0, 12.0, 13.0, 14.0, 4.5, 5.5], device="cuda")
    out = da.clone()
    for i in range(6):
        r, sign = (0 if R == 1 else 130 + 17 * i), (1.0, -1.0)
        for k in range(2):
            for at in (7 + 16 * i + k, C - 21 + i + 7 * k):
                da[r, at], out[r, at] = sign[k] * ties[i], sign[k] * want[i]
    for dtype in (F32, BF16, F16):  # (all values are in each type)
        q, s, qc, sc = fp8.block_codes(R, C), fp8.block_scales(R, C), fp8.block_codes(R, C), fp8.block_scales(C, R)
        fp8.fp8_act_bwd(ck, cs, da.to(dtype), ACTS[kind], fp8.FP8_E4M3, 0, q, s, qc, sc)
        got = torch.empty_like(da)
        fp8.fp8_block_decode(q, s, fp8.FP8_E4M3, 1, got)
        assert torch.equal(got, out), dtype
        if R > 1:  # (a column of one element has a scale of its own)
            fp8.fp8_block_decode(qc, sc, fp8.FP8_E4M3, 0, got)
            assert torch.equal(got, out), dtype


@pytest.mark.parametrize("cols", [2304, 2297])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_column_scales_of_many_tiles(dtype, cols):
    """The scale bytes of blocks along the rows, from the forms for many tiles:
    128 rows at a time the bytes of the forms for few, and 127 in the padding."""
    from _block import scale_address

    R, C, S = 1500, fp8.block_codes, fp8.block_scales
    h, da = (dev(data(R, cols, "coltiles", i), dtype) for i in range(2))

    def run(h, da):
        r = h.shape[0]
        q, ck, ck_s, row_s = C(r, cols), C(r, cols), S(r, cols), S(r, cols)
        out = {k: S(cols, r).fill_(GUARD) for k in ("cast", "alone", "square", "dh", "a")}
        fp8.fp8_block_cast(h, fp8.FP8_E5M2, 0, q, row_s, C(r, cols), out["cast"])
        fp8.fp8_block_cast(h, fp8.FP8_E4M3, 0, q_col=q, s_col=out["alone"])
        fp8.fp8_block_cast_square(h, fp8.FP8_E4M3, 0, q, row_s, out["square"])
        fp8.fp8_act_fwd(h, fp8.FP8_ACT_SILU, 0, ck, ck_s)
        fp8.fp8_act_bwd(ck, ck_s, da, fp8.FP8_ACT_SILU, fp8.FP8_E5M2, 0, dh_q_col=q, dh_s_col=out["dh"], a_q_col=C(r, cols),
                        a_s_col=out["a"])
        return {k: v.cpu().numpy() for k, v in out.items()}

    whole, c, blocks = run(h, da), np.arange(cols), -(-R // 128)
    for k, got in whole.items():
        rest = np.ones(len(got), dtype=bool)
        for b in range(blocks):
            rest[scale_address(c, b, R)] = False
        assert np.all(got[rest] == 127), k
    for b in range(blocks):
        part = run(h[b * 128:(b + 1) * 128], da[b * 128:(b + 1) * 128])
        for k, got in whole.items():
            assert np.array_equal(got[scale_address(c, b, R)], part[k][scale_address(c, 0, 128)]), (k, b)
    # the few-tile forms' own bytes, of the first rows
    x = f64(h[:128])
    assert np.array_equal(part["cast"][scale_address(c, 0, 128)],
                          (127 - exponents(blocks_of(f64(h[(blocks - 1) * 128:]), 128, 1), "e5m2")[0]).astype(np.uint8))
    assert np.array_equal(whole["alone"][scale_address(c, 0, R)], (127 - exponents(blocks_of(x, 128, 1), "e4m3")[0]).astype(np.uint8))
    assert fp8.fp8_get_status() == 0


def test_several_passes_in_flight():
    """`kept` taken after each forward pass and set before its backward pass; otherwise the last pass's."""
    M, N, K = 160, 264, 520
    w, w2 = synth.device_normal((N, K), 0.02, 101, BF16, "cuda"), synth.device_normal((K, N), 0.02, 102, BF16, "cuda")
    for layer in (BlockLinear(w), BlockMLP(w, w2)):
        keep = {"keep": True} if isinstance(layer, BlockLinear) else {}
        xs = [synth.device_normal((M + i, K), 1.0, 103 + i, BF16, "cuda") for i in range(3)]
        dys, want, kept = [], [], []
        for x in xs:
            dys.append(synth.device_normal(layer.forward(x, **keep).shape, 1e-3, 110 + len(dys), BF16, "cuda"))
            want.append(layer.backward(dys[-1]))
        for x in xs:
            layer.forward(x, **keep)
            kept.append(layer.kept)
        with pytest.raises(ValueError):
            layer.backward(dys[0])  # another pass's: other tokens
        for i in (1, 0, 2):
            layer.kept = kept[i]
            for got, ref in zip(layer.backward(dys[i]), want[i], strict=True):
                assert torch.equal(got, ref)
        assert layer.kept is None


def test_pairs_take_and_give_back_tensor_memory_many_times():
    """Products on CTA pairs among other kernels of the stream, without a pause
    and some millions of pairs long: a pair that waits for its tensor memory
    for good would show once in about ten million.  In a process of its own,
    so that it could be ended."""
    code = """
import torch
from fp8_mixed_precision_tensor_b200 import fp8, synth
C, S = fp8.block_codes, fp8.block_scales
M, K, N = 2720, 167, 656
x, w, dy = (synth.device_normal(s, v, 7, torch.bfloat16, "cuda") for s, v in (((M, K), 1.0), ((N, K), 0.02), ((M, N), 1e-3)))
xq, xs, gq, gs, ck, cs = C(M, K), S(M, K), C(M, N), S(M, N), C(M, N), S(M, N)
xqc, xsc, gqc, gsc, aq, a_s = C(M, K), S(K, M), C(M, N), S(N, M), C(M, N), S(M, N)
wq, ws, wsc, w2, w2s, w2c = C(N, K), S(N, K), S(K, N), C(K, N), S(K, N), S(N, K)
y, z, dx, dw = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((M, N), (M, K), (M, K), (N, K)))
fp8.fp8_block_cast_square(w, 0, 0, wq, ws, wsc)
fp8.fp8_block_cast_square(w.t().contiguous(), 0, 0, w2, w2s, w2c)
def step():
    fp8.fp8_block_cast(x, 0, 0, xq, xs, xqc, xsc)
    fp8.fp8_block_linear_fwd(xq, xs, wq, ws, y)
    fp8.fp8_act_fwd(y, 1, 0, ck, cs, aq, a_s)
    fp8.fp8_block_linear_fwd(aq, a_s, w2, w2s, z)
    fp8.fp8_block_cast(dy, 1, 0, gq, gs, gqc, gsc)
    fp8.fp8_block_linear_wgrad(gqc, gsc, 1, xqc, xsc, dw)
    fp8.fp8_block_linear_dgrad(gq, gs, 1, wq, wsc, dx)
step()
first = [t.clone() for t in (y, z, dx, dw)]
for _ in range(40):
    for _ in range(1000):
        step()
    torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (y, z, dx, dw))) and fp8.fp8_get_status() == 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_products_read_what_the_kernels_before_them_have_just_written():
    """The few-token form brings x and weights into L2 before the kernel in
    front of it has ended; operands that change from call to call, without a
    pause, give what they give with a pause after every kernel."""
    M, N, K, n = 24, 2304, 2048, 40
    C, S = fp8.block_codes, fp8.block_scales
    hs = [synth.device_normal((M, K), 1.0, 200 + i, BF16, "cuda") for i in range(n)]
    w32 = [synth.device_normal((N, K), 0.02, 300 + i, BF16, "cuda") for i in range(4)]
    ck, cs, x, wq, ws, wsc = C(M, K), S(M, K), torch.empty_like(hs[0]), C(N, K), S(N, K), S(K, N)
    xq, xs = C(M, K), S(M, K)
    got = {}
    for pause in (False, True):
        ys = [torch.empty((M, N), dtype=BF16, device="cuda") for _ in range(3 * n)]
        wait = torch.cuda.synchronize if pause else (lambda: None)
        for _ in range(5):
            for i in range(n):
                for f in (lambda: fp8.fp8_block_cast_square(w32[i % 4], 0, 0, wq, ws, wsc),
                          lambda: fp8.fp8_act_fwd(hs[i], fp8.FP8_ACT_SILU, 0, ck, cs, a=x),
                          lambda: fp8.fp8_block_linear_tokens(x, wq, ws, ys[3 * i]),
                          lambda: fp8.fp8_block_decode(ck, cs, fp8.FP8_E4M3, 1, x),
                          lambda: fp8.fp8_block_linear_tokens(x, wq, ws, ys[3 * i + 1]),
                          lambda: fp8.fp8_block_cast(x, fp8.FP8_E4M3, 0, xq, xs),
                          lambda: fp8.fp8_block_linear_fwd(xq, xs, wq, ws, ys[3 * i + 2])):
                    f()
                    wait()
        torch.cuda.synchronize()
        got[pause] = ys
    for a, b in zip(got[False], got[True]):
        assert torch.equal(a, b)
    assert len({float(y.float().sum()) for y in got[True]}) > n
    assert fp8.fp8_get_status() == 0
