"""Norms with gate and residual, log probabilities and distillation on the GPU against binary64 (tests/_passes.py,
where the bounds are derived)."""
import math
import zlib

import pytest
import torch

from fp8_mixed_precision_tensor_b200 import fp8
from _passes import EPS, HALF, U, Norm64, Rows64, check, rounding
from test_gpu_block import check_codes, col_blocks, f64, row_blocks

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KIND = {"none": fp8.FP8_NORM_NONE, "rms": fp8.FP8_NORM_RMS, "layer": fp8.FP8_NORM_LAYER}
FORM = {"top": fp8.FP8_DISTILL_TOP, "tail": fp8.FP8_DISTILL_TAIL}
GUARD = 77.0


def rng(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def normal(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


class Strided:
    """A [rows, cols] matrix in rows `pad` elements longer, starting at element `offset`, all else a pattern."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0, values=None):
        self.buf = torch.full((offset + rows * (cols + pad) + 16,), GUARD, dtype=dtype, device="cuda")
        self.t = self.buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        if values is not None:
            self.t.copy_(values)
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False

    def intact(self):
        return bool((self.buf[self.mask] == GUARD).all())


# ---------------------------------------------------------------- norms
def norm_inputs(rows, cols, dtype, res, pre, post, gate, seed=0, pad=0, offset=0, pdtype=None):
    g = rng(rows, cols, pre, post, gate, seed)
    pdtype = pdtype or dtype
    h = normal(g, rows, cols) + 0.3
    h[:, cols // 2] *= 30.0
    r = normal(g, rows, cols, std=2.0)
    if rows > 2:
        h[1] = 0.0
        r[1] = 0.0
    vec = lambda mean, std, *s: (mean + torch.randn(s or (cols,), device="cuda", generator=g) * std).to(pdtype)  # noqa: E731
    gates = {"none": 0, "channel": 1}.get(gate, gate)
    p = dict(w=vec(1, 0.2), b=vec(0, 0.2) if pre == "layer" else None, post_w=vec(1, 0.2) if post != "none" else None,
             post_b=vec(0, 0.2) if post == "layer" else None, res_scale=0.75,
             gate=None if not gates else vec(0, 0.5) if gate == "channel" else vec(0, 0.5, gates, cols))
    if pre == "none":
        p["w"] = None
    s = lambda t, dt: Strided(rows, cols, dt, pad, offset, t).t  # noqa: E731
    return s(h, dtype), s(r, res), p, s(normal(g, rows, cols, std=1e-2), dtype), s(normal(g, rows, cols, std=1e-2), res)


def run_norm(h, r, p, dx, dr_out, pre, post, pad=0, offset=0, with_dr=True):
    """Forward and backward pass; every output checked against binary64."""
    rows, cols = r.shape
    new = lambda like: Strided(rows, cols, like.dtype, pad, offset)  # noqa: E731
    r_out, x = new(r), new(h)
    stats = torch.empty(rows, 4, device="cuda")
    kinds = dict(pre=KIND[pre], post=KIND[post])
    fp8.fp8_norm_fwd(h, r, r_out.t, stats, **kinds, **p, eps=EPS, x=x.t if pre != "none" else None)
    ref = Norm64(h, r, r_out.t, pre, post, p["w"], p["b"], p["post_w"], p["post_b"], p["gate"], p["res_scale"])
    check(r_out.t, ref.r_new, 32 * U * ref.r_mag, "r_out")
    if pre != "none":
        check(x.t, ref.x, 32 * U * ref.x_mag, "x")
    dh, dr = new(h), new(r)
    grads = {"d" + k: torch.full_like(p[k], GUARD) for k in ("w", "b", "post_w", "post_b", "gate") if p[k] is not None}
    gates = p["gate"].shape[0] if p["gate"] is not None and p["gate"].dim() == 2 else 1
    ws = torch.full((fp8.fp8_norm_workspace_bytes(rows, cols, rows // gates) // 4,), float("nan"), device="cuda")
    q = {k: v for k, v in p.items() if k != "b"}
    fp8.fp8_norm_bwd(dx if pre != "none" else None, dr_out if with_dr else None, h, r_out.t, stats, **kinds, **q,
                     dh=dh.t, dr=dr.t, workspace=ws, **grads)
    want = ref.backward(dx, dr_out if with_dr else None)
    check(dr.t, *bounded(want["dr"], 64), "dr")
    check(dh.t, *bounded(want["dh"], 128), "dh")
    for k, t in grads.items():  # a cluster adds up its rows, 148 clusters at the most follow
        v, m = want[k]
        check(t, v.view(t.shape), (128 + rows + 148) * U * m.view(t.shape), k)
    for s in (r_out, x, dh, dr):
        assert s.intact()
    assert fp8.fp8_get_status() == 0
    return r_out.t, x.t, dh.t, dr.t, grads


def bounded(pair, n):
    return pair[0], n * U * pair[1]


SIZES = [(1, 1), (1, 4096), (3, 130), (5, 33), (7, 1001), (70, 256), (33, 4104), (2, 12288), (300, 64), (3, 8200), (2, 16384)]


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("size", SIZES)
def test_norm(size, types):
    (rows, cols), (dtype, res) = size, types
    for pre, post, gate in (("rms", "rms", "channel"), ("layer", "none", "none"), ("layer", "layer", rows)):
        run_norm(*norm_inputs(rows, cols, dtype, res, pre, post, gate), pre, post)


@pytest.mark.parametrize("pre,post", [("none", "rms"), ("none", "layer"), ("none", "none"), ("rms", "none"), ("rms", "layer")])
@pytest.mark.parametrize("gate", ["none", "channel", 4, 1])
def test_norm_forms(pre, post, gate):
    run_norm(*norm_inputs(24, 520, BF16, F32, pre, post, gate), pre, post)
    run_norm(*norm_inputs(24, 520, F32, F32, pre, post, gate), pre, post, with_dr=pre == "none")


@pytest.mark.parametrize("rows,gates", [(777, 7), (900, 300), (600, 600), (2000, 2)])
def test_norm_gates_of_many_rows(rows, gates):
    run_norm(*norm_inputs(rows, 72, F16, F32, "rms", "rms", gates), "rms", "rms")


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (8, 8), (5, 3)])
@pytest.mark.parametrize("cols", [256, 1003])
def test_norm_strided_and_unaligned_rows(cols, pad, offset):
    args = norm_inputs(9, cols, BF16, BF16, "layer", "rms", "channel", 0, pad, offset)
    run_norm(*args, "layer", "rms", pad, offset)


def test_norm_parameters_of_other_types_and_a_strided_gate():
    h, r, p, dx, dr_out = norm_inputs(12, 384, BF16, F32, "layer", "layer", 3, pdtype=F32)
    p["w"], p["post_b"] = p["w"].to(F16), p["post_b"].to(BF16)
    wide = torch.zeros(3, 6 * 384, device="cuda")
    wide[:, 768:1152] = p["gate"]
    p["gate"] = wide[:, 768:1152]  # a chunk of a modulation's output
    run_norm(h, r, p, dx, dr_out, "layer", "layer")
    dgate = torch.zeros(3, 6 * 384, device="cuda")
    stats, r_out = torch.empty(12, 4, device="cuda"), torch.empty_like(r)
    kinds = dict(pre=KIND["layer"], post=KIND["layer"])
    fp8.fp8_norm_fwd(h, r, r_out, stats, **kinds, **p)
    ws = torch.empty(fp8.fp8_norm_workspace_bytes(12, 384, 4), dtype=torch.uint8, device="cuda")
    q = {k: v for k, v in p.items() if k != "b"}
    fp8.fp8_norm_bwd(dx, dr_out, h, r_out, stats, **kinds, **q, dgate=dgate[:, 384:768], workspace=ws)
    want = Norm64(h, r, r_out, "layer", "layer", *(p[k] for k in ("w", "b", "post_w", "post_b", "gate", "res_scale")))
    v, m = want.backward(dx, dr_out)["dgate"]
    check(dgate[:, 384:768], v, 300 * U * m)
    assert not dgate[:, :384].any() and not dgate[:, 768:].any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cols", [264, 1001, 4096])
def test_norm_residual_takes_its_scale_as_written(cols, dtype):
    """0.9f is not 0.9, but 0.9f * 10 rounds to 9: sums halfway between two 16-bit numbers go to the even one."""
    g = rng(cols, str(dtype))
    r = torch.randint(-2000, 2000, (50, cols), device="cuda", generator=g).to(dtype)
    h = torch.randint(-2000, 2000, (50, cols), device="cuda", generator=g).to(dtype) / 8
    r_out = torch.empty_like(r)
    fp8.fp8_norm_fwd(h, r, r_out, None, pre=KIND["none"], res_scale=0.9)
    assert torch.equal(r_out, (r.float() * 0.9 + h.float()).to(dtype))


def test_norm_in_place():
    for dtype, res in ((BF16, BF16), (F16, F32)):
        h, r, p, dx, dr_out = norm_inputs(40, 1096, dtype, res, "rms", "rms", "channel")
        r_out, x, dh, dr, _ = run_norm(h, r, p, dx, dr_out, "rms", "rms")
        h2, r2, stats = h.clone(), r.clone(), torch.empty(40, 4, device="cuda")
        kinds = dict(pre=KIND["rms"], post=KIND["rms"])
        fp8.fp8_norm_fwd(h2, r2, r2, stats, **kinds, **p, x=h2)
        assert torch.equal(r2, r_out) and torch.equal(h2, x)
        q = {k: v for k, v in p.items() if k != "b"}
        for over_h in (False, True):
            dx2, dr2, h3 = dx.clone(), dr_out.clone(), h.clone()
            fp8.fp8_norm_bwd(dx2, dr2, h3, r_out, stats, **kinds, **q, dh=h3 if over_h else dx2, dr=dr2)
            assert torch.equal(h3 if over_h else dx2, dh) and torch.equal(dr2, dr)


def test_norm_without_a_sublayer():
    _, r, p, dx, dr_out = norm_inputs(6, 264, BF16, BF16, "layer", "none", "none")
    x, stats = torch.empty_like(r), torch.empty(6, 4, device="cuda")
    q = dict(w=p["w"], pre=KIND["layer"])
    fp8.fp8_norm_fwd(None, r, None, stats, b=p["b"], x=x, **q)
    ref = Norm64(None, r, r, "layer", "none", p["w"], p["b"], None, None, None, 1.0)
    check(x, ref.x, 32 * U * ref.x_mag)
    dr, dw, db = torch.empty_like(r), torch.empty(264, device="cuda"), torch.empty(264, device="cuda", dtype=BF16)
    ws = torch.empty(fp8.fp8_norm_workspace_bytes(6, 264), dtype=torch.uint8, device="cuda")
    fp8.fp8_norm_bwd(dx, dr_out, None, r, stats, dr=dr, dw=dw, db=db, workspace=ws, **q)
    want = ref.backward(dx, dr_out)
    check(dr, *bounded(want["dr"], 64))
    check(dw, *bounded(want["dw"], 300))
    check(db, *bounded(want["db"], 300))
    r2 = torch.empty_like(r)  # the residual's scale alone
    fp8.fp8_norm_fwd(None, r, r2, None, pre=KIND["none"], res_scale=0.5)
    assert torch.equal(r2, r * 0.5)


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 130), (130, 264), (257, 1001), (3, 12300), (128, 384)])
@pytest.mark.parametrize("res", [F32, BF16])
def test_norm_codes_are_those_of_the_values(rows, cols, res):
    """The codes of x equal the casts of x in binary32: what a float32 h gives for the same values."""
    h, r, p, _, _ = norm_inputs(rows, cols, BF16, res, "layer", "rms", "channel")
    kinds = dict(pre=KIND["layer"], post=KIND["rms"])
    stats = torch.empty(rows, 4, device="cuda")
    r_out, x = torch.empty_like(r), torch.empty_like(h)
    xr, xc = row_blocks(rows, cols), col_blocks(rows, cols)
    fp8.fp8_norm_fwd(h, r, r_out, stats, **kinds, **p, x=x, margin=1, x_q=xr.q, x_s=xr.s, x_q_col=xc.q, x_s_col=xc.s)
    # r_out is stored: the norm of it, with a float32 output, is x before its rounding
    x32 = torch.empty(rows, cols, device="cuda")
    fp8.fp8_norm_fwd(None, r_out.float(), None, stats, w=p["w"], b=p["b"], pre=KIND["layer"], x=x32)
    assert torch.equal(x32.to(BF16), x)
    check_codes(xr, f64(x32), "e4m3", 1, 128, 1, "rows")
    check_codes(xc, f64(x32), "e4m3", 128, 1, 1, "columns")
    only = row_blocks(rows, cols)
    fp8.fp8_norm_fwd(h, r, r_out, None, **kinds, **p, margin=1, x_q=only.q, x_s=only.s)
    assert torch.equal(only.q, xr.q) and torch.equal(only.s, xr.s)
    assert fp8.fp8_get_status() == 0


def test_norm_of_rows_that_are_not_finite():
    h, r, p, dx, dr_out = norm_inputs(9, 300, BF16, F32, "layer", "rms", "channel")
    clean = run_norm(h, r, p, dx, dr_out, "layer", "rms")
    h, r = h.clone(), r.clone()
    h[3, 7], r[5, 299] = float("inf"), float("nan")
    r_out, x = torch.empty_like(r), torch.empty_like(h)
    codes = row_blocks(9, 300)
    fp8.fp8_norm_fwd(h, r, r_out, None, pre=KIND["layer"], post=KIND["rms"], **p, x=x, x_q=codes.q, x_s=codes.s)
    assert bool(x[3].isnan().all()) and bool(x[5].isnan().all())
    keep = [i for i in range(9) if i not in (3, 5)]
    assert torch.equal(x[keep], clean[1][keep]) and torch.equal(r_out[keep], clean[0][keep])
    assert fp8.fp8_get_status() == fp8.FP8_STATUS_NONFINITE


def test_norm_of_no_rows():
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    h, r, w = e(0, 64), e(0, 64), torch.ones(64, device="cuda")
    fp8.fp8_norm_fwd(h, r, e(0, 64), e(0, 4), w=w, x=e(0, 64))
    dw = torch.full((64,), GUARD, device="cuda")
    fp8.fp8_norm_bwd(e(0, 64), None, h, r, e(0, 4), w=w, dw=dw, dh=e(0, 64))
    assert not dw.any()


def test_norm_gradients_against_differences():
    """A function of the outputs, differenced in binary64 on the definition, against the kernel's gradients."""
    h, r, p, dx, dr_out = norm_inputs(4, 40, F32, F32, "layer", "rms", 2)
    r_out, _, dh, dr, grads = run_norm(h, r, p, dx, dr_out, "layer", "rms")

    def value(**over):
        q = {"h": h, "r": r, **p} | over
        n = Norm64(q["h"], q["r"], q["r"], "layer", "rms", q["w"], q["b"], q["post_w"], q["post_b"], q["gate"], 0.75)
        full = Norm64(q["h"], q["r"], n.r_new, "layer", "rms", q["w"], q["b"], q["post_w"], q["post_b"], q["gate"], 0.75)
        return float((full.x * dx.double()).sum() + (full.r_new * dr_out.double()).sum())

    for name, grad in {"h": dh, "r": dr, **{k[1:]: v for k, v in grads.items()}}.items():
        t = {"h": h, "r": r, **p}[name].double()
        d = torch.randn(t.shape, device="cuda", generator=rng(name), dtype=torch.float64)
        e = 1e-8
        diff = (value(**{name: t + e * d}) - value(**{name: t - e * d})) / (2 * e)
        got = float((grad.double() * d).sum())
        # the row of zeros has rstd = EPS^-1/2 in either norm: a step e is e / EPS of what the second one's root is
        # made of, and the difference is off by the square of that, three times; binary64's rounding of the value goes
        # by 1 / e; the kernel's by binary32's units
        scale = float((grad.double().abs() * d.abs()).sum())
        bound = scale * (3 * (8 * e / EPS) ** 2 + 600 * U) + 160 * 2.0 ** -52 * (1 + abs(value())) / e
        assert abs(got - diff) <= bound, name


# ---------------------------------------------------------------- log probabilities
def logits_of(rows, cols, dtype, pad=0, offset=0, seed=0, std=3.0):
    g = rng(rows, cols, seed, "logits")
    z = normal(g, rows, cols, std=std)
    t = torch.randint(0, cols, (rows,), device="cuda", generator=g)
    z[torch.arange(rows, device="cuda"), t] += 6.0
    if rows > 2:
        t[1] = -1
    return Strided(rows, cols, dtype, pad, offset, z), t, g


def run_of(cols):
    """Terms that a thread adds up in a row, at the most: every CTA has 128 threads or more, and 8 elements a vector."""
    return cols // 128 + 8


def top_reference(z, n):
    key = torch.where(z.isnan(), torch.full_like(z, float("inf"), dtype=torch.float64), z.double())
    order = torch.sort(key, dim=1, descending=True, stable=True)[1]
    nan_first = torch.gather(z.isnan(), 1, order)
    order = torch.gather(order, 1, torch.sort(nan_first.int(), dim=1, descending=True, stable=True)[1])
    return order[:, :n]


def run_logprob(z, tokens, g, inv_temp, top, grad=True):
    rows, cols = z.t.shape
    e = lambda *s: torch.full(s, GUARD, device="cuda")  # noqa: E731
    logp, ent, stats = e(rows), e(rows), e(rows, 4)
    top_logp, top_ids = e(rows, top), torch.zeros(rows, top, dtype=torch.int32, device="cuda")
    before = z.t.clone()
    fp8.fp8_logprob_fwd(z.t, tokens, logp, stats, inv_temp=inv_temp, entropy=ent, top_logp=top_logp if top else None,
                        top_ids=top_ids if top else None)
    ref = Rows64(z.t, inv_temp, run_of(cols))
    at = tokens.long().clamp_min(0)[:, None]
    there = tokens >= 0
    lp, a = ref.lp.gather(1, at)[:, 0], ref.a.gather(1, at)[:, 0]
    check(logp, torch.where(there, lp, 0.0), ref.logp_bound(lp, a), "logp")
    check(ent, ref.entropy, ref.entropy_bound(), "entropy")
    if top:
        ids = top_reference(z.t, top)
        assert torch.equal(top_ids.long(), ids)
        lt = ref.lp.gather(1, ids)
        check(top_logp, lt, ref.logp_bound(lt, ref.a.gather(1, ids)), "top")
    plain = e(rows)  # without the entropy: another instance of the kernel
    fp8.fp8_logprob_fwd(z.t, tokens.int(), plain, None, inv_temp=inv_temp)
    check(plain, torch.where(there, lp, 0.0), ref.logp_bound(lp, a), "logp alone")
    if not grad:
        return logp, ent, stats
    dlogp = torch.randn(rows, device="cuda", generator=g)
    dent = torch.randn(rows, device="cuda", generator=g) * 0.3
    for gl, ge in ((dlogp, None), (None, dent), (dlogp, dent)):
        d = Strided(rows, cols, z.t.dtype, z.t.stride(0) - cols if rows > 1 else 0, 0)
        fp8.fp8_logprob_bwd(z.t, None if gl is None else tokens, stats, gl, inv_temp=inv_temp, dentropy=ge, dlogits=d.t)
        v, b = logprob_grad(ref, tokens, gl, ge, inv_temp)
        check(d.t, v, b, "dlogits")
        assert d.intact()
    assert torch.equal(z.t, before) and z.intact()
    assert fp8.fp8_get_status() == 0
    return logp, ent, stats


def logprob_grad(ref, tokens, gl, ge, inv_temp):
    v, b = torch.zeros_like(ref.p), torch.zeros_like(ref.p)
    if gl is not None:
        w = torch.where(tokens >= 0, gl, 0.0).double()[:, None]
        hit = torch.zeros_like(ref.p).scatter_(1, tokens.long().clamp_min(0)[:, None], 1.0)
        v, b = w * (hit - ref.p), w.abs() * (ref.p * (ref.p_units + 8) + 8 * hit)
    if ge is not None:
        w = ge.double()[:, None]
        low = torch.special.entr(ref.p)
        v = v + w * (low - ref.p * ref.entropy[:, None])
        off = ref.entropy_bound()[:, None] / U
        b = b + w.abs() * ref.p * ((ref.p_units + 8) * (ref.a + ref.log_total.abs()[:, None] + ref.entropy[:, None]) + off)
    return v * inv_temp, b * inv_temp * U


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("size", [(1, 1), (2, 7), (3, 100), (5, 1001), (4, 4096), (1, 50304), (2, 50257), (40, 2056), (300, 515),
                                  (1, 131072)])
def test_logprob(size, dtype):
    z, tokens, g = logits_of(*size, dtype)
    run_logprob(z, tokens, g, 1.0, min(size[1], 20))
    run_logprob(z, tokens, g, 0.6, min(size[1], 32), grad=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (16, 8), (5, 3), (1, 2)])
def test_logprob_of_strided_and_unaligned_rows(pad, offset, dtype):
    z, tokens, g = logits_of(6, 5000, dtype, pad, offset)
    run_logprob(z, tokens, g, 1.5, 7)


@pytest.mark.parametrize("rows", [2, 700])
def test_top_alternatives_with_ties_and_masks(rows):
    cols = 9000
    z = torch.full((rows, cols), -math.inf, device="cuda")
    z[0, ::2] = 1.0                                  # a constant: the lowest columns
    z[1, [8999, 17, 4000]] = torch.tensor([2.0, 1.0, 2.0], device="cuda")  # fewer finite logits than alternatives
    if rows > 2:
        z[2] = 0.0
        z[3] = torch.finfo(BF16).min                 # a mask of the type's lowest value
        z[3, 100:103] = 5.0
        z[4, ::2048] = torch.arange(5, device="cuda").float()
        z[5] = torch.arange(cols, device="cuda").float().div(64).floor()  # ascending, in steps
        z[6] = -torch.arange(cols, device="cuda").float()
        z[7] = torch.randint(-2, 2, (cols,), device="cuda", generator=rng("t")).float()
        z[8] = 0.0
        z[8, ::2] = -0.0
        z[9, 5], z[9, 4] = 1.0, -1.0
        # large values at a stride of the threads' own: few threads hold thousands of them
        z[10] = torch.where(torch.arange(cols, device="cuda") % 2048 < 300, 3.0 + torch.arange(cols, device="cuda") % 7, 0.0)
    for dtype in (BF16, F32):
        t = Strided(rows, cols, dtype, values=z)
        for top in (1, 20, 32):
            e = lambda *s: torch.full(s, GUARD, device="cuda")  # noqa: E731
            lp, ids = e(rows, top), torch.zeros(rows, top, dtype=torch.int32, device="cuda")
            fp8.fp8_logprob_fwd(t.t, None, None, None, top_logp=lp, top_ids=ids)
            assert torch.equal(ids.long(), top_reference(t.t, top)), (dtype, top)
            ref = Rows64(t.t, 1.0, run_of(cols))
            want = ref.lp.gather(1, ids.long())
            fine = want.isfinite()
            assert torch.equal(fine, lp.isfinite()) and bool((lp[~fine] == -math.inf).all())
            b = ref.logp_bound(ref.lp, ref.a).gather(1, ids.long())
            check(torch.where(fine, lp, 0.0), torch.where(fine, want, 0.0), torch.where(fine, b, 0.0))


@pytest.mark.parametrize("cols,stride", [(65536, 4096), (65536, 8192), (131072, 2048)])
def test_top_alternatives_that_few_threads_hold(cols, stride):
    """Thousands of large logits in the columns of a few threads, more than the list of candidates takes."""
    g = rng(cols, stride)
    z = torch.zeros(3, cols, device="cuda")
    at = torch.arange(cols, device="cuda") % stride < 200
    z[:, at] = 10.0 + torch.randint(0, 50, (3, int(at.sum())), device="cuda", generator=g).float() / 4
    for rows in (1, 3):
        ids = torch.zeros(rows, 32, dtype=torch.int32, device="cuda")
        lp = torch.empty(rows, 32, device="cuda")
        fp8.fp8_logprob_fwd(z[:rows], None, None, None, top_logp=lp, top_ids=ids)
        assert torch.equal(ids.long(), top_reference(z[:rows], 32))
    big = z[:1].repeat(700, 1)
    ids, lp = torch.zeros(700, 32, dtype=torch.int32, device="cuda"), torch.empty(700, 32, device="cuda")
    fp8.fp8_logprob_fwd(big, None, None, None, top_logp=lp, top_ids=ids)
    assert torch.equal(ids.long(), top_reference(z[:1], 32).expand(700, 32))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rows_without_a_distribution_and_values_that_are_not_finite(dtype):
    rows, cols = 6, 3001
    z, tokens, g = logits_of(rows, cols, dtype)
    tokens = tokens.clamp_min(0)
    z.t[2] = -math.inf
    z.t[3, 11], z.t[4, 3000] = math.nan, math.inf
    tokens[5] = 9
    z.t[5, 9] = -math.inf  # a masked token
    e = lambda *s: torch.full(s, GUARD, device="cuda")  # noqa: E731
    logp, ent, stats, top, ids = e(rows), e(rows), e(rows, 4), e(rows, 3), torch.zeros(rows, 3, dtype=torch.int32, device="cuda")
    fp8.fp8_logprob_fwd(z.t, tokens, logp, stats, entropy=ent, top_logp=top, top_ids=ids)
    assert logp[2] == -math.inf and ent[2] == 0 and bool((top[2] == -math.inf).all()) and ids[2].tolist() == [0, 1, 2]
    assert logp[5] == -math.inf and bool(ent[5].isfinite())
    for i in (3, 4):
        assert bool(logp[i].isnan()) and bool(ent[i].isnan()) and bool(top[i].isnan().all())
    assert ids[3, 0] == 11 and ids[4, 0] == 3000
    d = torch.empty_like(z.t)
    one = torch.ones(rows, device="cuda")
    fp8.fp8_logprob_bwd(z.t, tokens, stats, one, dentropy=one, dlogits=d)
    assert not d[2].any() and bool(d[3].isnan().all()) and bool(d[4].isnan().all()) and bool(d[5].isfinite().all())
    ref = Rows64(z.t[5:], 1.0, run_of(cols))
    check(d[5:], *logprob_grad(ref, tokens[5:], one[5:], one[5:], 1.0))
    assert fp8.fp8_get_status() == 0


def test_a_token_beyond_the_vocabulary_is_reported_and_absent():
    z, tokens, _ = logits_of(4, 640, BF16)
    tokens[2], tokens[3] = 640, 1 << 40
    logp, stats = torch.empty(4, device="cuda"), torch.empty(4, 4, device="cuda")
    fp8.fp8_logprob_fwd(z.t, tokens, logp, stats)
    assert logp[2] == 0 and logp[3] == 0 and fp8.fp8_get_status() == fp8.FP8_STATUS_BAD_INDEX
    d = torch.full((4, 640), GUARD, dtype=BF16, device="cuda")
    fp8.fp8_logprob_bwd(z.t, tokens, stats, torch.ones(4, device="cuda"), dlogits=d)
    assert not d[1:].any() and d[0].any() and fp8.fp8_get_status() == fp8.FP8_STATUS_BAD_INDEX


def check_gradient_codes(call, rows, cols, dtype, fmt):
    """The codes that call(**outputs) writes are the casts of its float32 gradient, with d itself beside them or not."""
    d32 = torch.empty(rows, cols, device="cuda")
    call(F32, dlogits=d32)
    for with_d in (False, True):
        dr, dc = row_blocks(rows, cols), col_blocks(rows, cols)
        d = torch.empty(rows, cols, dtype=dtype, device="cuda") if with_d else None
        call(dtype, fmt=fp8.FP8_E5M2 if fmt == "e5m2" else fp8.FP8_E4M3, margin=1, d_q=dr.q, d_s=dr.s, d_q_col=dc.q,
             d_s_col=dc.s, dlogits=d)
        check_codes(dr, f64(d32), fmt, 1, 128, 1, "rows")
        check_codes(dc, f64(d32), fmt, 128, 1, 1, "columns")
        if with_d:
            assert torch.equal(d, d32.to(dtype))
    only = col_blocks(rows, cols)
    call(dtype, fmt=fp8.FP8_E5M2 if fmt == "e5m2" else fp8.FP8_E4M3, margin=1, d_q_col=only.q, d_s_col=only.s)
    assert torch.equal(only.q, dc.q) and torch.equal(only.s, dc.s)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (129, 300), (300, 1001), (40, 5000)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprob_gradient_codes(rows, cols, dtype):
    z, tokens, g = logits_of(rows, cols, dtype)
    stats, logp, ent = torch.empty(rows, 4, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    fp8.fp8_logprob_fwd(z.t, tokens, logp, stats, inv_temp=0.8, entropy=ent)
    gl, ge = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)

    def call(dt, **out):
        fp8.fp8_logprob_bwd(z.t.to(dt), tokens, stats, gl, inv_temp=0.8, dentropy=ge, **out)

    check_gradient_codes(call, rows, cols, dtype, "e5m2" if rows != 129 else "e4m3")


def test_gradients_in_the_logits_place():
    z, tokens, g = logits_of(30, 3000, BF16)
    logp, stats = torch.empty(30, device="cuda"), torch.empty(30, 4, device="cuda")
    gl = torch.randn(30, device="cuda", generator=g)
    ids, values = torch.topk(z.t.float() + 1, 9, dim=1)[::-1]
    lists = (torch.empty(30, 9, dtype=torch.int32, device="cuda"), torch.empty(30, 9, device="cuda"))
    for codes in (False, True):
        for distill in (False, True):
            if distill:
                fp8.fp8_distill_fwd(z.t, ids, values, logp, stats, *lists)
                bwd = lambda zz, **o: fp8.fp8_distill_bwd(zz, *lists, stats, gl, **o)  # noqa: E731
            else:
                fp8.fp8_logprob_fwd(z.t, tokens, logp, stats)
                bwd = lambda zz, **o: fp8.fp8_logprob_bwd(zz, tokens, stats, gl, **o)  # noqa: E731
            out = {}
            if codes:
                c = col_blocks(30, 3000)
                out = dict(d_q_col=c.q, d_s_col=c.s)
            d, over = torch.empty_like(z.t), z.t.clone()
            bwd(z.t, dlogits=d, **out)
            bwd(over, dlogits=over, **out)
            assert torch.equal(over, d)


# ---------------------------------------------------------------- distillation
def distill_inputs(rows, cols, K, dtype, form, vdtype=F32, seed=0, pad=0, offset=0, inv_temp=1.0):
    z, _, g = logits_of(rows, cols, dtype, pad, offset, seed)
    t = z.t.float() + normal(g, rows, cols)
    values, ids = torch.topk(t, K, dim=1)
    if form == "tail":
        values = values * inv_temp - torch.logsumexp(t * inv_temp, 1, keepdim=True)
    order = torch.randperm(K, device="cuda", generator=g)
    return z, values[:, order].to(vdtype).contiguous(), ids[:, order].contiguous(), g


def distill_reference(z, ids, values, form, inv_temp):
    """(rows, loss, its bound, gradient for a loss weight of 1, its bound)."""
    rows, cols = z.shape
    ref = Rows64(z, inv_temp, run_of(cols))
    ids, v = ids.long(), values.double()
    there = (ids >= 0) & (ids < cols) & ~torch.isneginf(v)
    for j in range(ids.shape[1]):  # listed before
        there[:, j] &= ~((ids[:, :j] == ids[:, j:j + 1]) & there[:, :j]).any(1)
    at = ids.clamp(0, cols - 1)
    if form == "top":
        lv = torch.where(there, v * inv_temp, -math.inf)
        lq = torch.where(there, lv - torch.logsumexp(lv, 1, keepdim=True), -math.inf)
        spread = torch.where(there, (lv.amax(1, keepdim=True) - lv), 0.0)
    else:
        lq = torch.where(there, v, -math.inf)
        spread = torch.where(there, v.abs(), 0.0)
    q = torch.exp(lq)
    # q: the rounded argument of exp, exp itself (2 units of 2^-23), the sum of at most 1024 and the division
    q_units = 4 * spread + 8 + (40 if form == "top" else 0)
    lp, a = ref.lp.gather(1, at), ref.a.gather(1, at)
    term = torch.where(q > 0, q * (lq - lp), 0.0)
    lp_b = ref.logp_bound(lp, a) / U
    size = torch.where(q > 0, q * ((lq - lp).abs() * (q_units + 8 + ids.shape[1]) + q_units + 4 * lq.abs() + 4 * lp.abs() + lp_b), 0.0)
    loss, off = term.sum(1), size.sum(1)
    listed = torch.zeros_like(ref.p, dtype=torch.bool)
    listed.scatter_(1, at, there) if rows == 0 else [listed[i].index_fill_(0, at[i][there[i]], True) for i in range(rows)]
    Q = q.sum(1)
    Q_off = (q * q_units).sum(1) + 40
    any_ = there.any(1)
    dense = torch.zeros_like(ref.p).scatter_add_(1, at, torch.where(there, q, 0.0))
    dense_off = torch.zeros_like(ref.p).scatter_add_(1, at, torch.where(there, q * q_units, 0.0))
    if form == "top":
        w = any_.double()[:, None]
        d, d_off = w * ref.p - dense, ref.p * (ref.p_units + 8) + dense_off + 4 * dense
    else:
        q_r = (1.0 - Q).clamp_min(0.0)
        p_r = torch.where(listed, 0.0, ref.p).sum(1)
        rest = (q_r > 0) & (p_r > 0)
        ratio = torch.where(rest, q_r / p_r.clamp_min(1e-300), 0.0)
        far = torch.where(listed, 0.0, ref.p * ref.p_units).sum(1) / p_r.clamp_min(1e-300)  # relative error of p_r, units
        lr = torch.where(rest, torch.log(ratio.clamp_min(1e-300)), 0.0)
        loss = loss + torch.where(rest, q_r * lr, 0.0)
        off = off + torch.where(rest, (Q_off + 2) * (lr.abs() + 1) + q_r * (far + ref.total_units + 8 * lr.abs() + 8 + 4 * torch.log(p_r.clamp_min(1e-300)).abs()), 0.0)
        whole = Q + torch.where(rest, q_r, 0.0)
        f = torch.where(listed, whole[:, None], (whole - ratio)[:, None])
        f_off = Q_off[:, None] * 2 + torch.where(listed, 0.0, (torch.where(rest, (Q_off + 2) / p_r.clamp_min(1e-300), 0.0)
                                                                + ratio * (far + ref.total_units + 8))[:, None])
        d, d_off = ref.p * f - dense, ref.p * (f.abs() * (ref.p_units + 8) + f_off) + dense_off + 4 * dense
    none = ref.none & any_
    loss = torch.where(any_, loss, 0.0).where(~none, math.inf)
    d = torch.where(none[:, None], 0.0, d) * inv_temp
    return loss, off * U, d, d_off * U * inv_temp


def run_distill(z, ids, values, g, form, inv_temp):
    rows, cols = z.t.shape
    K = ids.shape[1]
    loss, stats = torch.full((rows,), GUARD, device="cuda"), torch.empty(rows, 4, device="cuda")
    li, lq = torch.full((rows, K), -7, dtype=torch.int32, device="cuda"), torch.full((rows, K), GUARD, device="cuda")
    fp8.fp8_distill_fwd(z.t, ids, values, loss, stats, li, lq, form=FORM[form], inv_temp=inv_temp)
    want, off, d64, d_off = distill_reference(z.t, ids, values, form, inv_temp)
    assert bool((li[:, 1:] >= li[:, :-1]).all())
    fine = want.isfinite()
    assert torch.equal(loss.isfinite(), fine) and bool((loss[~fine] == math.inf).all())
    check(torch.where(fine, loss, 0.0), torch.where(fine, want, 0.0), torch.where(fine, off, 0.0), "loss")
    w = torch.randn(rows, device="cuda", generator=g)
    d = Strided(rows, cols, z.t.dtype, z.t.stride(0) - cols if rows > 1 else 0, 0)
    fp8.fp8_distill_bwd(z.t, li, lq, stats, w, inv_temp=inv_temp, dlogits=d.t)
    wd = w.double()[:, None]
    check(d.t, d64 * wd, d_off * wd.abs() + 8 * U * (d64 * wd).abs(), "dlogits")
    assert d.intact() and z.intact()
    return loss, stats, li, lq


@pytest.mark.parametrize("form", ["top", "tail"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("size", [(1, 1, 1), (2, 9, 3), (5, 130, 130), (3, 1001, 7), (4, 4096, 64), (1, 50257, 200), (300, 515, 16),
                                  (2, 20000, 1024)])
def test_distill(size, dtype, form):
    rows, cols, K = size
    z, values, ids, g = distill_inputs(rows, cols, K, dtype, form)
    run_distill(z, ids, values, g, form, 1.0)
    z, values, ids, g = distill_inputs(rows, cols, K, dtype, form, vdtype=dtype, inv_temp=0.5)
    run_distill(z, ids.int(), values, g, form, 0.5)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("form", ["top", "tail"])
@pytest.mark.parametrize("pad,offset", [(3, 0), (0, 1), (5, 3), (8, 8)])
def test_distill_of_strided_and_unaligned_rows(pad, offset, form):
    for dtype in (BF16, F32):
        z, values, ids, g = distill_inputs(5, 3000, 33, dtype, form, pad=pad, offset=offset)
        ids[0, :5] = torch.tensor([0, 1, 2999, 2998, 5], device="cuda")  # the row's ends
        run_distill(z, ids, values, g, form, 1.0)


@pytest.mark.parametrize("form", ["top", "tail"])
def test_distill_entries_that_are_absent(form):
    z, values, ids, g = distill_inputs(7, 2000, 12, F32, form)
    ids[0] = -1                              # nothing listed
    values[1] = -math.inf
    ids[2, 3:] = -1
    ids[3, 6], ids[3, 9] = ids[3, 2].item(), ids[3, 2].item()  # listed again
    values[4, ::2] = -math.inf
    z.t[5] = -math.inf                       # a student without a distribution
    z.t[6, ids[6, 0]] = -math.inf            # one that excludes what the teacher expects
    run_distill(z, ids, values, g, form, 1.0)
    assert fp8.fp8_get_status() == 0
    ids[2, 5] = 2000
    run_distill(z, ids, values, g, form, 1.0)
    assert fp8.fp8_get_status() == fp8.FP8_STATUS_BAD_INDEX


@pytest.mark.parametrize("form", ["top", "tail"])
@pytest.mark.parametrize("rows,cols,K", [(1, 1, 1), (3, 130, 40), (129, 300, 17), (300, 1001, 200)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distill_gradient_codes(rows, cols, K, dtype, form):
    z, values, ids, g = distill_inputs(rows, cols, K, dtype, form)
    if rows > 2:
        ids[2, 0] = -1
        ids[1] = torch.arange(K, device="cuda") + 64 if cols > K + 64 else torch.arange(K, device="cuda")  # all in a tile or two
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda")
    li, lq = torch.empty(rows, K, dtype=torch.int32, device="cuda"), torch.empty(rows, K, device="cuda")
    fp8.fp8_distill_fwd(z.t, ids, values, loss, stats, li, lq, form=FORM[form])
    w = torch.randn(rows, device="cuda", generator=g)

    def call(dt, **out):
        fp8.fp8_distill_bwd(z.t.to(dt), li, lq, stats, w, **out)

    check_gradient_codes(call, rows, cols, dtype, "e5m2")


def test_losses_of_no_rows():
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    i = lambda *s: torch.empty(s, dtype=torch.int64, device="cuda")  # noqa: E731
    fp8.fp8_logprob_fwd(e(0, 9), i(0), e(0), e(0, 4))
    fp8.fp8_logprob_bwd(e(0, 9), i(0), e(0, 4), e(0), dlogits=e(0, 9))
    fp8.fp8_distill_fwd(e(0, 9), i(0, 2), e(0, 2), e(0), e(0, 4), i(0, 2).int(), e(0, 2))
    fp8.fp8_distill_bwd(e(0, 9), i(0, 2).int(), e(0, 2), e(0, 4), e(0), dlogits=e(0, 9))
