"""Norms, log probabilities and distillation: what is refused on the host before anything reaches a GPU, the
binding's own checks, and the references of the GPU tests against torch."""
import ctypes
import math
import os

import pytest
import torch

from _passes import EPS, Norm64, Rows64

FAKE = 0x10000  # never read: every call below fails its host checks first


@pytest.fixture(scope="module")
def fp8():
    from fp8_mixed_precision_tensor_b200 import build, fp8

    build.build()
    fp8.load_library()
    return fp8


def _b(fp8, q=FAKE, s=FAKE, ld=256):
    return ctypes.byref(fp8._Blocks(q, s, ld))


def norm_params(fp8, **kw):
    p = fp8._NormParams()
    p.rows, p.cols, p.dtype, p.res_dtype, p.pre, p.post = 8, 256, fp8.FP8_DT_BF16, fp8.FP8_DT_F32, 1, 0
    p.gate_rows, p.ld_gate, p.res_scale, p.eps = 8, 256, 1.0, 1e-5
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_norm_forward_rejects_bad_arguments(fp8):
    lib = fp8.load_library()
    V = fp8._Vec

    def call(h=FAKE, ldh=256, r=FAKE, ldr=256, ro=FAKE, ldro=256, stats=FAKE, x=FAKE, ldx=256, margin=0, row=None,
             col=None, **kw):
        return lib.fp8_norm_fwd(ctypes.byref(norm_params(fp8, **kw)), h, ldh, r, ldr, ro, ldro, stats, x, ldx, margin, row, col, None)

    INV, UNA, UNS = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_UNALIGNED, fp8.FP8_ERR_UNSUPPORTED
    for kw in (dict(dtype=3), dict(res_dtype=2), dict(dtype=0, res_dtype=1), dict(rows=-1), dict(cols=-1), dict(pre=3),
               dict(post=-1), dict(eps=-1.0), dict(eps=math.nan), dict(res_scale=math.inf), dict(margin=65), dict(margin=-1),
               dict(r=None), dict(ldh=255), dict(ldr=255), dict(ldro=255), dict(ldx=255), dict(ro=None), dict(h=None, post=1),
               dict(h=None, gate=V(FAKE, 0)), dict(pre=0), dict(col=_b(fp8), stats=None), dict(row=_b(fp8, None)),
               dict(row=_b(fp8, ld=240)), dict(w=V(FAKE, 5)), dict(gate=V(FAKE, 0), gate_rows=0),
               dict(gate=V(FAKE, 0), ld_gate=255), dict(h=None, ro=None, res_scale=0.5)):
        assert call(**kw) == INV, kw
    for kw in (dict(h=FAKE + 1), dict(r=FAKE + 2), dict(x=FAKE + 1), dict(stats=FAKE + 4), dict(w=V(FAKE + 2, 0)),
               dict(b=V(FAKE + 1, 1)), dict(row=_b(fp8, FAKE + 8)), dict(col=_b(fp8, ld=264))):
        assert call(**kw) == UNA, kw
    for kw in (dict(cols=16385, ldh=40000, ldr=40000, ldro=40000, ldx=40000), dict(rows=2 ** 31 - 1)):
        assert call(**kw) == UNS, kw
    assert lib.fp8_norm_fwd(None, FAKE, 256, FAKE, 256, FAKE, 256, FAKE, FAKE, 256, 0, None, None, None) == INV
    assert call(rows=0) == fp8.FP8_OK and call(cols=0) == fp8.FP8_OK


def test_norm_backward_rejects_bad_arguments(fp8):
    lib = fp8.load_library()
    V = fp8._Vec

    def call(dx=FAKE, dro=FAKE, h=FAKE, ro=FAKE, stats=FAKE, dh=FAKE, dr=FAKE, ws=FAKE, n=1 << 30, lddx=256, lddh=256,
             grads=None, **kw):
        g = fp8._NormGrads()
        g.ld_gate = 256
        for k, v in (grads or {}).items():
            setattr(g, k, v)
        return lib.fp8_norm_bwd(ctypes.byref(norm_params(fp8, **kw)), dx, lddx, dro, 256, h, 256, ro, 256, stats, dh, lddh,
                                dr, 256, ctypes.byref(g), ws, n, None)

    INV, UNA = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_UNALIGNED
    w = dict(w=V(FAKE, 0))
    for kw in (dict(dx=None), dict(pre=0), dict(pre=0, dx=None, grads=w), dict(ro=None), dict(stats=None), dict(h=None),
               dict(grads=dict(post_w=V(FAKE, 0))), dict(grads=dict(gate=V(FAKE, 0))), dict(lddx=255), dict(lddh=255),
               dict(dh=None, dr=None), dict(grads=w, ws=None, n=0), dict(grads=w, n=fp8.fp8_norm_workspace_bytes(8, 256) - 1),
               dict(gate=V(FAKE, 0), grads=dict(gate=V(FAKE, 0), ld_gate=255)), dict(grads=dict(w=V(FAKE, 7)))):
        assert call(**kw) == INV, kw
    for kw in (dict(dx=FAKE + 1), dict(dr=FAKE + 2), dict(ws=FAKE + 8, grads=w), dict(stats=FAKE + 8),
               dict(grads=dict(w=V(FAKE + 1, 1)))):
        assert call(**kw) == UNA, kw
    assert call(cols=0) == fp8.FP8_OK


def test_norm_workspace_is_that_of_the_partial_sums(fp8):
    need = fp8.fp8_norm_workspace_bytes
    assert need(0, 5) == 0 and need(5, 0) == 0 and need(-1, 4) == 0 and need(4, 40000) == 0 and need(4, 4, 0) == 0
    for rows in (1, 7, 148, 149, 4096, 100003):
        for cols in (1, 64, 4096, 4097, 12288, 16384):
            for gate_rows in (1, 3, rows, 10 * rows):
                n = need(rows, cols, gate_rows)
                line = 2 * (-(-cols // 8) * 8) * 4  # whole groups of eight
                sums = n // line
                assert n == sums * line and 2 <= sums <= 3 * 2 * 148 + -(-rows // gate_rows) + 1


def test_losses_reject_bad_arguments(fp8):
    lib = fp8.load_library()
    INV, UNA, UNS = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_UNALIGNED, fp8.FP8_ERR_UNSUPPORTED
    base = dict(z=FAKE, dt=1, rows=4, cols=256, ld=256, beta=1.0)
    bad_rows = (dict(z=None), dict(dt=3), dict(rows=-1), dict(cols=-1), dict(ld=255), dict(beta=0.0), dict(beta=-1.0),
                dict(beta=math.nan), dict(beta=math.inf))

    def fwd(tok=FAKE, tb=8, logp=FAKE, ent=None, top=0, tl=None, ti=None, stats=FAKE, **kw):
        a = {**base, **kw}
        return lib.fp8_logprob_fwd(*a.values(), tok, tb, logp, ent, top, tl, ti, stats, None)

    for kw in (*bad_rows, dict(tok=None), dict(logp=None), dict(tb=2), dict(top=33, tl=FAKE, ti=FAKE), dict(top=-1),
               dict(top=2, tl=FAKE), dict(top=2, ti=FAKE), dict(top=20, tl=FAKE, ti=FAKE, cols=19),
               dict(tok=None, logp=None, stats=None), dict(cols=0), dict(tl=FAKE, ti=FAKE)):
        assert fwd(**kw) == INV, kw
    for kw in (dict(z=FAKE + 1), dict(tok=FAKE + 4), dict(stats=FAKE + 4), dict(logp=FAKE + 2), dict(ent=FAKE + 1)):
        assert fwd(**kw) == UNA, kw
    assert fwd(rows=2 ** 31 - 1) == UNS and fwd(rows=0) == fp8.FP8_OK

    def bwd(tok=FAKE, tb=8, stats=FAKE, g=FAKE, ge=None, fmt=1, margin=0, row=None, col=None, d=FAKE, ldd=256, **kw):
        a = {**base, **kw}
        return lib.fp8_logprob_bwd(*a.values(), tok, tb, stats, g, ge, fmt, margin, row, col, d, ldd, None)

    for kw in (*bad_rows, dict(tok=None), dict(g=None), dict(tok=None, g=None), dict(stats=None), dict(fmt=2), dict(margin=65),
               dict(d=None), dict(ldd=255), dict(row=_b(fp8, None)), dict(col=_b(fp8, ld=240)), dict(tb=3)):
        assert bwd(**kw) == INV, kw
    for kw in (dict(d=FAKE + 1), dict(stats=FAKE + 8), dict(col=_b(fp8, FAKE + 8)), dict(g=FAKE + 1), dict(tok=FAKE + 4)):
        assert bwd(**kw) == UNA, kw

    def dfwd(form=0, top=8, ids=FAKE, ib=4, v=FAKE, vd=0, loss=FAKE, stats=FAKE, li=FAKE, lq=FAKE, **kw):
        a = {**base, **kw}
        return lib.fp8_distill_fwd(*a.values(), form, top, ids, ib, v, vd, loss, stats, li, lq, None)

    for kw in (*bad_rows, dict(form=2), dict(top=0), dict(top=1025), dict(ids=None), dict(v=None), dict(loss=None), dict(ib=2),
               dict(stats=None), dict(li=None), dict(lq=None), dict(vd=3), dict(cols=0)):
        assert dfwd(**kw) == INV, kw
    for kw in (dict(ids=FAKE + 4, ib=8), dict(v=FAKE + 2), dict(stats=FAKE + 4), dict(li=FAKE + 2), dict(z=FAKE + 1)):
        assert dfwd(**kw) == UNA, kw
    assert dfwd(cols=2 ** 20 + 1, ld=2 ** 21) == UNS

    def dbwd(top=8, li=FAKE, lq=FAKE, stats=FAKE, g=FAKE, fmt=1, margin=0, row=None, col=None, d=FAKE, ldd=256, **kw):
        a = {**base, **kw}
        return lib.fp8_distill_bwd(*a.values(), top, li, lq, stats, g, fmt, margin, row, col, d, ldd, None)

    for kw in (*bad_rows, dict(top=0), dict(top=1025), dict(li=None), dict(lq=None), dict(g=None), dict(stats=None), dict(d=None),
               dict(fmt=2), dict(margin=-1)):
        assert dbwd(**kw) == INV, kw
    assert dbwd(cols=2 ** 20 + 1, ld=2 ** 21, ldd=2 ** 21) == UNS
    assert dbwd(rows=0) == fp8.FP8_OK


def test_the_binding_takes_device_tensors_only(fp8):
    x, s = torch.zeros(4, 64), torch.zeros(4, 4)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.fp8_norm_fwd(x, x, x, s)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.fp8_norm_bwd(x, None, x, x, s, dh=x)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.fp8_logprob_fwd(x, torch.zeros(4, dtype=torch.int64), s[:, 0], s)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.fp8_distill_bwd(x, s.int(), s, s, s[:, 0], dlogits=x)
    with pytest.raises(TypeError):
        fp8.fp8_logprob_fwd(x.double(), None, None, s)
    with pytest.raises(ValueError, match="gradient is needed"):
        fp8.fp8_norm_bwd(None, None, None, None, s)


# ---------------------------------------------------------------- the references
@pytest.mark.parametrize("pre,post,gate", [("rms", "rms", 1), ("layer", "layer", 3), ("layer", "none", 0), ("none", "rms", 1)])
def test_norm_reference_is_what_autograd_gives(pre, post, gate):
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    rows, cols = 6, 20
    t = dict(h=rand(rows, cols), r=rand(rows, cols), w=rand(cols), b=rand(cols), post_w=rand(cols), post_b=rand(cols),
             gate=rand(gate, cols) if gate else None)
    if post == "none":
        t["post_w"] = t["post_b"] = None
    if pre == "none":
        t["w"] = t["b"] = None
    leaves = {k: v.clone().requires_grad_() for k, v in t.items() if v is not None}

    def norm(v, kind, w, b):
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, (cols,), w, b, EPS)
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w + b

    u = leaves["h"] if post == "none" else norm(leaves["h"], post, leaves["post_w"], leaves["post_b"])
    gv = leaves["gate"].repeat_interleave(rows // gate, 0) if gate else 1.0
    r_out = 0.7 * leaves["r"] + gv * u
    dx, dro = rand(rows, cols), rand(rows, cols)
    outs, weights = [r_out], [dro]
    if pre != "none":
        outs.append(norm(r_out, pre, leaves["w"], leaves["b"]))
        weights.append(dx)
    ref = Norm64(*(t[k] for k in ("h", "r")), r_out.detach(), pre, post, *(t[k] for k in ("w", "b", "post_w", "post_b", "gate")), 0.7)
    assert torch.allclose(ref.r_new, r_out.detach(), atol=1e-12)
    if pre != "none":
        assert torch.allclose(ref.x, outs[1].detach(), atol=1e-12)
    want = torch.autograd.grad(outs, list(leaves.values()), weights)
    got = ref.backward(dx, dro)
    for k, v in zip(leaves, want):
        assert torch.allclose(got["d" + k][0].view(v.shape), v, atol=1e-11), k


def test_softmax_reference_is_what_torch_gives():
    g = torch.Generator().manual_seed(6)
    z = torch.randn(5, 300, generator=g, dtype=torch.float64) * 4
    z[1, ::3] = -math.inf
    z[2] = -math.inf
    ref = Rows64(z, 0.5, 3)
    keep = [0, 1, 3, 4]
    assert torch.allclose(ref.lp[keep], torch.log_softmax(z * 0.5, 1)[keep], atol=1e-12)
    p = torch.softmax(z[keep] * 0.5, 1)
    assert torch.allclose(ref.p[keep], p) and torch.allclose(ref.entropy[keep], torch.special.entr(p).sum(1))
    assert not ref.p[2].any() and ref.entropy[2] == 0
    assert bool((ref.entropy_bound()[keep] > 0).all())


def test_the_message_of_an_unsupported_shape_names_these_limits(fp8):
    text = fp8.fp8_strerror(fp8.FP8_ERR_UNSUPPORTED)
    assert "16384" in text and "1048576" in text and os.linesep not in text
