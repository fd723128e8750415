"""Norms, log probabilities and distillation at their edges."""
import ctypes
import threading

import pytest
import torch

from fp8_mixed_precision_tensor_b200 import fp8
from fp8_mixed_precision_tensor_b200.block_linear import BlockLinear, BlockNorm
from test_gpu_block import row_blocks
from test_gpu_passes import BF16, F16, F32, FORM, GUARD, KIND, Strided, check_gradient_codes, normal, rng, run_distill


pytestmark = pytest.mark.gpu

ROUTES = ["calls", "python"]


@pytest.fixture
def route(request, monkeypatch):
    """The calls through the C++ module, or through Python alone."""
    if request.param == "python":
        fp8.load_library()
        monkeypatch.setattr(fp8, "_calls", fp8._PythonRoute())
    return request.param


# ---------------------------------------------------------------- no rows
@pytest.mark.parametrize("route", ROUTES, indirect=True)
@pytest.mark.parametrize("gates", [None, 1, 5])
def test_norm_gradients_of_no_rows_are_zero(gates, route):
    """Of every parameter, a gate's too, and nothing beside them is written."""
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    vec = lambda: torch.ones(72, device="cuda")  # noqa: E731
    gate = vec() if gates is None else torch.ones(gates, 72, device="cuda")
    out = {k: torch.full((72,), GUARD, device="cuda") for k in ("dw", "db", "dpost_w", "dpost_b")}
    d = Strided(gates or 1, 72, F32, pad=0 if gates is None else 8, values=torch.full((gates or 1, 72), GUARD, device="cuda"))
    dgate = d.t[0] if gates is None else d.t
    fp8.fp8_norm_bwd(e(0, 72), None, e(0, 72), e(0, 72), e(0, 4), pre=KIND["layer"], post=KIND["layer"], w=vec(), post_w=vec(),
                     post_b=vec(), gate=gate, dh=e(0, 72), dr=e(0, 72), dgate=dgate, **out)
    for k, t in out.items():
        assert not t.any(), k
    assert not dgate.any() and d.intact()


@pytest.mark.parametrize("shape", [(64,), (3, 64)])
def test_a_norm_that_got_no_tokens(shape):
    gate = torch.ones(shape, device="cuda", dtype=BF16)
    norm = BlockNorm(torch.ones(64, device="cuda"), post=KIND["rms"], post_w=torch.ones(64, device="cuda"), gate=gate)
    h = torch.empty(0, 64, device="cuda", dtype=BF16)
    junk = [torch.full(shape, GUARD, device="cuda", dtype=BF16) for _ in range(64)]
    del junk  # memory that the gradients may get
    norm.forward(h, h, keep=True)
    dh, dr, grads = norm.backward(h, h)
    assert dh.shape == dr.shape == (0, 64) and grads["gate"].shape == shape
    assert all(not g.any() for g in grads.values())


# ---------------------------------------------------------------- a float32 residual
def test_the_first_norm_of_a_float32_residual_writes_for_16_bit_layers():
    """A norm alone: x and its codes are those of the call, the layer behind it gives its type, and the residual's
    gradient has the residual's."""
    g = rng("first")
    r, w = normal(g, 70, 256), torch.ones(256, device="cuda", dtype=BF16)
    norm, lin = BlockNorm(w), BlockLinear(normal(g, 128, 256, std=0.05, dtype=BF16))
    want, stats, x32 = torch.empty(70, 256, device="cuda", dtype=BF16), torch.empty(70, 4, device="cuda"), torch.empty_like(r)
    fp8.fp8_norm_fwd(None, r, None, stats, w=w, x=want)
    fp8.fp8_norm_fwd(None, r, None, None, w=w, x=x32)
    r_out, x = norm.forward(None, r, dtype=BF16)
    assert torch.equal(x, want) and torch.equal(r_out, r)
    r_out, x = norm.forward(None, r, codes=True, keep=True, dtype=BF16)
    c = row_blocks(70, 256)
    fp8.fp8_block_cast(x32, fp8.FP8_E4M3, 0, c.q, c.s, None, None)
    assert x.dtype is BF16 and torch.equal(x.q, c.q) and torch.equal(x.s, c.s)
    y = lin.forward(x, keep=True)
    dx, dw = lin.backward(torch.ones_like(y))
    assert y.dtype is dx.dtype is dw.dtype is BF16
    none, dr, grads = norm.backward(dx, r)
    d = torch.empty_like(r)
    fp8.fp8_norm_bwd(dx, r, None, r, stats, w=w, dr=d)
    assert none is None and torch.equal(dr, d) and grads["w"].dtype is BF16


@pytest.mark.parametrize("h,r,dtype", [(BF16, F32, F32), (BF16, BF16, F32), (None, BF16, F32), (None, BF16, F16), (None, F32, torch.float64)])
def test_a_norm_gives_x_in_no_other_type(h, r, dtype):
    e = lambda t: None if t is None else torch.zeros(2, 8, device="cuda", dtype=t)  # noqa: E731
    with pytest.raises(ValueError, match="dtype"):
        BlockNorm(torch.ones(8, device="cuda")).forward(e(h), e(r), dtype=dtype)


@pytest.mark.parametrize("cols", [300000, 327680])
def test_a_tail_whose_marks_end_just_below_48_kb(cols):
    """8 KB for the list and 40 for the marks, beside what the kernel has of its own."""
    g = rng("marks", cols)
    z = Strided(75, cols, F16, values=normal(g, 75, cols, std=2.0))
    ids = torch.stack([torch.randperm(cols, device="cuda", generator=g)[:16] for _ in range(75)])
    values = torch.log_softmax(normal(g, 75, 17), 1)[:, :16].contiguous()
    run_distill(z, ids, values, g, "tail", 1.0)
    assert fp8.fp8_get_status() == 0


# ---------------------------------------------------------------- side by side
def codes_of(calls, rounds):
    """What each of `calls` (functions of the C library with their arguments) returns, made again and again in a thread
    of its own at the same time as the others: the interpreter is given up in each call."""
    found = [set() for _ in calls]
    start = threading.Barrier(len(calls))

    def run(k):
        f, args = calls[k]
        start.wait()
        for _ in range(rounds):
            found[k].add(f(*args))

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(calls))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    return found


def p_(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("shapes", [((4096, True), (4096, False)), ((9000, False), (12288, False))])
def test_norms_of_one_kernel_with_other_sizes_side_by_side(shapes):
    """A launch has the shared memory that it needs, whatever another thread launches meanwhile."""
    lib, n = fp8.load_library(), ctypes.c_size_t
    calls, backward, outs = [], [], []
    for cols, bias in shapes * 4:
        g = rng("side", cols, bias)
        h, r, w = normal(g, 2, cols, dtype=BF16), normal(g, 2, cols, dtype=BF16), torch.ones(cols, device="cuda")
        b = normal(g, cols) if bias else None
        r_out, x, st, dh, dr = torch.empty_like(r), torch.empty_like(h), torch.empty(2, 4, device="cuda"), torch.zeros_like(h), torch.zeros_like(r)
        s = torch.cuda.Stream()
        p = fp8._norm_params(h, r, 0, 2, cols, KIND["layer"], KIND["none"], w, b, None, None, None, 1.0, 1e-5)
        grads, stream, ld = fp8._NormGrads(), ctypes.c_void_p(s.cuda_stream), n(cols)
        calls.append((lib.fp8_norm_fwd, (p, p_(h), ld, p_(r), ld, p_(r_out), ld, p_(st), p_(x), ld, 0, None, None, stream)))
        backward.append((lib.fp8_norm_bwd, (p, p_(x), ld, None if bias else p_(r), n(0) if bias else ld, p_(h), ld, p_(r_out), ld, p_(st),
                                            p_(dh), ld, p_(dr), ld, grads, None, n(0), stream)))
        outs.append((s, w, b, h, r, st, r_out, x, dh, dr))
    torch.cuda.synchronize()
    for group in (calls, backward):
        alone = [f(*a) for f, a in group]
        assert alone == [0] * len(group)
        torch.cuda.synchronize()
        want = [[t.clone() for t in o[5:]] for o in outs]
        torch.cuda.synchronize()
        assert codes_of(group, 10000) == [{0}] * len(group)
        assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o[5:], w))


def test_tails_of_two_vocabularies_side_by_side():
    lib, n = fp8.load_library(), ctypes.c_size_t
    calls, outs = [], []
    for cols in (420000, 800000) * 3:
        g = rng("tails", cols)
        z = normal(g, 75, cols, dtype=BF16)
        ids = torch.randint(0, cols, (75, 4), device="cuda", generator=g)
        v = torch.full((75, 4), -2.0, device="cuda")
        o = [torch.empty(75, device="cuda"), torch.empty(75, 4, device="cuda"), torch.empty(75, 4, dtype=torch.int32, device="cuda"),
             torch.empty(75, 4, device="cuda")]
        s = torch.cuda.Stream()
        calls.append((lib.fp8_distill_fwd, (p_(z), fp8.FP8_DT_BF16, 75, cols, n(cols), 1.0, FORM["tail"], 4, p_(ids), 8, p_(v),
                                            fp8.FP8_DT_F32, *map(p_, o), ctypes.c_void_p(s.cuda_stream))))
        outs.append((s, z, ids, v, *o))
    torch.cuda.synchronize()
    assert [f(*a) for f, a in calls] == [0] * len(calls)
    torch.cuda.synchronize()
    want = [[t.clone() for t in o[4:]] for o in outs]
    torch.cuda.synchronize()
    assert codes_of(calls, 2000) == [{0}] * len(calls)
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o[4:], w))


# ---------------------------------------------------------------- lists
@pytest.mark.parametrize("form", ["top", "tail"])
def test_an_entry_listed_again_with_a_larger_value_counts_for_nothing(form):
    """The first of them counts, also where the value of another is the largest of the list by far."""
    g = rng("again", form)
    z = Strided(6, 700, F32, values=normal(g, 6, 700, std=2.0))
    ids = torch.stack([torch.randperm(700, device="cuda", generator=g)[:9] for _ in range(6)])
    values = normal(g, 6, 9, std=1.0) - 4.0
    for row, (at, of, v) in enumerate(((3, 0, 300.0), (8, 2, 120.0), (1, 0, 2e4), (5, 4, 88.0), (2, 1, float("nan")))):
        ids[row, at], values[row, at] = ids[row, of].item(), v
    if form == "tail":
        values = torch.where(values.isnan(), values, values.clamp_max(-3.0))
    values_of_reference = torch.where(values.isnan(), 0.0, values)  # (of the entry that does not count)
    loss, stats, li, lq = run_distill(z, ids, values_of_reference, rng("w", form), form, 1.0)
    more = [torch.empty_like(t) for t in (loss, stats, li, lq)]
    fp8.fp8_distill_fwd(z.t, ids, values, *more, form=FORM[form])
    assert all(torch.equal(a, b) for a, b in zip(more, (loss, stats, li, lq)))


def far_student(rows, cols, K, dtype, gaps, inv_temp=1.0):
    """Logits whose listed ones lie a gap above all others, and a teacher that gives the others a quarter."""
    g = rng("far", rows, cols, K, str(dtype), inv_temp)
    z = normal(g, rows, cols, std=1.5)
    ids = torch.stack([torch.randperm(cols, device="cuda", generator=g)[:K] for _ in range(rows)])
    gap = torch.tensor([gaps[i % len(gaps)] for i in range(rows)], device="cuda")[:, None]
    z.scatter_add_(1, ids, (gap / inv_temp).expand(-1, K))
    values = torch.log(0.75 * torch.softmax(normal(g, rows, K), 1))
    return Strided(rows, cols, dtype, values=z), values, ids, g


GAPS = (0.0, 30.0, 80.0, 84.0, 86.0, 87.0, 87.5, 88.0, 89.0, 95.0, 103.0, 120.0, 300.0, 600.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,cols,K", [(14, 515, 5), (14, 50257, 64), (200, 2056, 33), (28, 77, 70)])
def test_a_student_that_is_sure_of_what_is_listed(rows, cols, K, dtype):
    """The rest's term and gradient where its probability is below what binary32 holds: -log p' is of the gap's size."""
    z, values, ids, g = far_student(rows, cols, K, dtype, GAPS)
    run_distill(z, ids, values, g, "tail", 1.0)
    z, values, ids, g = far_student(rows, cols, K, dtype, GAPS, 4.0)
    run_distill(z, ids, values, g, "tail", 4.0)
    assert fp8.fp8_get_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_codes_of_a_sure_student(dtype):
    z, values, ids, g = far_student(150, 700, 20, dtype, GAPS)
    loss, stats = torch.empty(150, device="cuda"), torch.empty(150, 4, device="cuda")
    li, lq = torch.empty(150, 20, dtype=torch.int32, device="cuda"), torch.empty(150, 20, device="cuda")
    fp8.fp8_distill_fwd(z.t, ids, values, loss, stats, li, lq, form=FORM["tail"])
    w = torch.randn(150, device="cuda", generator=g)
    check_gradient_codes(lambda dt, **out: fp8.fp8_distill_bwd(z.t.to(dt), li, lq, stats, w, **out), 150, 700, dtype, "e5m2")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_student_that_excludes_all_that_is_not_listed(dtype):
    """Masked to -inf: p' is 0, and the rest has no term; masked by a large number it has one."""
    for mask in (-float("inf"), -1e4, -60000.0):
        g = rng("mask", mask, str(dtype))
        z = torch.full((5, 900), mask, device="cuda")
        ids = torch.stack([torch.randperm(900, device="cuda", generator=g)[:6] for _ in range(5)])
        z.scatter_(1, ids, normal(g, 5, 6))
        values = torch.log(0.9 * torch.softmax(normal(g, 5, 6), 1))
        s = Strided(5, 900, dtype, values=z)
        loss = torch.empty(5, device="cuda")
        stats, li, lq = torch.empty(5, 4, device="cuda"), torch.empty(5, 6, dtype=torch.int32, device="cuda"), torch.empty(5, 6, device="cuda")
        fp8.fp8_distill_fwd(s.t, ids, values, loss, stats, li, lq, form=FORM["tail"])
        zl = s.t.gather(1, ids).double()
        lp, q = torch.log_softmax(zl, 1), values.double().exp()  # (the others' e^-10000 is nothing to the sum)
        want = (q * (values.double() - lp)).sum(1)
        if mask > -float("inf"):
            rest = 1.0 - q.sum(1)
            lp_rest = mask_of(s.t, ids) + torch.tensor(894.0, device="cuda", dtype=torch.float64).log() - torch.logsumexp(zl, 1)
            want = want + rest * (rest.log() - lp_rest)
        # each product and sum rounded: some 20 units of what is added up, and 1 - sum q off by 8 units of 1
        size = 20 * (want.abs() + 10) + (8 * abs(mask) if mask > -float("inf") else 0)
        assert bool(((loss.double() - want).abs() <= 2.0 ** -24 * size).all()), mask
        d = torch.empty(5, 900, device="cuda")
        fp8.fp8_distill_bwd(s.t.float(), li, lq, stats, torch.ones(5, device="cuda"), dlogits=d)
        assert bool(d.isfinite().all())
        whole = 1.0 if mask > -float("inf") else float(q.sum(1)[0])
        rest = 0.0 if mask == -float("inf") else 0.1
        listed = torch.zeros(5, 900, dtype=torch.bool, device="cuda").scatter_(1, ids, True)
        out = d.masked_fill(listed, 0.0).double().sum(1)  # the rest's share of the gradient: -q' in all
        assert bool((out + rest).abs().max() <= 64 * 2.0 ** -24), mask
        got = d.double().gather(1, ids)
        assert bool((got - (lp.exp() * whole - q)).abs().max() <= 64 * 2.0 ** -24), mask


def mask_of(z, ids):
    """The masked logits' value, as stored."""
    return z.masked_fill(torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids, True), -float("inf")).amax(1).double()


@pytest.mark.parametrize("rows", [3, 200])
def test_a_rest_that_student_and_teacher_agree_about(rows):
    """One rare outcome listed: the loss is q' log(q' / p'), both almost 1.  q', p' and their ratio have four roundings,
    the sum one and the logarithm one; the listed term is 10^-4 of what it would need to count."""
    g = rng("agree", rows)
    z = normal(g, rows, 30000, std=0.1)
    ids = torch.randint(0, 30000, (rows, 1), device="cuda", generator=g)
    lp = torch.log_softmax(z.double(), 1)
    values = (lp.gather(1, ids) + 0.1).float()
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda")
    fp8.fp8_distill_fwd(z, ids, values, loss, stats, torch.empty(rows, 1, dtype=torch.int32, device="cuda"),
                        torch.empty(rows, 1, device="cuda"), form=FORM["tail"])
    lq = values.double()
    q, p = lq.exp()[:, 0], lp.gather(1, ids).exp()[:, 0]
    want = (q * (lq - lp.gather(1, ids))[:, 0]) + (1 - q) * ((1 - q) / (1 - p)).log()
    assert bool(((loss.double() - want).abs() <= 6 * 2.0 ** -24).all())


# ---------------------------------------------------------------- unsorted
@pytest.mark.parametrize("codes", [False, True])
def test_a_list_in_another_order_is_read_inside_its_bounds(codes):
    """The last rows' entries in falling order, and numbers that are no columns: nothing beyond the list is looked at, and
    rows whose list is in order have their gradient."""
    g = rng("order")
    rows, cols, K = 140, 300, 40
    z = normal(g, rows, cols)
    ids = torch.stack([torch.randperm(cols, device="cuda", generator=g)[:K] for _ in range(rows)])
    loss, stats, li, lq = (torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda"),
                           torch.empty(rows, K, dtype=torch.int32, device="cuda"), torch.empty(rows, K, device="cuda"))
    fp8.fp8_distill_fwd(z, ids, normal(g, rows, K), loss, stats, li, lq)
    other = li.clone()
    other[70:] = li[70:].flip(1)
    other[-1] = torch.tensor([-2 ** 31, -1, 2 ** 31 - 1, cols] * (K // 4), dtype=torch.int32, device="cuda")
    w = torch.randn(rows, device="cuda", generator=g)

    def values(ids_):
        if not codes:
            d = torch.empty_like(z)
            fp8.fp8_distill_bwd(z, ids_, lq, stats, w, dlogits=d)
            return d[:64]
        q, s = fp8.block_codes(rows, cols, "cuda"), fp8.block_scales(rows, cols, "cuda")
        fp8.fp8_distill_bwd(z, ids_, lq, stats, w, d_q=q, d_s=s)
        return q[:64]

    assert torch.equal(values(other), values(li))
    assert fp8.fp8_get_status() == 0


# ---------------------------------------------------------------- zeros
@pytest.mark.parametrize("loss", ["logprob", "entropy", "top", "tail"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_without_a_gradient_are_zeros_of_one_sign(loss, dtype):
    """No token, or nothing listed: the codes are the casts of the gradient there too, to the sign of a zero."""
    rows, cols, K = 140, 300, 5
    g = rng("zeros", loss)
    z = normal(g, rows, cols, std=2.0, dtype=dtype)
    none = torch.arange(rows, device="cuda") % 3 == 1
    first, stats, w = torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda"), torch.randn(rows, device="cuda", generator=g)
    if loss in ("logprob", "entropy"):
        tokens = torch.where(none, -1, torch.randint(0, cols, (rows,), device="cuda", generator=g))
        ent = torch.empty(rows, device="cuda") if loss == "entropy" else None
        fp8.fp8_logprob_fwd(z, tokens, first, stats, entropy=ent)
        went = None if ent is None else torch.where(none, 0.0, w)
        call = lambda dt, **out: fp8.fp8_logprob_bwd(z.to(dt), tokens, stats, w, dentropy=went, **out)  # noqa: E731
    else:
        ids = torch.stack([torch.randperm(cols, device="cuda", generator=g)[:K] for _ in range(rows)]).masked_fill(none[:, None], -1)
        li, lq = torch.empty(rows, K, dtype=torch.int32, device="cuda"), torch.empty(rows, K, device="cuda")
        fp8.fp8_distill_fwd(z, ids, normal(g, rows, K) - 3.0, first, stats, li, lq, form=FORM[loss])
        call = lambda dt, **out: fp8.fp8_distill_bwd(z.to(dt), li, lq, stats, w, **out)  # noqa: E731
    d = torch.empty(rows, cols, device="cuda")
    call(F32, dlogits=d)
    assert not d[none].any() and bool((first[none] == 0).all())
    check_gradient_codes(call, rows, cols, dtype, "e5m2")
