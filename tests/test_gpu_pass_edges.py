"""Norms, log probabilities and distillation at their edges."""
import ctypes
import threading

import pytest
import torch

from fp8_mixed_precision_tensor_b200 import fp8
from fp8_mixed_precision_tensor_b200.block_linear import BlockNorm
from test_gpu_passes import BF16, F16, F32, FORM, GUARD, KIND, Strided, normal, rng, run_distill


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
