"""Norms, log probabilities and distillation at their edges."""
import pytest
import torch

from fp8_mixed_precision_tensor_b200 import fp8
from fp8_mixed_precision_tensor_b200.block_linear import BlockNorm
from test_gpu_passes import BF16, F16, F32, GUARD, KIND, Strided, normal, rng, run_distill


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
