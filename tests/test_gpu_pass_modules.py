"""BlockNorm and BlockHead, a run of the passes together, and how the calls behave around the kernels: streams,
captured graphs, calls side by side, the way through Python."""
import threading

import pytest
import torch

from fp8_mixed_precision_tensor_b200 import fp8
from fp8_mixed_precision_tensor_b200.block_linear import BlockCodes, BlockHead, BlockLinear, BlockMLP, BlockNorm
from _passes import Norm64, Rows64
from test_gpu_passes import BF16, F16, F32, normal, rng

pytestmark = pytest.mark.gpu

RMS, LAYER, NONE = fp8.FP8_NORM_RMS, fp8.FP8_NORM_LAYER, fp8.FP8_NORM_NONE


def parts(M=200, D=256, F=512, V=640, dtype=BF16, seed=1):
    g = rng("model", M, D, V, seed)
    r = normal(g, M, D, std=1.0, dtype=F32)
    vec = lambda mean, std: (mean + torch.randn(D, device="cuda", generator=g) * std).to(dtype)  # noqa: E731
    first = BlockNorm(vec(1, 0.1), pre=RMS)
    mlp = BlockMLP(normal(g, F, D, std=0.05, dtype=dtype), normal(g, D, F, std=0.05, dtype=dtype))
    last = BlockNorm(vec(1, 0.1), vec(0, 0.1), pre=LAYER, post=RMS, post_w=vec(1, 0.1), gate=vec(0.5, 0.1), res_scale=0.9)
    head = BlockHead(normal(g, V, D, std=0.1, dtype=dtype))
    tokens = torch.randint(0, V, (M,), device="cuda", generator=g)
    tokens[3] = -1
    return r, first, mlp, last, head, tokens, g


def step(r, first, mlp, last, head, tokens, dtype=BF16, stream=None):
    """A training step of a residual block and the loss: every output and gradient."""
    M = r.shape[0]
    r1, x1 = first.forward(None, r.to(dtype), codes=True, keep=True, stream=stream)
    h = mlp.forward(x1, stream=stream)
    r2, x2 = last.forward(h, r1, codes=True, keep=True, stream=stream)
    out = head.log_probs(x2, tokens, entropy=True, keep=True, stream=stream)
    g = torch.full((M,), -1.0 / M, device="cuda")
    dx2, dw = head.backward(g, torch.full((M,), 0.01 / M, device="cuda"), stream=stream)
    dh, dr1, grads2 = last.backward(dx2, stream=stream)
    dx1, dw1, dw2 = mlp.backward(dh, stream=stream)
    none, dr, grads1 = first.backward(dx1, dr1, stream=stream)
    assert none is None
    return [out["logp"], out["entropy"], dx2, dw, dh, dr1, dx1, dw1, dw2, dr, r2, *grads1.values(), *grads2.values()]


def test_a_step_is_the_sequence_of_its_calls():
    r, first, mlp, last, head, tokens, _ = parts()
    got = step(r, first, mlp, last, head, tokens)
    M, D, V, F = 200, 256, 640, 512
    C, S = fp8.block_codes, fp8.block_scales
    e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    x, st1, st2, st3 = r.to(BF16), e(M, 4, dt=F32), e(M, 4, dt=F32), e(M, 4, dt=F32)
    r1 = e(M, D)
    xq, xs, xqc, xsc = C(M, D), S(M, D), C(M, D), S(D, M)
    w = first.params["w"]
    fp8.fp8_norm_fwd(None, x, r1, st1, w=w, x_q=xq, x_s=xs, x_q_col=xqc, x_s_col=xsc)
    h1, h = e(M, F), e(M, D)
    fp8.fp8_block_linear_fwd(xq, xs, mlp.w1.q, mlp.w1.s, h1)
    ck, cks, aq, a_s = C(M, F), S(M, F), C(M, F), S(M, F)
    fp8.fp8_act_fwd(h1, mlp.act, 0, ck, cks, aq, a_s)
    fp8.fp8_block_linear_fwd(aq, a_s, mlp.w2.q, mlp.w2.s, h)
    p = last.params
    r2 = e(M, D)
    yq, ys, yqc, ysc = C(M, D), S(M, D), C(M, D), S(D, M)
    kinds = dict(pre=LAYER, post=RMS, res_scale=0.9)
    fp8.fp8_norm_fwd(h, r1, r2, st2, **kinds, **p, x_q=yq, x_s=ys, x_q_col=yqc, x_s_col=ysc)
    z = e(M, V)
    fp8.fp8_block_linear_fwd(yq, ys, head.weight.q, head.weight.s, z)
    logp, ent = e(M, dt=F32), e(M, dt=F32)
    fp8.fp8_logprob_fwd(z, tokens, logp, st3, entropy=ent)
    dq, ds, dqc, dsc = C(M, V), S(M, V), C(M, V), S(V, M)
    g, ge = torch.full((M,), -1.0 / M, device="cuda"), torch.full((M,), 0.01 / M, device="cuda")
    fp8.fp8_logprob_bwd(z, tokens, st3, g, dentropy=ge, d_q=dq, d_s=ds, d_q_col=dqc, d_s_col=dsc)
    dx2, dw = e(M, D), e(V, D)
    fp8.fp8_block_linear_dgrad(dq, ds, fp8.FP8_E5M2, head.weight.q, head.weight.s_col, dx2)
    fp8.fp8_block_linear_wgrad(dqc, dsc, fp8.FP8_E5M2, yqc, ysc, dw)
    dh, dr1 = e(M, D), e(M, D)
    q = {k: v for k, v in p.items() if k != "b"}
    fp8.fp8_norm_bwd(dx2, None, h, r2, st2, **kinds, **q, dh=dh, dr=dr1)
    for a, b in zip(got, (logp, ent, dx2, dw, dh, dr1)):
        assert torch.equal(a, b)
    assert torch.equal(got[10], r2) and fp8.fp8_get_status() == 0
    # and in binary64 from what the step stored: the loss, and the last norm's gradients
    ref = Rows64(z, 1.0, 32)
    lp = ref.lp.gather(1, tokens.clamp_min(0)[:, None])[:, 0]
    assert bool((torch.where(tokens >= 0, lp, 0.0) - logp).abs().max() < 1e-5)
    n = Norm64(h, r1, r2, "layer", "rms", p["w"], p["b"], p["post_w"], None, p["gate"], 0.9)
    for k, (v, m) in n.backward(dx2, None).items():
        if k in ("dh", "dr"):
            t = {"dh": dh, "dr": dr1}[k]
            assert bool(((t.double() - v).abs() <= 2.0 ** -8 * v.abs() + 128 * 2.0 ** -24 * m).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_head_gradients_are_those_of_the_loss(dtype):
    """dx and dw against binary64 on the layer's own logits: an operand's rounding to E5M2 is off by 2^-3 of it (and
    of its block's smallest step, 2^-16 of the block's largest), to E4M3 by 2^-4 (2^-10 of the block's largest)."""
    M, K, V = 150, 200, 700
    g = rng("head", str(dtype))
    x, w = normal(g, M, K, dtype=dtype), normal(g, V, K, std=0.1, dtype=dtype)
    tokens = torch.randint(0, V, (M,), device="cuda", generator=g)
    values, ids = torch.randn(M, 8, device="cuda", generator=g), torch.randint(0, V // 8, (M, 8), device="cuda", generator=g)
    ids = ids + torch.arange(8, device="cuda") * (V // 8)
    for loss in ("logp", "distill"):
        head = BlockHead(w, logits_dtype=F32)
        if loss == "logp":
            head.log_probs(x, tokens, keep=True)
        else:
            head.distill(x, ids, values, keep=True)
        z = next(t for t in head.kept[3].tensors if t.shape == (M, V) and t.dtype is F32)
        ref = Rows64(z, 1.0, 32)
        gl = torch.randn(M, device="cuda", generator=g).to(F32) * (64 if dtype is F16 else 1)
        dx, dw = head.backward(gl)
        if loss == "logp":
            d = torch.zeros_like(ref.p).scatter_(1, tokens[:, None], 1.0) - ref.p
        else:
            d = ref.p - torch.zeros_like(ref.p).scatter_(1, ids, torch.softmax(values.double(), 1))
        d = d * gl.double()[:, None]
        xv, wv = x.double(), w.double()
        pad = lambda t, dim: torch.nn.functional.pad(t, (0, -t.shape[1] % 128) if dim else (0, 0, 0, -t.shape[0] % 128))  # noqa: E731

        def peak(t, dim):  # the largest of each element's block
            u = pad(t.abs(), dim)
            u = u.view(u.shape[0], -1, 128).amax(2).repeat_interleave(128, 1) if dim else u.view(-1, 128, u.shape[1]).amax(1).repeat_interleave(128, 0)
            return u[:t.shape[0], :t.shape[1]]

        def off(t, dim, half, least):
            return half * t.abs() + least * peak(t, dim)

        d_r, d_c = off(d, 1, 2.0 ** -3, 2.0 ** -16), off(d, 0, 2.0 ** -3, 2.0 ** -16)
        w_o, x_o = 2.0 ** -4 * wv.abs() + 2.0 ** -10 * wv.abs().max(), off(xv, 0, 2.0 ** -4, 2.0 ** -10)
        want, tol = d @ wv, (d.abs() + d_r) @ (wv.abs() + w_o) - d.abs() @ wv.abs()
        assert bool(((dx.double() - want).abs() <= tol * 1.01 + 2.0 ** -8 * want.abs() + 1e-6).all())
        want, tol = d.T @ xv, (d.abs() + d_c).T @ (xv.abs() + x_o) - d.abs().T @ xv.abs()
        assert bool(((dw.double() - want).abs() <= tol * 1.01 + 2.0 ** -8 * want.abs() + 1e-6).all())


def test_few_tokens_and_what_is_shown_beside_them():
    g = rng("decode")
    w, x = normal(g, 1000, 128, std=0.1, dtype=BF16), normal(g, 4, 128, dtype=BF16)
    head = BlockHead(w)
    out = head.log_probs(x, torch.tensor([1, 2, 3, -1], device="cuda"), entropy=True, top=5)
    z = torch.empty(4, 1000, dtype=BF16, device="cuda")
    fp8.fp8_block_linear_tokens(x, head.weight.q, head.weight.s, z)
    lp = torch.log_softmax(z.double(), 1)
    assert torch.allclose(out["logp"][:3].double(), lp[torch.arange(3), torch.arange(1, 4)], atol=1e-5) and out["logp"][3] == 0
    assert torch.equal(out["top_ids"].long(), torch.sort(z, dim=1, descending=True, stable=True)[1][:, :5])
    assert torch.allclose(out["entropy"].double(), torch.special.entr(lp.exp()).sum(1), atol=1e-5)
    assert head.kept is None


def test_modules_refuse_what_was_not_kept():
    r, first, mlp, last, head, tokens, _ = parts(M=8)
    for call in (lambda: first.backward(r), lambda: head.backward(r[:, 0])):
        with pytest.raises(RuntimeError):
            call()
    _, x = first.forward(None, r.to(BF16), codes=True)  # row blocks only
    with pytest.raises(ValueError):
        head.log_probs(x, tokens, keep=True)
    head.log_probs(r.to(BF16), tokens, keep=True)
    with pytest.raises(ValueError):
        head.backward(r[:, 0].contiguous(), dentropy=r[:, 0].contiguous())


def test_codes_serve_a_linear_layer():
    g = rng("codes")
    h, r, w = normal(g, 70, 384, dtype=BF16), normal(g, 70, 384, dtype=BF16), normal(g, 256, 384, std=0.05, dtype=BF16)
    norm, lin = BlockNorm(torch.ones(384, device="cuda")), BlockLinear(w)
    _, x = norm.forward(h, r, codes=True, keep=True)
    assert isinstance(x, BlockCodes) and x.shape == (70, 384)
    y = lin.forward(x, keep=True)
    want = torch.empty_like(y)
    fp8.fp8_block_linear_fwd(x.q, x.s, lin.weight.q, lin.weight.s, want)
    assert torch.equal(y, want)
    dx, dw = lin.backward(torch.ones_like(y))
    assert dx.shape == (70, 384) and bool(dw.isfinite().all())


def test_a_step_on_another_stream():
    r, first, mlp, last, head, tokens, _ = parts()
    want = step(r, first, mlp, last, head, tokens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r2 = r + 0.0
    s.wait_stream(torch.cuda.current_stream())
    got = step(r2, first, mlp, last, head, tokens, stream=s)
    del r2
    junk = [torch.full((200, 256), 9.0, device="cuda") for _ in range(20)]  # memory that was dropped, taken again
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and junk


def test_a_captured_step_replays_on_new_inputs():
    r, first, mlp, last, head, tokens, g = parts()
    x = r.clone()
    step(x, first, mlp, last, head, tokens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step(x, first, mlp, last, head, tokens)
        with torch.cuda.graph(graph, stream=s):
            got = step(x, first, mlp, last, head, tokens)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        x.copy_(normal(g, 200, 256))
        tokens.copy_(torch.randint(0, 640, (200,), device="cuda", generator=g))
        graph.replay()
        now = [t.clone() for t in got]
        want = step(x, first, mlp, last, head, tokens)
        assert all(torch.equal(a, b) for a, b in zip(now, want))


def test_calls_side_by_side_on_two_streams_and_threads():
    """Each call with buffers of its own; the same bits as one after another."""
    inputs = []
    for seed in (1, 2):
        g = rng("two", seed)
        z = normal(g, 400, 9000, std=2.0, dtype=BF16)
        inputs.append((z, torch.randint(0, 9000, (400,), device="cuda", generator=g), normal(g, 400, 2048, dtype=BF16)))

    def work(z, t, h, stream=None):
        e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        lp, st, ids, tl = e(400), e(400, 4), e(400, 9, dt=torch.int32), e(400, 9)
        r_out, x, nst, w = torch.empty_like(h), torch.empty_like(h), e(400, 4), torch.ones(2048, device="cuda")
        dw, dh = e(2048), torch.empty_like(h)
        ws = torch.empty(fp8.fp8_norm_workspace_bytes(400, 2048), dtype=torch.uint8, device="cuda")
        d = torch.empty_like(z)
        torch.cuda.current_stream().synchronize()
        for _ in range(5):
            fp8.fp8_logprob_fwd(z, t, lp, st, top_logp=tl, top_ids=ids, stream=stream)
            fp8.fp8_logprob_bwd(z, t, st, lp, dlogits=d, stream=stream)
            fp8.fp8_norm_fwd(h, h, r_out, nst, w=w, x=x, stream=stream)
            fp8.fp8_norm_bwd(x, None, h, r_out, nst, w=w, dh=dh, dw=dw, workspace=ws, stream=stream)
        return lp, ids, tl, d, x, dw, dh

    want = [work(*i) for i in inputs]
    torch.cuda.synchronize()
    got = [None, None]

    def run(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[k] = work(*inputs[k], stream=torch.cuda.current_stream())

    threads = [threading.Thread(target=run, args=(k,)) for k in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_way_through_python_gives_the_same(monkeypatch):
    r, first, mlp, last, head, tokens, _ = parts(M=40)
    want = step(r, first, mlp, last, head, tokens)
    monkeypatch.setattr(fp8, "_calls", fp8._PythonRoute())
    got = step(r, first, mlp, last, head, tokens)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ids, values = torch.randint(0, 80, (40, 8), device="cuda") * 8 + torch.arange(8, device="cuda"), torch.randn(40, 8, device="cuda")
    loss = head.distill(r.to(BF16), ids, values, keep=True)
    dx, dw = head.backward(loss)
    monkeypatch.undo()
    loss2 = head.distill(r.to(BF16), ids, values, keep=True)
    dx2, dw2 = head.backward(loss2)
    assert torch.equal(loss, loss2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_wrong_shapes_and_types_are_named():
    x, s = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 4, device="cuda")
    with pytest.raises(ValueError, match="stats"):
        fp8.fp8_norm_fwd(x, x, x.clone(), s[:3], w=x[0], x=x.clone())
    with pytest.raises(TypeError, match="h: dtype"):
        fp8.fp8_norm_bwd(x, x, x.half(), x, s, dh=x.clone())
    with pytest.raises(ValueError, match="gate: 3 rows for 4"):
        fp8.fp8_norm_fwd(x, x, x.clone(), s, gate=torch.zeros(3, 64, device="cuda"))
    with pytest.raises(ValueError, match="dgate has gate's shape"):
        fp8.fp8_norm_bwd(x, x, x, x, s, gate=torch.zeros(2, 64, device="cuda"), dgate=torch.zeros(64, device="cuda"))
    with pytest.raises(TypeError, match="tokens: dtype"):
        fp8.fp8_logprob_fwd(x, torch.zeros(4, device="cuda"), s[:, 0].contiguous(), s)
    with pytest.raises(ValueError, match="logp"):
        fp8.fp8_logprob_fwd(x, torch.zeros(4, dtype=torch.int64, device="cuda"), s[:, 0], s)  # strided
    with pytest.raises(ValueError, match="list_ids"):
        fp8.fp8_distill_bwd(x, torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda"), s,
                            torch.zeros(4, device="cuda"), dlogits=x.clone())
    with pytest.raises(fp8.FP8Error):
        fp8.fp8_norm_bwd(x, x, x, x, s, w=x[0], dh=x.clone(), dw=torch.zeros(64, device="cuda"))  # no workspace
    with pytest.raises(fp8.FP8Error):
        fp8.fp8_logprob_bwd(x, None, s, None, dlogits=x.clone())
