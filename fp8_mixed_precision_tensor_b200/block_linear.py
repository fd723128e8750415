"""Block-scaled FP8 linear layers and a feed-forward block whose forward pass
keeps only 8-bit tensors for the backward pass.

"Training and inference of large language models using 8-bit floating point",
제안 방법 (scale, cast, multiply, undo the scale), with one scale per 128
elements instead of per tensor.  Weights are cast in 128x128 blocks, so one
set of codes serves the forward product and dgrad; activations and output
gradients in 1x128 blocks for the products over features and in 128x1 blocks
for the weight gradient, which reduces over tokens.  What a layer keeps of its
input is the 128x1 codes that its wgrad reads: one byte per element and one
scale byte per 128.

Every number is produced by the library's kernels; this module allocates the
buffers and orders the calls.  With `stream` (a torch.cuda.Stream or its handle)
a pass allocates and works on that stream, its outputs included; the caller
orders it after whatever produced its arguments and the layer's weights.  What
it reads may be dropped while it runs.
"""
from __future__ import annotations

import contextlib

import torch

from . import fp8


def _on(stream, *args: torch.Tensor):
    """The pass's stream as the current one; args, tensors of the caller's, are
    in use on it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    for t in args:
        t.record_stream(stream)
    return torch.cuda.stream(stream)


class _Kept:
    """Tensors that outlive a pass, and the stream that their memory goes back to."""

    def __init__(self, *tensors: torch.Tensor):
        self.tensors, self.stream = tensors, fp8._stream(None)

    def take(self, *beside: torch.Tensor | None) -> tuple[torch.Tensor, ...]:
        """For use on the current stream (with `beside`, kept with them): their
        memory is not reused before that use has ended."""
        if fp8._stream(None) != self.stream:
            now = torch.cuda.current_stream()
            for t in (*self.tensors, *beside):
                if t is not None:
                    t.record_stream(now)
        return self.tensors


class BlockWeight:
    """E4M3 codes of a weight [N, K] in 128x128 blocks, and their scales in the
    order of the forward product (`s`) and of dgrad (`s_col`)."""

    def __init__(self, weight: torch.Tensor, margin: int = 0):
        N, K = weight.shape
        dev = weight.device
        self.margin = margin
        self.q = fp8.block_codes(N, K, dev)
        self.s = fp8.block_scales(N, K, dev)
        self.s_col = fp8.block_scales(K, N, dev)
        self.kept = _Kept(self.q, self.s, self.s_col)
        self.update(weight)

    def update(self, weight: torch.Tensor, stream=None) -> None:
        """Cast the weight anew (after an optimizer step)."""
        with _on(stream, weight):
            self.kept.take()
            fp8.fp8_block_cast_square(weight, fp8.FP8_E4M3, self.margin, self.q, self.s, self.s_col)


class BlockCodes:
    """Row blocks (q, s) and / or column blocks (q_col, s_col) of a [rows, cols]
    tensor of this dtype: what a layer takes in place of the tensor itself where
    the pass before it (BlockNorm) writes them."""

    def __init__(self, shape, dtype: torch.dtype, device, row: bool, col: bool):
        M, K = self.shape = tuple(shape)
        self.dtype, self.device = dtype, device
        new = lambda outer, red: (fp8.block_codes(M, K, device), fp8.block_scales(outer, red, device))  # noqa: E731
        self.q, self.s = new(M, K) if row else (None, None)
        self.q_col, self.s_col = new(K, M) if col else (None, None)

    def record_stream(self, stream) -> None:
        for t in (self.q, self.s, self.q_col, self.s_col):
            if t is not None:
                t.record_stream(stream)


class _Cast(BlockCodes):
    """A tensor cast to such blocks."""

    def __init__(self, x: torch.Tensor, fmt: int, margin: int, row: bool, col: bool):
        super().__init__(x.shape, x.dtype, x.device, row, col)
        fp8.fp8_block_cast(x, fmt, margin, self.q, self.s, self.q_col, self.s_col)


def _operand(x: torch.Tensor | BlockCodes, margin: int, col: bool) -> BlockCodes:
    """x's E4M3 row blocks, and its column blocks where a backward pass needs them."""
    if not isinstance(x, BlockCodes):
        return _Cast(x, fp8.FP8_E4M3, margin, True, col)
    if x.q is None or (col and x.q_col is None):
        raise ValueError("codes of the rows are needed, and of the columns for a backward pass")
    return x


class BlockLinear:
    """y = x W^T (+ bias) with block-scaled FP8 operands.

    forward(x) with x [M, K] (or its BlockCodes) returns y in x's dtype;
    keep=True (training) keeps x's 8-bit column blocks for backward(dy), which returns (dx, dw) (the
    bias's gradient is the sum of dy's rows, the caller's).  Without keep, at
    most FP8_BLOCK_TOKENS_MAX tokens take the one-launch form.

    Not a torch.nn.Module: no parameters, no autograd.  One pass at a time:
    forward(keep=True) takes the place of what an earlier one kept.  With
    several in flight (micro-batches) take `kept` from the layer after each
    forward pass and set it again before the matching backward pass."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None, grad_fmt: int = fp8.FP8_E5M2,
                 margin: int = 0):
        self.N, self.K = weight.shape
        self.weight = BlockWeight(weight, margin)
        self.bias, self.grad_fmt, self.margin = bias, grad_fmt, margin
        self.kept = None

    def forward(self, x: torch.Tensor | BlockCodes, keep: bool = False, stream=None) -> torch.Tensor:
        with _on(stream, x):
            y = torch.empty((x.shape[0], self.N), dtype=x.dtype, device=x.device)
            w = self.weight
            w.kept.take(self.bias)
            if not keep and x.shape[0] <= fp8.FP8_BLOCK_TOKENS_MAX and not isinstance(x, BlockCodes):
                fp8.fp8_block_linear_tokens(x, w.q, w.s, y, bias=self.bias, margin=self.margin)
                return y
            c = _operand(x, self.margin, keep)
            fp8.fp8_block_linear_fwd(c.q, c.s, w.q, w.s, y, bias=self.bias)
            if keep:
                self.kept = _Kept(c.q_col, c.s_col)
            return y

    def backward(self, dy: torch.Tensor, stream=None, rto: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
        """(dx, dw) in dy's dtype (dw bfloat16 rounded to odd with rto, for a
        following FP8 gradient cast).  Uses up what forward kept."""
        if self.kept is None:
            raise RuntimeError("backward needs a forward pass with keep=True")
        with _on(stream, dy):
            M = dy.shape[0]
            self.weight.kept.take()
            g = _Cast(dy, self.grad_fmt, self.margin, True, True)
            dx = torch.empty((M, self.K), dtype=dy.dtype, device=dy.device)
            dw = torch.empty((self.N, self.K), dtype=torch.bfloat16 if rto else dy.dtype, device=dy.device)
            fp8.fp8_block_linear_dgrad(g.q, g.s, self.grad_fmt, self.weight.q, self.weight.s_col, dx)
            fp8.fp8_block_linear_wgrad(g.q_col, g.s_col, self.grad_fmt, *self.kept.take(), dw, rto=rto)
            self.kept = None
            return dx, dw


class BlockMLP:
    """y = act(x W1^T) W2^T, forward and backward, on block-scaled FP8.

    Kept for the backward pass: x's column blocks and the activation's input
    as an E4M3 checkpoint, 1 byte per element each; act(h) is recomputed from
    the checkpoint inside the pass that applies its derivative.  Not a
    torch.nn.Module, and one pass at a time, as BlockLinear; every forward pass
    keeps."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, act: int = fp8.FP8_ACT_GELU_TANH,
                 grad_fmt: int = fp8.FP8_E5M2, margin: int = 0):
        (self.F, self.K), (self.N, F2) = w1.shape, w2.shape
        if F2 != self.F:
            raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} do not chain")
        self.w1, self.w2 = BlockWeight(w1, margin), BlockWeight(w2, margin)
        self.act, self.grad_fmt, self.margin = act, grad_fmt, margin
        self.kept = None

    def forward(self, x: torch.Tensor | BlockCodes, stream=None) -> torch.Tensor:
        with _on(stream, x):
            M, dev = x.shape[0], x.device
            self.w1.kept.take(), self.w2.kept.take()
            c = _operand(x, self.margin, True)
            h = torch.empty((M, self.F), dtype=x.dtype, device=dev)
            fp8.fp8_block_linear_fwd(c.q, c.s, self.w1.q, self.w1.s, h)
            ck, ck_s = fp8.block_codes(M, self.F, dev), fp8.block_scales(M, self.F, dev)
            aq, a_s = fp8.block_codes(M, self.F, dev), fp8.block_scales(M, self.F, dev)
            fp8.fp8_act_fwd(h, self.act, self.margin, ck, ck_s, aq, a_s)
            y = torch.empty((M, self.N), dtype=x.dtype, device=dev)
            fp8.fp8_block_linear_fwd(aq, a_s, self.w2.q, self.w2.s, y)
            self.kept = _Kept(c.q_col, c.s_col, ck, ck_s)
            return y

    def kept_bytes(self) -> int:
        """Bytes that the forward pass keeps for the backward pass."""
        return 0 if self.kept is None else sum(t.untyped_storage().nbytes() for t in self.kept.tensors)

    def backward(self, dy: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(dx, dw1, dw2) in dy's dtype.  Uses up what forward kept."""
        if self.kept is None:
            raise RuntimeError("backward needs a forward pass")
        with _on(stream, dy):
            xq, xs, ck, ck_s = self.kept.take()
            M, dev, fmt = dy.shape[0], dy.device, self.grad_fmt
            self.w1.kept.take(), self.w2.kept.take()
            new = lambda *shape: torch.empty(shape, dtype=dy.dtype, device=dev)  # noqa: E731
            g = _Cast(dy, fmt, self.margin, True, True)
            da = new(M, self.F)
            fp8.fp8_block_linear_dgrad(g.q, g.s, fmt, self.w2.q, self.w2.s_col, da)
            dhq, dhs = fp8.block_codes(M, self.F, dev), fp8.block_scales(M, self.F, dev)
            dhq_c, dhs_c = fp8.block_codes(M, self.F, dev), fp8.block_scales(self.F, M, dev)
            aq_c, as_c = fp8.block_codes(M, self.F, dev), fp8.block_scales(self.F, M, dev)
            fp8.fp8_act_bwd(ck, ck_s, da, self.act, fmt, self.margin, dhq, dhs, dhq_c, dhs_c, aq_c, as_c)
            dw2, dx, dw1 = new(self.N, self.F), new(M, self.K), new(self.F, self.K)
            fp8.fp8_block_linear_wgrad(g.q_col, g.s_col, fmt, aq_c, as_c, dw2)
            fp8.fp8_block_linear_dgrad(dhq, dhs, fmt, self.w1.q, self.w1.s_col, dx)
            fp8.fp8_block_linear_wgrad(dhq_c, dhs_c, fmt, xq, xs, dw1)
            self.kept = None
            return dx, dw1, dw2


class BlockNorm:
    """What stands between two sublayers: r' = res_scale r + gate u with u the
    sublayer's output h or its norm, and x, the norm of r' for the next sublayer.

    forward(h, r) returns (r', x); with codes=True x is its BlockCodes, written
    by the norm itself, for BlockLinear, BlockMLP or BlockHead (with keep=True
    the column blocks of their weight gradient too).  h may be None (a norm
    alone); dtype then gives x's, r's own by default (a model of 16-bit layers
    with a float32 residual starts so).  keep=True keeps h, r' and each row's statistics for
    backward(dx, dr), which returns (dh, dr, grads): dr is the gradient of r' from
    what follows, or None, and grads has the gradient of each parameter given, in
    its dtype, by name.

    Not a torch.nn.Module, and one pass at a time, as BlockLinear."""

    def __init__(self, w: torch.Tensor | None, b: torch.Tensor | None = None, pre: int = fp8.FP8_NORM_RMS,
                 post: int = fp8.FP8_NORM_NONE, post_w: torch.Tensor | None = None, post_b: torch.Tensor | None = None,
                 gate: torch.Tensor | None = None, res_scale: float = 1.0, eps: float = 1e-5, margin: int = 0):
        if pre == fp8.FP8_NORM_NONE:
            raise ValueError("pre: the norm that gives x is needed")
        if post == fp8.FP8_NORM_NONE and (post_w is not None or post_b is not None):
            raise ValueError("post_w and post_b belong to a post norm: post is FP8_NORM_NONE")
        self.params = {"w": w, "b": b, "post_w": post_w, "post_b": post_b, "gate": gate}
        self.pre, self.post, self.res_scale, self.eps, self.margin = pre, post, float(res_scale), float(eps), margin
        self.kept = None

    def _in_use(self) -> None:
        """The parameters on the pass's stream."""
        now = torch.cuda.current_stream()
        for t in self.params.values():
            if t is not None:
                t.record_stream(now)

    def forward(self, h: torch.Tensor | None, r: torch.Tensor, codes: bool = False, keep: bool = False, stream=None,
                dtype: torch.dtype | None = None) -> tuple[torch.Tensor, torch.Tensor | BlockCodes]:
        of = r if h is None else h
        if dtype is None:
            dtype = of.dtype
        elif dtype != of.dtype and not (h is None and r.dtype is torch.float32 and dtype in (torch.bfloat16, torch.float16)):
            raise ValueError(f"dtype {dtype}: x has h's, or beside a float32 residual without h a 16-bit one")
        with _on(stream, *(t for t in (h, r) if t is not None)):
            if stream is not None:
                self._in_use()
            M, D = r.shape
            r_out = torch.empty_like(r, memory_format=torch.contiguous_format)
            stats = torch.empty((M, 4), dtype=torch.float32, device=r.device) if keep else None
            out = {}
            if codes:
                x = BlockCodes((M, D), dtype, r.device, True, keep)
                out = {"x_q": x.q, "x_s": x.s, "x_q_col": x.q_col, "x_s_col": x.s_col}
            else:
                x = out["x"] = torch.empty((M, D), dtype=dtype, device=r.device)
            fp8.fp8_norm_fwd(h, r, r_out, stats, pre=self.pre, post=self.post, res_scale=self.res_scale, eps=self.eps,
                             margin=self.margin, **self.params, **out)
            if keep:
                self.kept = (h is not None, _Kept(*((h,) if h is not None else ()), r_out, stats))
            return r_out, x

    def backward(self, dx: torch.Tensor, dr: torch.Tensor | None = None,
                 stream=None) -> tuple[torch.Tensor | None, torch.Tensor, dict[str, torch.Tensor]]:
        if self.kept is None:
            raise RuntimeError("backward needs a forward pass with keep=True")
        with _on(stream, *(t for t in (dx, dr) if t is not None)):
            if stream is not None:
                self._in_use()
            had, kept = self.kept
            *h, r_out, stats = kept.take()
            M, D = r_out.shape
            gate = self.params["gate"]
            need = fp8.fp8_norm_workspace_bytes(M, D, M // gate.shape[0] if gate is not None and gate.dim() == 2 and M else M)
            work = torch.empty(need, dtype=torch.uint8, device=dx.device) if need else None
            new = lambda like: torch.empty(like.shape, dtype=like.dtype, device=dx.device)  # noqa: E731
            dh, dr_in = new(h[0]) if had else None, new(r_out)
            grads = {k: new(t) for k, t in self.params.items() if t is not None}
            given = {k: t for k, t in self.params.items() if k != "b"}
            fp8.fp8_norm_bwd(dx, dr, h[0] if had else None, r_out, stats, pre=self.pre, post=self.post,
                             res_scale=self.res_scale, **given, dh=dh, dr=dr_in, workspace=work,
                             **{"d" + k: t for k, t in grads.items()})
            self.kept = None
            return dh, dr_in, grads


class BlockHead:
    """The last linear layer, logits = x W^T with W [V, K], and what is computed
    from its logits: log probabilities of tokens, or the divergence from a
    teacher's top logits.  The gradient of the logits is only ever written as the
    8-bit codes that the layer's own dgrad and wgrad read.

    log_probs(x, tokens) and distill(x, ids, values) take x [M, K] or its
    BlockCodes.  The logits are stored in x's dtype, and what is computed from them
    carries that rounding (half a step of bfloat16 at a logit of 20 is 0.06),
    unless logits_dtype asks for another (float32).  keep=True keeps the logits and x's column blocks for backward(g),
    g the gradient of what was returned for each row, which returns (dx, dw) in
    x's dtype.

    Not a torch.nn.Module, and one pass at a time, as BlockLinear."""

    def __init__(self, weight: torch.Tensor, grad_fmt: int = fp8.FP8_E5M2, margin: int = 0,
                 logits_dtype: torch.dtype | None = None):
        self.N, self.K = weight.shape
        self.weight = BlockWeight(weight, margin)
        self.grad_fmt, self.margin, self.logits_dtype = grad_fmt, margin, logits_dtype
        self.kept = None

    def _logits(self, x: torch.Tensor | BlockCodes, keep: bool) -> tuple[torch.Tensor, tuple]:
        w = self.weight
        w.kept.take()
        logits = torch.empty((x.shape[0], self.N), dtype=self.logits_dtype or x.dtype, device=x.device)
        if not keep and x.shape[0] <= fp8.FP8_BLOCK_TOKENS_MAX and not isinstance(x, BlockCodes):
            fp8.fp8_block_linear_tokens(x, w.q, w.s, logits, margin=self.margin)
            return logits, ()
        c = _operand(x, self.margin, keep)
        fp8.fp8_block_linear_fwd(c.q, c.s, w.q, w.s, logits)
        return logits, (c.q_col, c.s_col)

    def log_probs(self, x: torch.Tensor | BlockCodes, tokens: torch.Tensor, inv_temp: float = 1.0, entropy: bool = False,
                  top: int = 0, keep: bool = False, stream=None) -> dict[str, torch.Tensor]:
        """{"logp": [M]} and, where asked for, "entropy" [M], "top_logp" and "top_ids" [M, top]."""
        with _on(stream, x, tokens):
            logits, cols = self._logits(x, keep)
            M, dev = logits.shape[0], logits.device
            f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)  # noqa: E731
            out = {"logp": f32(M)}
            if entropy:
                out["entropy"] = f32(M)
            if top:
                out |= {"top_logp": f32(M, top), "top_ids": torch.empty((M, top), dtype=torch.int32, device=dev)}
            stats = f32(M, 4) if keep else None
            more = {k: v for k, v in out.items() if k != "logp"}
            fp8.fp8_logprob_fwd(logits, tokens, out["logp"], stats, inv_temp=float(inv_temp), **more)
            if keep:
                self.kept = ("entropy" if entropy else "logp", x.dtype, float(inv_temp), _Kept(*cols, logits, stats, tokens))
            return out

    def distill(self, x: torch.Tensor | BlockCodes, ids: torch.Tensor, values: torch.Tensor,
                form: int = fp8.FP8_DISTILL_TOP, inv_temp: float = 1.0, keep: bool = False, stream=None) -> torch.Tensor:
        """The divergence of each row, [M]."""
        with _on(stream, x, ids, values):
            logits, cols = self._logits(x, keep)
            M, dev = logits.shape[0], logits.device
            f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)  # noqa: E731
            loss, stats, list_q = f32(M), f32(M, 4), f32(*ids.shape)
            list_ids = torch.empty(ids.shape, dtype=torch.int32, device=dev)
            fp8.fp8_distill_fwd(logits, ids, values, loss, stats, list_ids, list_q, form=form, inv_temp=float(inv_temp))
            if keep:
                self.kept = ("distill", x.dtype, float(inv_temp), _Kept(*cols, logits, stats, list_ids, list_q))
            return loss

    def backward(self, g: torch.Tensor, dentropy: torch.Tensor | None = None,
                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """(dx, dw).  dentropy: the gradient of the entropies, which log_probs then computed.  Uses up what was kept."""
        if self.kept is None:
            raise RuntimeError("backward needs log_probs or distill with keep=True")
        kind, dtype, inv_temp, kept = self.kept
        if dentropy is not None and kind != "entropy":
            raise ValueError("dentropy needs log_probs with entropy=True")
        with _on(stream, *(t for t in (g, dentropy) if t is not None)):
            xq, xs, logits, stats, *rest = kept.take()
            w, fmt = self.weight, self.grad_fmt
            w.kept.take()
            d = BlockCodes(logits.shape, logits.dtype, logits.device, True, True)
            out = dict(inv_temp=inv_temp, fmt=fmt, margin=self.margin, d_q=d.q, d_s=d.s, d_q_col=d.q_col, d_s_col=d.s_col)
            if kind != "distill":
                fp8.fp8_logprob_bwd(logits, rest[0], stats, g, dentropy=dentropy, **out)
            else:
                fp8.fp8_distill_bwd(logits, *rest, stats, g, **out)
            dx = torch.empty((logits.shape[0], self.K), dtype=dtype, device=logits.device)
            dw = torch.empty((self.N, self.K), dtype=dtype, device=logits.device)
            fp8.fp8_block_linear_dgrad(d.q, d.s, fmt, w.q, w.s_col, dx)
            fp8.fp8_block_linear_wgrad(d.q_col, d.s_col, fmt, xq, xs, dw)
            self.kept = None
            return dx, dw
