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


class _Cast:
    """Row and / or column blocks of a tensor."""

    def __init__(self, x: torch.Tensor, fmt: int, margin: int, row: bool, col: bool):
        M, K = x.shape
        new = lambda outer, red: (fp8.block_codes(M, K, x.device), fp8.block_scales(outer, red, x.device))  # noqa: E731
        self.q, self.s = new(M, K) if row else (None, None)
        self.q_col, self.s_col = new(K, M) if col else (None, None)
        fp8.fp8_block_cast(x, fmt, margin, self.q, self.s, self.q_col, self.s_col)


class BlockLinear:
    """y = x W^T (+ bias) with block-scaled FP8 operands.

    forward(x) with x [M, K] returns y in x's dtype; keep=True (training) keeps
    x's 8-bit column blocks for backward(dy), which returns (dx, dw) (the
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

    def forward(self, x: torch.Tensor, keep: bool = False, stream=None) -> torch.Tensor:
        with _on(stream, x):
            y = torch.empty((x.shape[0], self.N), dtype=x.dtype, device=x.device)
            w = self.weight
            w.kept.take(self.bias)
            if not keep and x.shape[0] <= fp8.FP8_BLOCK_TOKENS_MAX:
                fp8.fp8_block_linear_tokens(x, w.q, w.s, y, bias=self.bias, margin=self.margin)
                return y
            c = _Cast(x, fp8.FP8_E4M3, self.margin, True, keep)
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

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        with _on(stream, x):
            M, dev = x.shape[0], x.device
            self.w1.kept.take(), self.w2.kept.take()
            c = _Cast(x, fp8.FP8_E4M3, self.margin, True, True)
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
