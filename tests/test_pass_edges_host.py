"""Norms, log probabilities and distillation at their edges: what is refused on the host."""
import ctypes

import pytest
import torch

from test_passes_host import FAKE, fp8, norm_params  # noqa: F401


def test_a_gate_gradient_of_fewer_than_no_rows_is_refused(fp8):  # noqa: F811
    lib, V = fp8.load_library(), fp8._Vec
    g = fp8._NormGrads()
    g.gate, g.ld_gate, g.gates = V(FAKE, 0), 256, -1
    p = norm_params(fp8, rows=0, gate=V(FAKE, 0))
    args = (None, 256, None, 256, None, 256, None, 256, None, None, 256, None, 256, ctypes.byref(g), None, 0, None)
    assert lib.fp8_norm_bwd(ctypes.byref(p), *args) == fp8.FP8_ERR_INVALID_ARG


def test_a_norm_layer_refuses_parameters_of_a_norm_that_it_lacks(fp8):  # noqa: F811
    """Its forward pass would leave them out and its backward pass, asked for their gradients, fail."""
    from fp8_mixed_precision_tensor_b200.block_linear import BlockNorm

    w = torch.ones(8)
    for kw in (dict(post_w=w), dict(post_b=w), dict(post_w=w, post=fp8.FP8_NORM_NONE)):
        with pytest.raises(ValueError, match="post norm"):
            BlockNorm(w, **kw)
    with pytest.raises(ValueError, match="pre"):
        BlockNorm(w, pre=fp8.FP8_NORM_NONE)
    BlockNorm(w, post=fp8.FP8_NORM_RMS, post_w=w)


@pytest.mark.parametrize("inv_temp", [2.3591e38, 3.4e38])
def test_a_temperature_whose_exponents_overflow_is_refused(fp8, inv_temp):  # noqa: F811
    """inv_temp / log 2, the factor of every exponent, is beyond binary32 from 2^128 log 2 = 2.3587e38 on."""
    lib, bad = fp8.load_library(), fp8.FP8_ERR_INVALID_ARG
    z = (FAKE, fp8.FP8_DT_F32, 4, 256, 256, inv_temp)
    assert lib.fp8_logprob_fwd(*z, FAKE, 8, FAKE, None, 0, None, None, FAKE, None) == bad
    assert lib.fp8_logprob_bwd(*z, FAKE, 8, FAKE, FAKE, None, 1, 0, None, None, FAKE, 256, None) == bad
    assert lib.fp8_distill_fwd(*z, 0, 8, FAKE, 4, FAKE, 0, FAKE, FAKE, FAKE, FAKE, None) == bad
    assert lib.fp8_distill_bwd(*z, 8, FAKE, FAKE, FAKE, FAKE, 1, 0, None, None, FAKE, 256, None) == bad
    empty = (FAKE, fp8.FP8_DT_F32, 0, 256, 256, 2.3e38)
    assert lib.fp8_distill_bwd(*empty, 8, FAKE, FAKE, FAKE, FAKE, 1, 0, None, None, FAKE, 256, None) == fp8.FP8_OK
