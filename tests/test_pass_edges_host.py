"""Norms, log probabilities and distillation at their edges: what is refused on the host."""
import ctypes

from test_passes_host import FAKE, fp8, norm_params  # noqa: F401


def test_a_gate_gradient_of_fewer_than_no_rows_is_refused(fp8):  # noqa: F811
    lib, V = fp8.load_library(), fp8._Vec
    g = fp8._NormGrads()
    g.gate, g.ld_gate, g.gates = V(FAKE, 0), 256, -1
    p = norm_params(fp8, rows=0, gate=V(FAKE, 0))
    args = (None, 256, None, 256, None, 256, None, 256, None, None, 256, None, 256, ctypes.byref(g), None, 0, None)
    assert lib.fp8_norm_bwd(ctypes.byref(p), *args) == fp8.FP8_ERR_INVALID_ARG
