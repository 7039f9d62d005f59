"""Outputs in the place of inputs that other rows or tiles still read are refused, before any HIP call."""
import pytest

pytest.importorskip("torch")

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402
from test_head_cpu import ARG, LINEAR, LINEAR_BWD, NORM, NORM_BWD, RULES, P, _call  # noqa: E402

Q = 16 * P   # another place


@pytest.mark.parametrize("fn,defaults,over,needle", [
    ("lce_rms_norm", NORM, dict(), "y must not be weight"),
    ("lce_rms_norm", NORM, dict(weight=Q, sum=Q, lds=64), "sum must not be weight"),
    ("lce_rms_norm", NORM, dict(weight=Q, weight_dtype=lce.LCE_F32, rstd=Q), "rstd must not be weight"),
    ("lce_rms_norm", NORM, dict(weight=Q, y_dtype=lce.LCE_E4M3, scale=Q), "scale must not be weight"),
    ("lce_rms_norm_backward", NORM_BWD, dict(), "grad_x must not be weight"),
    ("lce_logits_process", RULES, dict(bias_ids=Q, bias_values=P, B=100, ldbi=100, ldbv=100), "out must not be bias_values"),
    ("lce_logits_process", RULES, dict(repetition=P), "out must not be repetition"),
    ("lce_logits_process", RULES, dict(presence=P), "out must not be presence"),
    ("lce_logits_process", RULES, dict(frequency=P), "out must not be frequency"),
    ("lce_logits_process", RULES, dict(temperature=P), "out must not be temperature"),
    ("lce_linear", LINEAR, dict(out=Q, bias=Q), "out must not be bias"),
    ("lce_linear", LINEAR, dict(out=2 * Q, preact=Q, ldp=40, bias=Q, bias_dtype=lce.LCE_BF16), "preact must not be bias"),
    ("lce_linear_backward", LINEAR_BWD, dict(grad_out=Q, grad_bias=Q), "grad_bias must not be grad_out"),
    ("lce_linear_backward", LINEAR_BWD, dict(preact=Q, grad_bias=Q), "grad_bias must not be preact"),
    ("lce_linear_backward", LINEAR_BWD, dict(x=Q, grad_bias=Q), "grad_bias must not be x"),
    ("lce_linear_backward", LINEAR_BWD, dict(weight=Q, grad_bias=Q), "grad_bias must not be weight"),
])
def test_refused(fn, defaults, over, needle):
    st, msg = _call(fn, defaults, over)
    assert st == ARG and needle in msg
