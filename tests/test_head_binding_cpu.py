"""Operands of the norm, the product and the rules by name, the first one too."""
import inspect

import pytest

torch = pytest.importorskip("torch")

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

X, W = torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((16, 16), dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: lce.lce_rms_norm(x=X, weight=W[0]),
    lambda: lce.lce_rms_norm_backward(grad_y=X, s=X, weight=W[0], rstd=torch.zeros(4)),
    lambda: lce.lce_linear(x=X, weight=W), lambda: lce.lce_linear(weight=W, x=X),
    lambda: lce.lce_linear_backward(grad_out=X, x=X, weight=W),
    lambda: lce.lce_logits_process(logits=X),
])
def test_first_operand_by_name(call):
    with pytest.raises(ValueError, match="GPU tensor"):   # as for host tensors given in order
        call()


@pytest.mark.parametrize("call", [lambda: lce.lce_linear(weight=W), lambda: lce.lce_rms_norm(),
                                  lambda: lce.lce_logits_process(softcap=1.0)])
def test_a_missing_first_operand_is_named(call):
    with pytest.raises(TypeError, match="'(x|logits)'"):
        call()


def test_signatures_name_the_operands():
    assert list(inspect.signature(lce.lce_linear).parameters)[:2] == ["x", "weight"]
