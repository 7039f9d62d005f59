"""What the autograd product hands to the library, on the CPU: the library is replaced by a recorder
and nothing is launched, so the operands may be host tensors."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402
from vocabulary_cross_entropy_row_amd import head  # noqa: E402

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
PREACT = 18   # positions among lce_linear's arguments


class _Recorder:
    def __init__(self):
        self.calls = []

    def lce_linear_workspace_bytes(self, *a):
        return 0

    def lce_linear_backward_workspace_bytes(self, *a):
        return 256

    def lce_linear(self, *a):
        self.calls.append(("forward", a))
        return lce.LCE_OK

    def lce_linear_backward(self, *a):
        self.calls.append(("backward", a))
        return lce.LCE_OK


@pytest.fixture
def calls(monkeypatch):
    recorder = _Recorder()
    monkeypatch.setattr(head, "lib", lambda: recorder)
    monkeypatch.setattr(head, "_on_gpu", lambda t, name: t.device)
    monkeypatch.setattr(head, "_current_stream", lambda index: 0)
    return recorder.calls


def test_gradients_reach_the_library(calls):
    x, w = torch.zeros(4, 16, dtype=BF16, requires_grad=True), torch.zeros(8, 16, dtype=BF16, requires_grad=True)
    lce.linear(x, w, activation="silu").sum().backward()
    assert [name for name, _ in calls] == ["forward", "backward"]
    assert x.grad.shape == x.shape and w.grad.shape == w.shape and calls[0][1][PREACT]


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("xt,wt", [(E4M3, E4M3), (BF16, E4M3), (E4M3, BF16), (torch.float32, torch.float32)])
def test_operands_other_than_bf16_are_refused(calls, xt, wt, grad):
    """The backward reads and writes two bytes a value: narrower operands would be overrun."""
    x, w = torch.zeros(4, 16).to(xt).requires_grad_(grad), torch.zeros(8, 16).to(wt).requires_grad_(grad)
    with pytest.raises(TypeError, match="must be torch.bfloat16"):
        lce.linear(x, w)
    assert not calls


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_without_gradients_any_width_and_no_preactivation(calls, mode):
    """A Parameter asks for a gradient inside no_grad too; the call there takes widths that only the
    backward refuses, and keeps nothing for it."""
    x, w = torch.zeros(4, 16, dtype=BF16), torch.nn.Parameter(torch.zeros(7, 16, dtype=BF16))
    with mode():
        y = lce.linear(x, w, activation="gelu")
    assert y.shape == (4, 7) and not y.requires_grad
    assert [name for name, _ in calls] == ["forward"] and not calls[0][1][PREACT]
    with pytest.raises(ValueError, match="multiple of 8"):
        lce.linear(x, w)


def test_residual_alone_keeps_no_preactivation(calls):
    x, w = torch.zeros(4, 16, dtype=BF16), torch.zeros(7, 16, dtype=BF16)
    r = torch.zeros(4, 7, dtype=BF16, requires_grad=True)
    lce.linear(x, w, activation="gelu", residual=r).sum().backward()
    assert [name for name, _ in calls] == ["forward"] and not calls[0][1][PREACT]
    assert torch.equal(r.grad, torch.ones_like(r))


def test_rows_far_apart_are_copied(calls):
    """As the last tokens of long sequences are: the library reads rows up to 16 MiB - 1 KB apart."""
    LDX, LDX_BACKWARD = 1, 4
    w = torch.zeros(8, 16, dtype=BF16)
    for ld, taken in (((1 << 23) - 512, (1 << 23) - 512), ((1 << 23) - 504, 16), (1 << 24, 16)):
        x = torch.empty(ld + 16, dtype=BF16)[:1].as_strided((2, 16), (ld, 1)).requires_grad_()
        lce.linear(x, w).backward(torch.zeros(2, 8, dtype=BF16))
        assert calls[-2][1][LDX] == calls[-1][1][LDX_BACKWARD] == taken
        assert x.grad.shape == (2, 16)
