"""Softcap and temperature at the ends of their ranges, against 64 bits.

Tolerance: half a step of the logits' type for the one rounding and 16 fp32 operations before it (2^-24
each), as for ordinary values; what lies past the type's largest value is an infinity."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def _check(got, want, dtype):
    got, want, info = got.double().cpu(), want.cpu(), torch.finfo(dtype)
    assert not bool(torch.isnan(got).any())
    tol = (info.eps / 2 + 16 * 2.0 ** -24) * want.abs() + info.tiny
    # between the type's largest value and half a step past it a value may round either way
    high = want.abs() > info.max * (1 + info.eps / 2 + 2.0 ** -20)
    low = want.abs() < info.max * (1 - 2.0 ** -20)
    assert torch.equal(got[high], torch.sign(want[high]) * math.inf)
    assert bool(((got - want).abs() <= tol)[low].all()), (got[low], want[low])


@pytest.mark.parametrize("listed", [False, True], ids=["no_lists", "history"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cap", [1e-30, 1e-3, 5.0, 30.0, 1e20, 1e38])
def test_softcap_and_temperature(cap, dtype, listed):
    base = [0.0, 1e-4, 0.3, 0.469, 1.0, 5.0, 7.4, 7.6, 20.0, 100.0, 1e4]
    x = torch.tensor([base + [-v for v in base] + [1e20, -1e20, 1e30, -1e30]], device=DEV)
    temps = torch.tensor([0.0, 1e-37, 5e-38, 1.2e-38, 1e-20, 0.5, 1.0, 1e20, 1e37], device=DEV)
    x = x.expand(temps.numel(), -1).contiguous().to(dtype)
    n, V = x.shape
    r = {}
    if listed:   # every other token, counted without a penalty: worked out apart from the rest
        r = dict(history=torch.arange(0, V, 2, device=DEV).expand(n, -1), repetition=torch.ones(n, device=DEV))
    got = lce.lce_logits_process(x, softcap=cap, temperature=temps, out=torch.empty_like(x), **r)
    c = float(torch.tensor(cap, dtype=F32))
    t = temps.double()[:, None]
    want = c * torch.tanh(x.double() / c)
    _check(got, torch.where(t > 0, want / torch.where(t > 0, t, 1.0), want), dtype)
