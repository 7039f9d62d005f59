"""The norm's values again under a comparison that a NaN fails, over every shape of a row.

The tests of test_gpu_norm.py take `difference > tolerance` as the fault, which a NaN is not; here the
same ones run with `not (difference <= tolerance)`, at their sizes and at widths that, with whole and with
cut last accesses, fill each choice of lanes and accesses per lane, several rows per workgroup included."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import test_gpu_norm as norm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
MORE = [(5, 401), (5, 1537), (5, 4095), (2100, 100), (2100, 103), (1100, 1000), (600, 8191), (530, 16383), (530, 16384),
        (300, 12292)]


@pytest.fixture(autouse=True)
def nan_fails(monkeypatch):
    def within(got, want, tol, what):
        off = (got.double() - want).abs() - tol
        bad = ~(off <= 0)
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst by {float(off.max()):.3g}"

    monkeypatch.setattr(norm, "_within", within)


def test_a_nan_fails():
    with pytest.raises(AssertionError, match="1 of 2 outside"):
        norm._within(torch.tensor([1.0, float("nan")]), torch.tensor([1.0, 1.0]), 0.1, "y")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H", norm.SHAPES + MORE)
def test_forward_and_backward(n, H, dtype):
    norm.test_forward_and_backward(n, H, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H", norm.SHAPES + MORE)
def test_eight_bits(n, H, dtype):
    norm.test_eight_bits(n, H, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,ld,first", [(64, 96, 0), (100, 113, 1), (256, 264, 8), (2048, 2056, 3), (8200, 8203, 1),
                                        (16384, 16400, 5)])
def test_strides_and_what_lies_beside(H, ld, first, dtype):
    norm.test_strides_and_what_lies_beside(H, ld, first, dtype)
