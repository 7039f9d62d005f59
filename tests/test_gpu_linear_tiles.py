"""The matrix product on the GPU against 64 bits, at sizes that take every shape of tile, with and without a
cut last step of K and a split along K (test_linear_plan_cpu.py holds them to that).  Tolerances as in
test_gpu_linear.py."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import test_gpu_linear as base  # noqa: E402
from linear_plan import COVER  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n,K,M", COVER["bf16"])
def test_bf16(n, K, M):
    base._check_forward(n, K, M, n + K + M, out_dtype=F32)
    base._check_forward(n, K, M, n * 3 + M, act=base.ACTS[(n + M) % 5], bias=BF16, residual=True, preact=True)


@pytest.mark.parametrize("n,K,M", COVER["e4m3"])
def test_e4m3(n, K, M):
    base._check_forward(n, K, M, n + K + M, e4m3=True)
    base._check_forward(n, K, M, n * 3 + M, e4m3=True, act=base.ACTS[(n + M + 2) % 5], bias=F32, residual=True)
