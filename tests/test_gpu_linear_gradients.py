"""Gradients of the matrix product on the GPU for upstream gradients that lie far apart in memory."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
WIDEST = (1 << 23) - 512   # the row stride of bf16 rows up to which the product reads them in place


@pytest.mark.parametrize("n,K,M,ld", [(2, 64, 40, (1 << 31) + 8), (130, 136, 264, (1 << 24) + 8),
                                      (40, 264, 136, WIDEST), (40, 264, 136, WIDEST + 8), (2, 512, 1000, 1 << 31)])
def test_grad_out_rows_far_apart(n, K, M, ld):
    """Tiles whose rows of grad_out span 4 GiB and more: the same gradients as from its contiguous copy."""
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randn(n, K, generator=g, device=DEV).to(BF16)
    w = (torch.randn(M, K, generator=g, device=DEV) / 8).to(BF16)
    near = torch.randn(n, M, generator=g, device=DEV).to(BF16)
    far = torch.empty(ld * (n - 1) + M, dtype=BF16, device=DEV).as_strided((n, M), (ld, 1))
    far.copy_(near)
    want = lce.lce_linear_backward(near, x, w, want_grad_bias=True)
    exact = near.double() @ w.double()
    size = near.double().abs() @ w.double().abs()
    # half a step of bf16, and the fp32 sum of M products
    assert bool(((want.grad_x.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + (M + 8) * 2.0 ** -24 * size).all())
    got = lce.lce_linear_backward(far, x, w, want_grad_bias=True)
    for name in ("grad_x", "grad_weight", "grad_bias"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    gx, gw = torch.autograd.grad(lce.linear(xl, wl), (xl, wl), far)
    assert torch.equal(gx, want.grad_x) and torch.equal(gw, want.grad_weight)


def test_last_tokens_of_long_sequences():
    """x's rows 32 MiB apart: the product and its gradients as from a contiguous copy."""
    B, T, K, M = 3, 4097, 4096, 264
    g = torch.Generator(device=DEV).manual_seed(1)
    hidden = torch.zeros(B, T, K, device=DEV, dtype=BF16)
    hidden[:, -1] = torch.randn(B, K, generator=g, device=DEV).to(BF16)
    w = (torch.randn(M, K, generator=g, device=DEV) / 64).to(BF16).requires_grad_()
    c = torch.randn(B, M, generator=g, device=DEV).to(BF16)
    near = hidden[:, -1].contiguous().requires_grad_()
    want = lce.linear(near, w, activation="silu")
    x = hidden[:, -1].requires_grad_()
    assert x.stride(0) * 2 > 1 << 24
    got = lce.linear(x, w, activation="silu")
    assert torch.equal(got, want)
    for a, b in zip(torch.autograd.grad(got, (x, w), c), torch.autograd.grad(want, (near, w), c)):
        assert torch.equal(a, b)


def test_a_parameter_of_odd_width_without_gradients():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(9, 128, generator=g, device=DEV).to(BF16)
    w = torch.nn.Parameter((torch.randn(1003, 128, generator=g, device=DEV) / 8).to(BF16))
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(lce.linear(x, w, activation="gelu"), lce.lce_linear(x, w.detach(), activation="gelu").out)
