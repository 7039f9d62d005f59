"""lce_linear_blocks_backward called by itself: gradients of either type, rows and scales of any strides, outputs
and a workspace that the caller brings, one gradient without the other.

Tolerances as in test_gpu_blocks.py: quantised operands are exact, products lose what the 8-bit instructions cut
off and (length + 8) 2^-24 of the sum of magnitudes, and the store half a step of its type.  grad_bias is a sum
of n values in fp32, (n + 8) 2^-24 of the sum of magnitudes, and a store."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402
from test_gpu_blocks import BF16, DEV, F32, HALF, U, cut_off, normal, quantised, spread, within  # noqa: E402

SIZES = [(1, 1, 1), (5, 300, 130), (40, 1001, 77), (129, 515, 1030), (300, 128, 384), (517, 256, 2051), (1030, 1024, 512)]


def operands(n, K, M, dtype):
    """grad_out [n, M] and the transposed 8-bit operands of a product with x [n, K], weight [M, K]."""
    r = normal(3 * n + K + M)
    x = (r(n, K) * torch.exp2(r(1, K))).to(BF16)
    w = (r(M, K) / math.sqrt(K)).to(BF16)
    g = (1e-3 * r(n, M) * torch.exp2(3 * r(n, 1))).to(dtype)
    xt = lce.lce_quantize_blocks(x, blocks=None, transposed="tile")
    wt = lce.lce_quantize_blocks(w, blocks=None, transposed="tile")
    return g, xt, wt


def product(got, a, b, length, what):
    z = a @ b.t()
    within(got, z, HALF * z.abs() + (length + 8) * U * (a.abs() @ b.abs().t()) + cut_off(a, b), what)


def check(got, g, xt, wt, K):
    n, M = g.shape
    if got.grad_x is not None:
        q, s = quantised(g, False)
        product(got.grad_x, q * spread(s, n, M, False), wt.values_t.double() * spread(wt.scale_t, K, M, True), M, "grad_x")
    if got.grad_weight is not None:
        q, s = quantised(g.t(), False)
        product(got.grad_weight, q * spread(s, M, n, False), xt.values_t.double() * spread(xt.scale_t, K, n, True), n, "grad_weight")
    if got.grad_bias is not None:
        s = g.double().sum(0)
        half = torch.finfo(got.grad_bias.dtype).eps / 2
        within(got.grad_bias, s, half * s.abs() + (n + 8) * U * g.double().abs().sum(0), "grad_bias")


@pytest.mark.parametrize("n,K,M", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_both_types_of_gradients(n, K, M, dtype):
    g, xt, wt = operands(n, K, M, dtype)
    for bias_dtype in (None, F32):
        got = lce.lce_linear_blocks_backward(g, xt.values_t, xt.scale_t, wt.values_t, wt.scale_t, want_grad_bias=True,
                                             grad_bias_dtype=bias_dtype)
        assert got.grad_x.shape == (n, K) and got.grad_weight.shape == (M, K) and got.grad_bias.dtype == (bias_dtype or BF16)
        check(got, g, xt, wt, K)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,K,M", [(5, 300, 130), (300, 515, 200)])
def test_one_gradient_alone(n, K, M, dtype):
    g, xt, wt = operands(n, K, M, dtype)
    both = lce.lce_linear_blocks_backward(g, xt.values_t, xt.scale_t, wt.values_t, wt.scale_t, want_grad_bias=True)
    only_x = lce.lce_linear_blocks_backward(g, wt=wt.values_t, scale_wt=wt.scale_t, want_grad_bias=True)
    only_w = lce.lce_linear_blocks_backward(g, xt.values_t, xt.scale_t)
    assert only_x.grad_weight is None and only_w.grad_x is None and only_w.grad_bias is None
    assert torch.equal(only_x.grad_x, both.grad_x) and torch.equal(only_x.grad_bias, both.grad_bias)
    assert torch.equal(only_w.grad_weight, both.grad_weight)
    check(both, g, xt, wt, K)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,K,M", [(5, 300, 130), (300, 515, 1030)])
def test_strides_given_outputs_and_workspace(n, K, M, dtype):
    g, xt, wt = operands(n, K, M, dtype)
    hold = torch.full((n + 2, M + 13), math.nan, dtype=dtype, device=DEV)
    rows = hold[1:n + 1, 5:M + 5]
    rows.copy_(g)
    scales = [s.t().contiguous().t() for s in (xt.scale_t, wt.scale_t)]   # block by block instead of row by row
    place = torch.full((n + 3, K + 9), 7.0, dtype=BF16, device=DEV)
    grad_x = place[2:n + 2, 3:K + 3]
    grad_weight = torch.full((M, K), 7.0, dtype=BF16, device=DEV)
    grad_bias = torch.full((M,), 7.0, device=DEV)
    need = lce.lce_linear_blocks_backward_workspace_bytes(n, K, M)
    room = torch.full((need + 512,), 171, dtype=torch.uint8, device=DEV)
    got = lce.lce_linear_blocks_backward(rows, xt.values_t, scales[0], wt.values_t, scales[1], grad_x=grad_x,
                                         grad_weight=grad_weight, grad_bias=grad_bias, workspace=room[:need])
    assert got.grad_x is grad_x and got.grad_weight is grad_weight and got.grad_bias is grad_bias
    check(got, g, xt, wt, K)
    outside = torch.ones_like(place, dtype=torch.bool)
    outside[2:n + 2, 3:K + 3] = False
    assert bool((place[outside] == 7).all()) and bool((room[need:] == 171).all())   # around them, as it was


def test_without_tokens():
    wt = lce.lce_quantize_blocks(normal(1)(24, 40), blocks=None, transposed="tile")
    xt = lce.lce_quantize_blocks(torch.empty(0, 40, device=DEV), blocks=None, transposed="tile")
    got = lce.lce_linear_blocks_backward(torch.empty(0, 24, device=DEV), xt.values_t, xt.scale_t, wt.values_t, wt.scale_t,
                                         want_grad_bias=True, grad_bias_dtype=F32)
    assert got.grad_x.shape == (0, 40) and not bool(got.grad_weight.any()) and not bool(got.grad_bias.any())


def test_captured_and_replayed():
    n, K, M = 200, 256, 384
    g, xt, wt = operands(n, K, M, F32)
    args = (g, xt.values_t, xt.scale_t, wt.values_t, wt.scale_t)
    lce.lce_linear_blocks_backward(*args, want_grad_bias=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = lce.lce_linear_blocks_backward(*args, want_grad_bias=True)
    for k in range(3):
        g.copy_(normal(k)(n, M))
        graph.replay()
        torch.cuda.synchronize()
        want = lce.lce_linear_blocks_backward(*args, want_grad_bias=True)
        for a, b in zip((held.grad_x, held.grad_weight, held.grad_bias), (want.grad_x, want.grad_weight, want.grad_bias)):
            assert torch.equal(a, b)
