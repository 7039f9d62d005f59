"""The root-mean-square norm on the GPU against its formulas in 64 bits.

Tolerances: a stored value is off by at most half a step of its type (torch.finfo(t).eps / 2 of
itself); the arithmetic before it is fp32, each operation off by 2^-24 of its result, sums by that
times their longest chain of additions (CHAIN covers the values of a lane, its lanes and the
workgroup) relative to the sum of the terms' magnitudes."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
CHAIN = 128


def _half(t):
    return torch.finfo(t).eps / 2


def _within(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    bad = off > 0
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst by {float(off.max()):.3g}"


def _inputs(n, H, dtype, seed, *, residual=True, wdtype=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = (r(n, H) * 2).to(dtype)
    res = (r(n, H) * 3).to(dtype) if residual else None
    w = None if wdtype is None else (1 + 0.3 * r(H)).to(wdtype)
    return x, res, w, (r(n, H) * 0.1).to(dtype), (r(n, H) * 0.1).to(dtype)


def _forward64(x, res, w, eps, offset):
    s = x.double() if res is None else (x.float() + res.float()).to(x.dtype).double()
    rstd = (s.square().mean(1) + eps).rsqrt()
    wd = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else w.double() + offset
    return s, rstd, wd


SHAPES = [(1, 1), (3, 7), (5, 64), (16, 128), (9, 129), (17, 512), (33, 1000), (7, 2048), (4, 4096), (3, 4099),
          (2, 6656), (3, 8192), (2, 8200), (2, 16384), (2, 16383), (1300, 256), (300, 1003),
          (41, 768), (7, 1536), (2, 3080), (700, 4160), (513, 2056)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H", SHAPES)
def test_forward_and_backward(n, H, dtype):
    eps = 1e-5
    for i, (residual, wdtype, offset) in enumerate([(True, dtype, 0.0), (False, F32, 1.0), (True, None, 0.0),
                                                    (False, BF16, 0.0)]):
        x, res, w, gy, gs = _inputs(n, H, dtype, 100 * n + H + i, residual=residual, wdtype=wdtype)
        r = lce.lce_rms_norm(x, w, residual=res, eps=eps, weight_offset=offset, want_rstd=True)
        s, rstd, wd = _forward64(x, res, w, eps, offset)
        if residual:
            assert torch.equal(r.sum.double(), s)
        else:
            assert r.sum is None
        _within(r.rstd, rstd, CHAIN * U * rstd, "rstd")
        y = s * rstd[:, None] * wd
        _within(r.y, y, (_half(dtype) + CHAIN * U) * y.abs(), "y")
        gx, gw = lce.lce_rms_norm_backward(gy, s.to(dtype), w, r.rstd, grad_sum=gs if residual else None,
                                           weight_offset=offset)
        a, q = gy.double() * wd, rstd[:, None]
        up = gs.double() if residual else torch.zeros_like(s)
        want = q * (a - s * q * q * (a * s).mean(1, keepdim=True)) + up
        size = q * (a.abs() + s.abs() * q * q * (a * s).abs().mean(1, keepdim=True)) + up.abs()
        _within(gx, want, _half(dtype) * want.abs() + 2 * CHAIN * U * size, "grad_x")
        if w is None:
            assert gw is None
        else:
            assert gw.dtype == w.dtype
            term = gy.double() * s * q
            want = term.sum(0)
            _within(gw, want, _half(w.dtype) * want.abs() + (CHAIN + n / 256 + 200) * U * term.abs().sum(0),
                    "grad_weight")


@pytest.mark.parametrize("n,H", SHAPES[:16])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_eight_bits(n, H, dtype):
    x, res, w, _, _ = _inputs(n, H, dtype, n + H, wdtype=dtype)
    x[n // 2] = 0
    res[n // 2] = 0   # a row of zeros
    r = lce.lce_rms_norm(x, w, residual=res, out_dtype=E4M3)
    s, rstd, wd = _forward64(x, res, w, 1e-6, 0.0)
    y = s * rstd[:, None] * wd
    scale = y.abs().amax(1) / 448
    scale[n // 2] = 1
    assert r.y.dtype == E4M3 and float(r.scale[n // 2]) == 1.0 and not bool(r.y[n // 2].float().any())
    _within(r.scale, scale, 2 * CHAIN * U * scale, "scale")
    v = y / scale[:, None]
    # half a step of a normal value is 2^-4 of it; below 2^-6 the step is 2^-9
    _within(r.y.float(), v, (2.0 ** -4 + 4 * CHAIN * U) * v.abs() + 2.0 ** -10 * (1 + 2.0 ** -6), "y / scale")
    assert bool((r.y.float().abs().amax(1) <= 448).all())


def test_tiny_rows_keep_finite_scales():
    x = torch.full((2, 64), 1e-38, device=DEV)
    x[1] = 1e-30
    r = lce.lce_rms_norm(x, torch.full((64,), 1e-7, device=DEV), eps=1.0, out_dtype=E4M3)
    assert bool(torch.isfinite(r.scale).all()) and bool((r.scale > 0).all())
    assert bool(torch.isfinite(r.y.float()).all())


def test_infinities_and_nans_stay_in_their_rows():
    x, res, w, gy, gs = _inputs(4, 100, F32, 3, wdtype=F32)
    clean = lce.lce_rms_norm(x, w, residual=res, want_rstd=True)
    x[1, 7], x[2, 9] = float("inf"), float("nan")
    r = lce.lce_rms_norm(x, w, residual=res, want_rstd=True)
    for row in (0, 3):
        assert torch.equal(r.y[row], clean.y[row])
    assert float(r.rstd[1]) == 0.0 and bool(torch.isnan(r.y[1, 7])) and float(r.y[1, 8]) == 0.0
    assert bool(torch.isnan(r.y[2]).all())
    gx, _ = lce.lce_rms_norm_backward(gy, r.sum, w, r.rstd)
    ref, _ = lce.lce_rms_norm_backward(gy, clean.sum, w, clean.rstd)
    assert torch.equal(gx[0], ref[0]) and torch.equal(gx[3], ref[3])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,ld,first", [(64, 96, 0), (100, 113, 1), (256, 264, 8), (2048, 2056, 3)])
def test_strides_and_what_lies_beside(H, ld, first, dtype):
    """Row strides, rows that start off a 16-byte boundary; columns past H and rows past n stay."""
    n = 5
    x, res, w, gy, gs = _inputs(n, H, dtype, H, wdtype=dtype)

    def wide(t=None, fill=7.0):
        b = torch.full((n + 1, ld), fill, dtype=dtype, device=DEV)
        v = b.reshape(-1)[first:first + n * ld].view(n, ld)[:, :H]
        if t is not None:
            v.copy_(t)
        return b, v

    (_, xv), (_, rv), (yb, yv), (sb, sv) = wide(x), wide(res), wide(), wide()
    r = lce.lce_rms_norm(xv, w, residual=rv, y=yv, sum_out=sv, want_rstd=True)
    ref = lce.lce_rms_norm(x, w, residual=res, want_rstd=True)
    assert torch.equal(sv, ref.sum)
    _within(r.y, ref.y.double(), (2 * _half(dtype) + CHAIN * U) * ref.y.double().abs(), "y")
    gb, gv = wide()
    gx, gw = lce.lce_rms_norm_backward(wide(gy)[1], sv, w, r.rstd, grad_sum=wide(gs)[1], grad_x=gv)
    gx0, gw0 = lce.lce_rms_norm_backward(gy, ref.sum, w, ref.rstd, grad_sum=gs)
    size = gx0.double().abs() + gy.double().abs() + 1
    _within(gx, gx0.double(), 2 * _half(dtype) * size + CHAIN * U * size, "grad_x")
    _within(gw, gw0.double(), 2 * _half(dtype) * gw0.double().abs() + 1e-5, "grad_weight")
    for b in (yb, sb, gb):
        flat, inside = b.reshape(-1), torch.zeros(b.numel(), dtype=torch.bool, device=DEV)
        inside[first:first + n * ld].view(n, ld)[:, :H] = True
        assert bool((flat[~inside] == 7.0).all())
    # over the residual's own buffer
    again = lce.lce_rms_norm(xv, w, residual=rv, sum_out=rv)
    assert torch.equal(again.sum, ref.sum) and torch.equal(again.y, r.y) and torch.equal(rv, ref.sum)


def test_offsets_past_32_bits():
    """Rows 2^31 elements apart: byte offsets past 32 bits in every operand."""
    H, ld = 1000, (1 << 31) + 8

    def far(t=None):
        v = torch.zeros(ld + H, dtype=BF16, device=DEV).as_strided((2, H), (ld, 1))
        return v if t is None else v.copy_(t)

    x, _, w, gy, _ = _inputs(2, H, BF16, 5, residual=False, wdtype=BF16)
    ref = lce.lce_rms_norm(x, w, want_rstd=True)
    xs, ys = far(x), far()
    r = lce.lce_rms_norm(xs, w, y=ys, want_rstd=True)
    assert torch.equal(r.y, ref.y) and torch.equal(r.rstd, ref.rstd)
    gx, gw = lce.lce_rms_norm_backward(gy, x, w, ref.rstd)
    got, gw2 = lce.lce_rms_norm_backward(far(gy), xs, w, r.rstd, grad_x=ys)
    assert torch.equal(got, gx) and torch.equal(gw2, gw)


def test_no_rows():
    x = torch.empty((0, 64), dtype=BF16, device=DEV)
    w = torch.ones(64, dtype=BF16, device=DEV)
    r = lce.lce_rms_norm(x, w, residual=x, want_rstd=True)
    assert r.y.shape == (0, 64)
    gw = torch.full((64,), 3.0, dtype=BF16, device=DEV)
    lce.lce_rms_norm_backward(x, x, w, r.rstd, grad_weight=gw)
    assert not bool(gw.any())


@pytest.mark.parametrize("residual", [False, True])
def test_autograd_matches_the_formula_and_differences(residual):
    torch.manual_seed(0)
    B, T, H = 2, 3, 40
    x = torch.randn(B, T, H, device=DEV, requires_grad=True)
    res = torch.randn(B, T, H, device=DEV, requires_grad=True) if residual else None
    w = torch.randn(H, device=DEV, requires_grad=True)
    cy, cs = torch.randn(B, T, H, device=DEV), torch.randn(B, T, H, device=DEV)
    leaves = [t for t in (x, w, res) if t is not None]

    def loss64(*ts):
        x_, w_ = ts[0], ts[1]
        s = x_ + ts[2] if residual else x_
        y = s / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt() * (w_ + 0.5)
        return (y * cy.double()).sum() + ((s * cs.double()).sum() if residual else 0.0)

    out = lce.rms_norm(x, w, residual=res, weight_offset=0.5)
    loss = (out[0] * cy).sum() + (out[1] * cs).sum() if residual else (out * cy).sum()
    got = torch.autograd.grad(loss, leaves)
    d = [t.detach().double().requires_grad_() for t in leaves]
    want = torch.autograd.grad(loss64(*d), d)
    for a, b in zip(got, want):
        _within(a, b, 1e-5 * (b.abs() + 1), "autograd")
    # and against differences of the 64-bit loss along one direction per leaf
    for i, t in enumerate(d):
        v = torch.randn_like(t)
        with torch.no_grad():
            hi = loss64(*[u + 1e-5 * v if j == i else u for j, u in enumerate(d)])
            lo = loss64(*[u - 1e-5 * v if j == i else u for j, u in enumerate(d)])
        slope = float((hi - lo) / 2e-5)
        assert float((got[i].double() * v).sum()) == pytest.approx(slope, rel=1e-4, abs=1e-4)


def test_autograd_of_strided_and_single_rows_on_another_stream():
    base = torch.randn(40, 3, 80, device=DEV)
    w = torch.randn(64, device=DEV, requires_grad=True)
    g = torch.randn(3, 40, 64, device=DEV)
    for view in (lambda t: t[:, :, 8:72].transpose(0, 1), lambda t: t[:1, :1, :64].expand(3, 40, 64),
                 lambda t: t[:1, 1:2, 3:67].transpose(0, 2).reshape(1, 64), lambda t: t[7:8, 0, ::1][:, :64]):
        x = view(base).detach().requires_grad_()
        cot = g if x.dim() == 3 else g[0, :1]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = lce.rms_norm(x, w)
            gx, gw = torch.autograd.grad(y, (x, w), cot)
        torch.cuda.synchronize()
        d, dw = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
        want = torch.autograd.grad(d / (d.square().mean(-1, keepdim=True) + 1e-6).sqrt() * dw, (d, dw), cot.double())
        for a, b in zip((gx, gw), want):
            _within(a, b, 1e-5 * (b.abs() + 1), "grad")


def test_autograd_with_only_one_output_used():
    x = torch.randn(4, 64, device=DEV, requires_grad=True)
    res = torch.randn(4, 64, device=DEV, requires_grad=True)
    w = torch.ones(64, device=DEV, requires_grad=True)
    y, s = lce.rms_norm(x, w, residual=res)
    gx, gr = torch.autograd.grad(s.sum(), (x, res), retain_graph=True)
    assert bool((gx == 1).all()) and bool((gr == 1).all())
    g = torch.randn_like(y)
    gx, gw = torch.autograd.grad(y, (x, w), g)
    a, b = lce.lce_rms_norm_backward(g, s.detach(), w.detach(), (s.detach().square().mean(1) + 1e-6).rsqrt())
    _within(gx, a.double(), 1e-5 * (a.double().abs() + 1), "grad_x")
    _within(gw, b.double(), 1e-5 * (b.double().abs() + 1), "grad_weight")


def test_gradients_of_gradients_are_refused():
    x = torch.randn(4, 64, device=DEV, requires_grad=True)
    w = torch.ones(64, device=DEV, requires_grad=True)
    (gx,) = torch.autograd.grad(lce.rms_norm(x, w).square().sum(), (x,), create_graph=True)
    (ref,) = torch.autograd.grad(lce.rms_norm(x, w).square().sum(), (x,))
    assert torch.equal(gx, ref)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.sum().backward()


def test_repeats_bit_for_bit_and_on_other_streams():
    x, res, w, gy, gs = _inputs(3000, 768, BF16, 9, wdtype=BF16)
    torch.cuda.synchronize()
    runs = []
    for st in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        r = lce.lce_rms_norm(x, w, residual=res, want_rstd=True, stream=st)
        runs.append((r.y, r.sum, *lce.lce_rms_norm_backward(gy, r.sum, w, r.rstd, grad_sum=gs, stream=st)))
    torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_captured_and_replayed():
    x, res, w, gy, gs = _inputs(257, 1000, BF16, 11, wdtype=F32)
    bufs = dict(y=torch.empty_like(x), sum_out=torch.empty_like(x), rstd=torch.empty(257, device=DEV))
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(lce.lce_rms_norm_workspace_bytes(257, 1000), dtype=torch.uint8, device=DEV)

    def step():
        lce.lce_rms_norm(x, w, residual=res, **bufs)
        lce.lce_rms_norm_backward(gy, bufs["sum_out"], w, bufs["rstd"], grad_sum=gs, grad_x=gx, grad_weight=gw,
                                  workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(torch.randn(257, 1000, device=DEV) + k)
        graph.replay()
        got = [t.clone() for t in (*bufs.values(), gx, gw)]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (*bufs.values(), gx, gw)))
