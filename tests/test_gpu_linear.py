"""The matrix product with its epilogue on the GPU against the formulas in 64 bits.

Tolerances: z is an fp32 sum of K products, off by at most K 2^-24 times the sum of their magnitudes
in any order (on the whole, as a random walk, by about sqrt(K) 2^-24 of it, which the 2-norm is held to
with a margin of 5); the activations' slopes are at most 1.13 and their own arithmetic is off by at
most 2^-20 (|z| + 1); the store is off by half a step of its type.  The backward is compared from the
pre-activation that the forward stored: dz is rounded to bf16, then summed like z.

The 8-bit matrix instructions bring eight neighbouring products to a unit of 2^-13 of the largest one's
power of two, cutting the rest off, before they add: each of the other seven is off by less than 2^-13
of the group's largest, and the groups' sums are fp32 as above."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _half(t):
    return torch.finfo(t).eps / 2


def _within(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    bad = ~(off <= 0)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst by {float(off.max()):.3g}"


def _act(kind, z):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2)),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
            "silu": lambda: z * torch.sigmoid(z)}[kind]()


def _slope(kind, z):
    z = z.detach().clone().requires_grad_()
    if kind == "relu":
        return (z > 0).double()
    return torch.autograd.grad(_act(kind, z).sum(), z)[0].detach()


def _normal(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device=DEV)


def _quantised(t):
    scale = t.abs().amax(1).clamp_min(1e-12) / 448
    return (t / scale[:, None]).to(E4M3), scale


def _cut_off(x, w):
    """Bound on what the 8-bit products lose: 7 2^-13 of each group's largest, summed over the groups."""
    n, K = x.shape
    rows = max(1, (1 << 27) // (w.shape[0] * K))
    parts = [(x[i:i + rows, None].abs() * w[None].abs()).view(-1, w.shape[0], K // 8, 8).amax(3).sum(2)
             for i in range(0, n, rows)]
    return 7 * 2.0 ** -13 * torch.cat(parts).double()


def _check_forward(n, K, M, seed, *, e4m3=False, act="none", bias=None, residual=False, out_dtype=BF16, preact=False):
    r = _normal(seed)
    x, w = r(n, K), r(M, K) / math.sqrt(K)
    kw = {}
    if e4m3:
        (x, sx), (w, sw) = _quantised(x), _quantised(w)
        kw.update(scale_x=sx, scale_w=sw)
        xd, wd = x.double() * sx.double()[:, None], w.double() * sw.double()[:, None]
    else:
        x, w = x.to(BF16), w.to(BF16)
        xd, wd = x.double(), w.double()
    b = None if bias is None else r(M).to(bias)
    res = r(n, M).to(out_dtype) if residual else None
    got = lce.lce_linear(x, w, bias=b, activation=act, residual=res, out_dtype=out_dtype, want_preact=preact, **kw)
    z, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    err = (K + 8) * U * size
    if e4m3:
        err = err + _cut_off(xd.float(), wd.float())
    if preact:
        _within(got.preact, z, _half(BF16) * z.abs() + err, "preact")
    y = _act(act, z)
    tol = 1.13 * err + (0 if act in ("none", "relu") else 2.0 ** -20) * (z.abs() + 1)
    if res is not None:
        y = y + res.double()
        tol = tol + 2 * U * (y.abs() + res.double().abs())
    _within(got.out, y, _half(out_dtype) * y.abs() + tol, "out")
    if out_dtype == F32 and act == "none":
        rel = float((got.out.double() - y).norm() / y.norm())
        assert rel <= 5 * math.sqrt(K + 8) * U, rel
    return got


# (n, K, M): one token to many, features that end inside a tile, K that ends inside a step, products
# that are split along K, and every tile shape
SIZES = [(1, 8, 1), (1, 64, 256), (2, 4096, 512), (3, 72, 7), (5, 1000, 33), (16, 6656, 1000), (17, 520, 129),
         (32, 2048, 4099), (33, 128, 127), (64, 4096, 256), (65, 264, 1000), (100, 640, 2049), (129, 1024, 128),
         (128, 8192, 640), (255, 200, 511), (300, 1000, 1003), (513, 512, 1025), (1000, 136, 2000), (1030, 2048, 4100),
         (2048, 512, 8192)]


@pytest.mark.parametrize("n,K,M", SIZES)
def test_bf16(n, K, M):
    _check_forward(n, K, M, n + K + M, out_dtype=F32)
    _check_forward(n, K, M, n * 3 + M, out_dtype=BF16, act=ACTS[(n + M) % 5], bias=BF16, residual=True, preact=True)


@pytest.mark.parametrize("n,K,M", [(n, -(-K // 16) * 16, M) for n, K, M in SIZES])
def test_e4m3(n, K, M):
    _check_forward(n, K, M, n + K + M, e4m3=True)
    _check_forward(n, K, M, n * 3 + M, e4m3=True, act=ACTS[(n + M + 2) % 5], bias=F32, residual=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bias,residual", [(None, False), (F32, True), (BF16, False), (None, True)])
def test_epilogues(act, out_dtype, bias, residual):
    for n, K, M in ((7, 1024, 200), (150, 4096, 130)):   # whole and split along K
        _check_forward(n, K, M, 17, act=act, out_dtype=out_dtype, bias=bias, residual=residual, preact=act != "none")


def test_activations_far_out():
    """Through an identity weight: the activations over a wide range, infinities and NaN."""
    K = 64
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 0.5, -0.5, 1, -1, 3, -3, 5.5, -5.5, 9, -9, 14, -14, 30,
                      -30, 90, -90, 1e4, -1e4, 1e30, -1e30], device=DEV, dtype=BF16)
    x = torch.zeros(1, K, device=DEV, dtype=BF16)
    x[0, :v.numel()] = v
    eye = torch.eye(K, device=DEV, dtype=BF16)
    for act in ACTS:
        got = lce.lce_linear(x, eye, activation=act, out_dtype=F32).out[0, :v.numel()].double()
        z = v.double()
        want = _act(act, z.clamp(-1e9, 1e9)) if act == "gelu_tanh" else _act(act, z)
        want = torch.where(z > 1e9, z, torch.where(z < -1e9, z if act == "none" else torch.zeros_like(z), want))
        _within(got, want, 2.0 ** -20 * (want.abs() + z.abs().clamp_max(20)) , act)
    x[0, 1] = float("nan")
    for act in ACTS:   # a NaN token stays one; other tokens are not touched by it
        two = torch.cat([x, torch.ones_like(x)])
        out = lce.lce_linear(two, eye, activation=act, out_dtype=F32).out
        assert bool(torch.isnan(out[0]).any()) and bool(torch.isfinite(out[1]).all())


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_far_out(act):
    """Far from zero every slope is 0 or 1, up to the largest bf16 value; a NaN stays one (relu's slope there is 0)."""
    big = torch.finfo(BF16).max
    pre = torch.tensor([[30, -30, 1e4, -1e4, 1e18, -1e18, 1e20, -1e20, 1e30, -1e30, 1e38, -1e38, big, -big, 0.5,
                         float("nan")]], device=DEV).to(BF16)
    g = torch.ones_like(pre)
    x, w = torch.ones(1, 8, device=DEV, dtype=BF16), torch.ones(16, 8, device=DEV, dtype=BF16)
    got = lce.lce_linear_backward(g, x, w, activation=act, preact=pre, want_grad_bias=True, grad_bias_dtype=F32).grad_bias
    want = (pre[0, :14] > 0).double()
    _within(got[:14], want, 2.0 ** -20, act)   # e^-30 30 < 2^-38
    assert bool(torch.isnan(got[15])) == (act != "relu")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,K,M", [(5, 96, 70), (70, 160, 200), (260, 4096, 300)])
def test_strides_and_what_lies_beside(n, K, M, e4m3):
    """Row strides of every operand, output rows off the 16-byte boundaries, NaN beside the operands."""
    r = _normal(n)
    dt, pad = (E4M3, 16) if e4m3 else (BF16, 8)
    x, w = r(n, K).to(dt), (r(M, K) / 8).to(dt)
    ot = BF16 if e4m3 else F32
    res = r(n, M).to(ot)

    def wide(t, extra):
        b = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=DEV).to(t.dtype)
        b[:, :t.shape[1]].copy_(t)
        return b[:, :t.shape[1]]

    ref = lce.lce_linear(x, w, residual=res, out_dtype=ot, activation="silu", want_preact=True)
    for first in (0, 1, 4):
        ob = torch.full(((n + 1) * (M + 3),), 7.0, device=DEV, dtype=ot)
        ov = ob[first:first + n * (M + 3)].view(n, M + 3)[:, :M]
        pb = torch.full(((n + 1) * (M + 5),), 7.0, device=DEV, dtype=BF16)
        pv = pb[first:first + n * (M + 5)].view(n, M + 5)[:, :M]
        got = lce.lce_linear(wide(x, pad), wide(w, 2 * pad), residual=wide(res, 9), out=ov, preact=pv, activation="silu")
        assert torch.equal(got.out, ref.out) and torch.equal(got.preact, ref.preact)
        for b, v, ld in ((ob, ov, M + 3), (pb, pv, M + 5)):
            inside = torch.zeros(b.numel(), dtype=torch.bool, device=DEV)
            inside[first:first + n * ld].view(n, ld)[:, :M] = True
            assert bool((b[~inside] == 7.0).all())
    # the residual's own buffer as the output
    own = res.clone()
    assert torch.equal(lce.lce_linear(x, w, residual=own, out=own, activation="silu").out, ref.out)


@pytest.mark.parametrize("n,K", [(3, 256), (40, 512), (40, 8192)])
def test_offsets_past_32_bits(n, K):
    """Output, residual and pre-activation rows far apart, x and weight with the widest strides: byte
    offsets past 32 bits, in the kernel for few tokens, in tiles and with K split."""
    M, ld = 96, (1 << 32) // n // 8 * 8 + 64
    r = _normal(n)
    x, w, res = r(n, K).to(BF16), (r(M, K) / 16).to(BF16), r(n, M).to(BF16)
    want = lce.lce_linear(x, w, residual=res, activation="silu", want_preact=True)
    flat = [torch.zeros(ld * (n - 1) + M, dtype=BF16, device=DEV) for _ in range(3)]
    far = [f.as_strided((n, M), (ld, 1)) for f in flat]
    far[0].copy_(res)
    got = lce.lce_linear(x, w, residual=far[0], out=far[1], preact=far[2], activation="silu")
    assert torch.equal(got.out, want.out) and torch.equal(got.preact, want.preact)
    del flat, far
    wide = (1 << 23) - 1024                          # elements: just under 16 MiB
    xs = torch.zeros(wide * (n - 1) + K, dtype=BF16, device=DEV).as_strided((n, K), (wide, 1))
    ws = torch.zeros(wide * (M - 1) + K, dtype=BF16, device=DEV).as_strided((M, K), (wide, 1))
    xs.copy_(x), ws.copy_(w)
    got = lce.lce_linear(xs, ws, residual=res, activation="silu", want_preact=True)
    assert torch.equal(got.out, want.out) and torch.equal(got.preact, want.preact)


@pytest.mark.parametrize("M,ld", [(32776, 32776), (32776, 32784), (32777, 32777)])
def test_outputs_larger_than_the_caches(M, ld):
    """Just past 256 MB of output: rows whole 16 bytes apart, with a gap, and at an odd width."""
    n, K = 4096, 64
    r = _normal(M)
    x, w = r(n, K).to(BF16), (r(M, K) / 8).to(BF16)
    flat = r(n, ld).to(BF16)
    out, res, gap = flat[:, :M], flat[:, :M].clone(), flat[:, M:].clone()
    lce.lce_linear(x, w, residual=out, out=out, activation="relu")
    for i in range(0, n, 1024):
        xd, wd, rd = x[i:i + 1024].double(), w.double(), res[i:i + 1024].double()
        want = (xd @ wd.t()).clamp_min(0) + rd
        _within(out[i:i + 1024], want, _half(BF16) * want.abs() + (K + 8) * U * (xd.abs() @ wd.abs().t() + rd.abs()), "out")
    assert torch.equal(flat[:, M:], gap)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,K,M", [(1, 8, 8), (3, 64, 40), (60, 512, 1000), (130, 200, 136), (257, 1024, 512),
                                   (1000, 264, 2048), (2100, 1032, 520)])
@pytest.mark.parametrize("gdtype", [BF16, F32], ids=["bf16", "f32"])
def test_backward(n, K, M, act, gdtype):
    r = _normal(n + M)
    x, w = r(n, K).to(BF16), (r(M, K) / math.sqrt(K)).to(BF16)
    g = (r(n, M) * 0.1).to(gdtype)
    pre = lce.lce_linear(x, w, activation=act, want_preact=act != "none").preact
    got = lce.lce_linear_backward(g, x, w, activation=act, preact=pre, want_grad_bias=True, grad_weight_dtype=F32,
                                  grad_bias_dtype=F32)
    gd, xd, wd = g.double(), x.double(), w.double()
    dz = gd if act == "none" else gd * _slope(act, pre.double())
    # the slope's arithmetic, then the rounding to bf16 (none where grad_out is bf16 and passes through)
    each = 2.0 ** -20 * gd.abs() + (0 if act == "none" and gdtype == BF16 else _half(BF16)) * dz.abs()
    def close(got, want, err, terms, chain, what):
        _within(got, want, _half(got.dtype) * want.abs() + err + (chain + 8) * U * terms, what)
    close(got.grad_x, dz @ wd, each @ wd.abs(), (dz.abs() + each) @ wd.abs(), M, "grad_x")
    close(got.grad_weight, dz.t().contiguous() @ xd, each.t().contiguous() @ xd.abs(),
          (dz.abs() + each).t().contiguous() @ xd.abs(), n, "grad_weight")
    raw = 2.0 ** -20 * gd.abs()   # the bias's sums take dz as it is
    close(got.grad_bias, dz.sum(0), raw.sum(0), (dz.abs() + raw).sum(0), 40 + n / 128, "grad_bias")
    # one gradient at a time, in bf16, and from a strided grad_out
    gs = torch.cat([g, torch.full_like(g, float("nan"))], 1)[:, :M]
    one = [lce.lce_linear_backward(gs, x, w, activation=act, preact=pre, want_grad_x=i == 0, want_grad_weight=i == 1,
                                   want_grad_bias=i == 2) for i in range(3)]
    assert torch.equal(one[0].grad_x, got.grad_x) and one[0].grad_weight is None and one[0].grad_bias is None
    assert torch.equal(one[1].grad_weight, got.grad_weight.to(BF16)) and one[1].grad_x is None
    assert torch.equal(one[2].grad_bias, got.grad_bias.to(BF16))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradients_in_place_of_inputs(act):
    """Each gradient in the place of an input of its type and shape (K = M)."""
    n = K = 264
    r = _normal(6)
    x, w, g = r(n, K).to(BF16), (r(K, K) / 16).to(BF16), r(n, K).to(BF16)
    pre = lce.lce_linear(x, w, activation=act, want_preact=True).preact
    ref = lce.lce_linear_backward(g, x, w, activation=act, preact=pre)
    for gx in range(4):
        for gw in range(4):
            t = [g.clone(), x.clone(), w.clone(), pre.clone()]
            if gx == gw:
                continue
            got = lce.lce_linear_backward(t[0], t[1], t[2], activation=act, preact=t[3], grad_x=t[gx], grad_weight=t[gw])
            assert torch.equal(got.grad_x, ref.grad_x) and torch.equal(got.grad_weight, ref.grad_weight), (gx, gw)


def test_no_rows():
    x, w = torch.empty((0, 64), device=DEV, dtype=BF16), torch.ones((40, 64), device=DEV, dtype=BF16)
    assert lce.lce_linear(x, w).out.shape == (0, 40)
    r = lce.lce_linear_backward(torch.empty((0, 40), device=DEV, dtype=BF16), x, w, want_grad_bias=True)
    assert r.grad_x.shape == (0, 64) and not bool(r.grad_weight.any()) and not bool(r.grad_bias.any())


def test_autograd_matches_the_formula_and_differences():
    r = _normal(5)
    B, T, K, M = 2, 9, 64, 48
    for act in ACTS:
        leaves = [r(B, T, K).to(BF16), (r(M, K) / 8).to(BF16), r(M).to(F32), r(B, T, M).to(BF16)]
        for t in leaves:
            t.requires_grad_()
        c = r(B, T, M).to(BF16)
        y = lce.linear(leaves[0], leaves[1], leaves[2], activation=act, residual=leaves[3])
        assert y.shape == (B, T, M) and y.dtype == BF16
        got = torch.autograd.grad(y, leaves, c)
        d = [t.detach().double().requires_grad_() for t in leaves]

        def loss(ts):
            return ((_act(act, ts[0] @ ts[1].t() + ts[2]) + ts[3]) * c.double()).sum()

        want = torch.autograd.grad(loss(d), d)
        for t, a, b in zip(leaves, got, want):
            assert a.dtype == t.dtype and a.shape == t.shape
            # bf16 roundings of the pre-activation (slopes bend by at most 1.13), of dz and of the store
            assert float((a.double() - b).norm() / b.norm()) <= 3.2 * _half(BF16)
        if act == "relu":
            continue   # a difference may step over its corner
        for i, t in enumerate(d):
            v = torch.randn_like(t)
            with torch.no_grad():
                hi = loss([u + 1e-6 * v if j == i else u for j, u in enumerate(d)])
                lo = loss([u - 1e-6 * v if j == i else u for j, u in enumerate(d)])
            slope = float((hi - lo) / 2e-6)
            near = 3.2 * _half(BF16) * float(got[i].double().norm() * v.norm())
            assert abs(float((got[i].double() * v).sum()) - slope) <= near + 1e-4 * abs(slope)


def test_autograd_asks_only_for_what_is_needed():
    x = torch.randn(4, 32, device=DEV).to(BF16).requires_grad_()
    w = torch.randn(16, 32, device=DEV).to(BF16)
    y = lce.linear(x, w, activation="gelu")
    (gx,) = torch.autograd.grad(y, (x,), torch.ones_like(y))
    assert gx.shape == x.shape
    with torch.no_grad():
        assert not lce.linear(x, w, activation="gelu").requires_grad


def test_repeats_bit_for_bit_on_other_streams():
    r = _normal(8)
    x, w, g = r(200, 4096).to(BF16), r(256, 4096).to(BF16), r(200, 256).to(BF16)   # split along K
    assert lce.lce_linear_workspace_bytes(200, 4096, 256) > 0
    torch.cuda.synchronize()
    runs = []
    for st in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        b = lce.lce_linear_backward(g, x, w, want_grad_bias=True, stream=st)
        runs.append((lce.lce_linear(x, w, stream=st).out, b.grad_x, b.grad_weight, b.grad_bias))
    torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_captured_and_replayed():
    n, K, M = 130, 4096, 264
    r = _normal(3)
    x, w, g = r(n, K).to(BF16), r(M, K).to(BF16), r(n, M).to(BF16)
    out, pre = torch.empty(n, M, device=DEV, dtype=BF16), torch.empty(n, M, device=DEV, dtype=BF16)
    ws = torch.empty(lce.lce_linear_workspace_bytes(n, K, M), dtype=torch.uint8, device=DEV)
    wsb = torch.empty(lce.lce_linear_backward_workspace_bytes(n, K, M), dtype=torch.uint8, device=DEV)
    gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty(M, device=DEV)

    def step():
        lce.lce_linear(x, w, activation="gelu", out=out, preact=pre, workspace=ws)
        lce.lce_linear_backward(g, x, w, activation="gelu", preact=pre, grad_x=gx, grad_weight=gw, grad_bias=gb,
                                workspace=wsb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(torch.randn(n, K, device=DEV))
        graph.replay()
        got = [t.clone() for t in (out, pre, gx, gw, gb)]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, pre, gx, gw, gb)))


def test_refusals_on_the_gpu():
    x, w = torch.zeros(4, 64, device=DEV, dtype=BF16), torch.zeros(8, 64, device=DEV, dtype=BF16)
    for call, needle in ((lambda: lce.lce_linear(x[:, :60], w[:, :60]), "multiples of 8"),
                         (lambda: lce.lce_linear(x.reshape(-1)[1:65].view(1, 64), w), "16-byte aligned"),
                         (lambda: lce.lce_linear(x.to(E4M3), w.to(E4M3), out_dtype=F32), "bf16 output"),
                         (lambda: lce.lce_linear_backward(torch.zeros(4, 7, device=DEV, dtype=BF16), x, w[:7]), "M must be")):
        with pytest.raises(lce.LCEError, match=needle) as e:
            call()
        assert e.value.status == lce.LCE_ERR_UNSUPPORTED
    for call in (lambda: lce.lce_linear(x.float(), w.float()), lambda: lce.lce_linear(x, w.to(E4M3)),
                 lambda: lce.lce_linear(x, w, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: lce.lce_linear(x, w, scale_x=torch.ones(4, device=DEV)),
                 lambda: lce.lce_linear(x, w, activation="tanh"),
                 lambda: lce.lce_linear_backward(torch.zeros(4, 8, device=DEV, dtype=BF16), x, w, activation="silu"),
                 lambda: lce.lce_linear(x, w, bias=torch.ones(7, device=DEV)),
                 lambda: lce.lce_linear(x, w, bias=torch.ones(9, device=DEV)),
                 lambda: lce.linear(x.clone().requires_grad_(), w[:7]),
                 lambda: lce.linear(x, w, residual=torch.ones(4, 7, device=DEV, dtype=BF16))):
        with pytest.raises(ValueError):
            call()
