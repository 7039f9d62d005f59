"""The quantiser into blocks of 128, the 8-bit product with a scale for each block, and its training form on
the GPU against the formulas in 64 bits.

Tolerances.  The quantiser's scales are powers of two, so x / scale is exact and each value is rounded
once: its outputs are held to equality.  The product: the 8-bit matrix instructions bring eight
neighbouring products to a unit of 2^-13 of the largest one's power of two and cut the rest off before
they add, so each of the other seven is off by less than 2^-13 of the group's largest (measured on the
device: beside +256 and -256 in one group of eight, 2^-5 is kept and 2^-6 is not; in another group 2^-9
is).  The groups' sums, the factors and the blocks' sums are fp32: at most (K + 8) 2^-24 of the sum of
magnitudes.  Activations' slopes are at most 1.13 and their own arithmetic is off by at most 2^-20
(|z| + 1); the store is off by half a step of bf16."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import blocks_plans  # noqa: E402
import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
U, HALF = 2.0 ** -24, torch.finfo(torch.bfloat16).eps / 2
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def normal(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device=DEV)


def within(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    bad = ~(off <= 0)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst by {float(off.max()):.3g}"


def spread(scale, n, K, tile):
    """A scale for each value."""
    s = scale.double().repeat_interleave(128, 1)[:, :K]
    return s.repeat_interleave(128, 0)[:n] if tile else s


def quantised(x, tile):
    """(values, scales) in 64 bits, by the definition."""
    n, K = x.shape
    rows = 128 if tile else 1
    v = x.double()
    pad = torch.nn.functional.pad(v.abs(), (0, -K % 128, 0, -n % rows))
    m = pad.view(pad.shape[0] // rows, rows, pad.shape[1] // 128, 128).amax((1, 3))
    e = torch.frexp(m / 448)[1].double()   # m / 448 < 2^e, and 2^(e - 1) <= m / 448
    e = torch.where(m == 448 * torch.exp2(e - 1), e - 1, e)
    s = torch.where(m == 0, torch.ones_like(m), torch.exp2(e).clamp_min(2.0 ** -126))
    u = v / spread(s, n, K, tile)
    step = torch.exp2(torch.frexp(u)[1].clamp_min(-5).double() - 4)
    return torch.round(u / step) * step, s


def check_quantiser(x, blocks, transposed, scale_dtype=None, **kw):
    got = lce.lce_quantize_blocks(x, blocks=blocks, transposed=transposed, scale_dtype=scale_dtype, **kw)
    for want, m, v, s in ((blocks, x, got.values, got.scale), (transposed, x.t(), got.values_t, got.scale_t)):
        if want is None:
            assert v is None and s is None
            continue
        qv, qs = quantised(m, want == "tile")
        assert s.dtype == (scale_dtype or E8M0) and s.shape == qs.shape and v.dtype == E4M3
        assert torch.equal(s.double(), qs), (want, "scale")
        assert torch.equal(v.double(), qv), (want, "values")
    return got


SHAPES = [(1, 1), (1, 128), (3, 127), (2, 129), (16, 6656), (127, 64), (128, 128), (129, 300), (300, 1001), (1, 4099),
          (4099, 1), (515, 2056), (1000, 128)]
KINDS = [("row", None), ("tile", None), ("row", "row"), ("row", "tile"), ("tile", "tile"), ("tile", "row"), (None, "row"),
         (None, "tile")]


@pytest.mark.parametrize("n,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantiser(n, K, dtype):
    r = normal(n * 7 + K)
    x = (r(n, K) * torch.exp2(4 * r(n, 1)) * torch.exp2(3 * r(1, K))).to(dtype)
    for blocks, transposed in KINDS:
        check_quantiser(x, blocks, transposed, F32 if (n + K) % 2 else None)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantiser_extremes(dtype):
    r = normal(3)
    x = r(130, 520).to(dtype)
    x[0] = 0                                     # blocks of zeros
    x[1, :128] = 448                             # on the border
    x[2, :128] = torch.finfo(dtype).max
    x[3, :128] = torch.finfo(dtype).tiny
    x[4, :128] = torch.finfo(dtype).smallest_normal / 4   # below the normal numbers
    x[5, :128] *= 2.0 ** -120
    x[6, 128:256] = torch.tensor(448.0).to(dtype).item() * 1.0078125   # just above the border, in bf16 too
    x[7, :128] = -0.0
    x[8, :128] = 0
    x[8, 5] = -7e-6
    for blocks, transposed in KINDS:
        check_quantiser(x[:, :128], blocks, transposed)
        check_quantiser(x, blocks, transposed)


def test_quantiser_marks_infinities_and_nans_in_their_blocks_alone():
    r = normal(4)
    x = r(300, 400)
    x[5, 130], x[7, 3], x[200, 390] = math.inf, math.nan, -math.inf
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    for blocks, transposed in KINDS:
        got = lce.lce_quantize_blocks(x, blocks=blocks, transposed=transposed)
        for want, m, c, v, s in ((blocks, x, clean, got.values, got.scale),
                                 (transposed, x.t(), clean.t(), got.values_t, got.scale_t)):
            if want is None:
                continue
            qv, qs = quantised(c, want == "tile")
            hit = spread(quantised(torch.isfinite(m).logical_not().float(), want == "tile")[1], *m.shape, want == "tile") != 1
            assert bool(torch.isnan(v.double()[hit]).all()) and torch.equal(v.double()[~hit], qv[~hit])
            each = spread(s, *m.shape, want == "tile")
            assert torch.equal(torch.isnan(each), hit)


def test_quantiser_strides_and_given_outputs():
    r = normal(5)
    wide = r(200, 900)
    x = wide[3:160, 5:620]   # rows off 16 bytes
    check_quantiser(x, "row", "tile")
    n, K = x.shape
    for shift, ldv in ((0, 640), (1, 617), (8, 632)):
        hold = torch.zeros(n * ldv + 64, dtype=torch.uint8, device=DEV).view(E4M3)
        hold_t = torch.zeros(K * 171 + 64, dtype=torch.uint8, device=DEV).view(E4M3)
        v = torch.as_strided(hold, (n, K), (ldv, 1), shift)
        vt = torch.as_strided(hold_t, (K, n), (171, 1), shift)
        scale = torch.full((n, 9), 7.0, device=DEV)[:, 2:7]
        scale_t = torch.full((2, K + 3), 7.0, device=DEV)[:, :K].t()
        got = check_quantiser(x, "row", "row", F32, values=v, values_t=vt, scale=scale, scale_t=scale_t)
        assert got.values is v and got.scale is scale
        outside = torch.ones(hold.numel(), dtype=torch.bool, device=DEV)
        torch.as_strided(outside, (n, K), (ldv, 1), shift).fill_(False)
        assert not bool(hold.view(torch.uint8)[outside].any())   # between the rows, as it was


def operands(n, K, M, seed, power):
    """Quantised x and weight; without ``power``, scales of any value."""
    r = normal(seed)
    x, w = r(n, K), r(M, K) / math.sqrt(K)
    x = x * torch.exp2(2 * r(1, K))
    qx = lce.lce_quantize_blocks(x, scale_dtype=E8M0 if power else F32)
    qw = lce.lce_quantize_blocks(w, blocks="tile", scale_dtype=E8M0 if power else F32)
    sx, sw = qx.scale, qw.scale
    if not power:
        sx, sw = sx * (0.5 + r(*sx.shape).abs()), sw * (0.5 + r(*sw.shape).abs())
    return qx.values, sx, qw.values, sw


def stands_for(q, s, tile):
    return q.double() * spread(s, *q.shape, tile)


def cut_off(x, w):
    """Bound on what the 8-bit products lose: 7 2^-13 of each group's largest, summed over the groups."""
    n, K = x.shape
    x, w = (torch.nn.functional.pad(t.float().abs(), (0, -K % 8)) for t in (x, w))
    K = x.shape[1]
    rows = max(1, (1 << 27) // (w.shape[0] * K))
    parts = [(x[i:i + rows, None] * w[None]).view(-1, w.shape[0], K // 8, 8).amax(3).sum(2) for i in range(0, n, rows)]
    return 7 * 2.0 ** -13 * torch.cat(parts).double()


def act_of(kind, z):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2)),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
            "silu": lambda: z * torch.sigmoid(z)}[kind]()


def check_product(x, sx, w, sw, *, act="none", bias=None, residual=None, preact=False):
    xd, wd = stands_for(x, sx, False), stands_for(w, sw, True)
    K = x.shape[1]
    got = lce.lce_linear_blocks(x, sx, w, sw, bias=bias, activation=act, residual=residual, want_preact=preact)
    z, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    err = (K + 8) * U * size + cut_off(xd, wd)
    if preact:
        within(got.preact, z, HALF * z.abs() + err, "preact")
    y = act_of(act, z)
    tol = 1.13 * err + (0 if act in ("none", "relu") else 2.0 ** -20) * (z.abs() + 1)
    if residual is not None:
        y = y + residual.double()
        tol = tol + 2 * U * (y.abs() + residual.double().abs())
    within(got.out, y, HALF * y.abs() + tol, "out")
    return got


SIZES = [(1, 1, 1), (1, 64, 256), (2, 4096, 512), (3, 72, 7), (5, 1000, 33), (16, 6656, 1000), (17, 520, 129),
         (32, 2048, 4099), (31, 1001, 300), (33, 128, 127), (64, 4096, 256), (65, 264, 1000), (100, 640, 2049),
         (129, 1024, 128), (128, 8192, 640), (255, 200, 511), (300, 1003, 1003), (513, 512, 1025), (1000, 136, 2000),
         (1030, 2048, 4100), (2048, 512, 8192)]


@pytest.mark.parametrize("n,K,M", SIZES)
@pytest.mark.parametrize("power", [True, False], ids=["e8m0", "f32"])
def test_product(n, K, M, power):
    x, sx, w, sw = operands(n, K, M, n + K + M, power)
    check_product(x, sx, w, sw)
    r = normal(n * 3 + M)
    check_product(x, sx, w, sw, act=ACTS[(n + M) % 5], bias=r(M).to(BF16 if n % 2 else F32), residual=r(n, M).to(BF16),
                  preact=True)
    if not power:   # one side's scales in a byte
        check_product(x, sx, w, lce.lce_quantize_blocks(stands_for(w, sw, True).float(), blocks="tile").scale)


@pytest.mark.parametrize("power,n,K,M", [(p, *size) for p in (True, False) for size in blocks_plans.COVER[p]])
def test_every_kernel_of_the_product(power, n, K, M):
    x, sx, w, sw = operands(n, K, M, n + K + M, power)
    r = normal(n * 5 + M)
    check_product(x, sx, w, sw, act=ACTS[(n + M) % 5], bias=r(M).to(F32 if n % 2 else BF16),
                  residual=r(n, M).to(BF16) if K % 2 else None)


@pytest.mark.parametrize("power", [True, False], ids=["e8m0", "f32"])
@pytest.mark.parametrize("n", [7, 40, 400])
def test_what_lies_past_the_width_does_not_matter(n, power):
    """Rows whose bytes past K are NaN, and scales in either order."""
    K, M = 201, 170
    x, sx, w, sw = operands(n, K, M, 11, power)
    want = check_product(x, sx, w, sw).out
    for ld in (208, 256, 400):
        px, pw = (torch.full((rows, ld), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3)[:, :K] for rows in (n, M))
        px.view(torch.uint8).copy_(x.view(torch.uint8))
        pw.view(torch.uint8).copy_(w.view(torch.uint8))
        other = sx.contiguous() if sx.stride(1) != 1 else sx.t().contiguous().t()
        assert torch.equal(lce.lce_linear_blocks(px, other, pw, sw.t().contiguous().t()).out, want)


@pytest.mark.parametrize("power", [True, False], ids=["e8m0", "f32"])
@pytest.mark.parametrize("n", [9, 40, 300])
def test_scales_far_from_one(n, power):
    """Each pair's product near 1, the scales themselves 2^100 and 2^-100; and pairs whose products differ by 2^60."""
    x, sx, w, sw = operands(n, 300, 260, n, power)
    for up in (100, -100):
        bx, bw = (t.float() * 2.0 ** e for t, e in ((sx, up), (sw, -up)))
        check_product(x, bx.to(sx.dtype), w, bw.to(sw.dtype))
    steps = torch.tensor([0.0, 60.0, -60.0], device=DEV)
    check_product(x, (sx.float() * torch.exp2(steps)).to(sx.dtype), w, sw)
    check_product(x, sx, w, (sw.float() * torch.exp2(-steps)).to(sw.dtype))


def test_a_nan_scale_reaches_its_rows_alone():
    for power in (True, False):
        for n in (9, 200):
            x, sx, w, sw = operands(n, 300, 260, 5, power)
            clean = lce.lce_linear_blocks(x, sx, w, sw).out
            sx, sw = sx.clone(), sw.clone()
            sx.view(torch.uint8 if power else F32)[3, 1] = 255 if power else math.nan
            sw.view(torch.uint8 if power else F32)[1, 0] = 255 if power else math.nan
            got = lce.lce_linear_blocks(x, sx, w, sw).out
            hit = torch.zeros_like(got, dtype=torch.bool)
            hit[3], hit[:, 128:256] = True, True
            assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], clean[~hit])


def test_one_residual_in_place_and_another_stream():
    x, sx, w, sw = operands(130, 700, 390, 6, True)
    res = normal(1)(130, 390).to(BF16)
    want = lce.lce_linear_blocks(x, sx, w, sw, residual=res).out
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = res.clone()
    torch.cuda.synchronize()
    got = lce.lce_linear_blocks(x, sx, w, sw, residual=out, out=out, stream=st).out
    st.synchronize()
    assert got is out and torch.equal(got, want)


# ---- training form -----------------------------------------------------------------------------

def check_training(n, K, M, seed, *, bias=None, residual=False, lead=None):
    r = normal(seed)
    x = (r(n, K) * torch.exp2(r(1, K))).to(BF16)
    w = (r(M, K) / math.sqrt(K)).to(BF16)
    g = (1e-3 * r(n, M)).to(BF16)
    b = None if bias is None else r(M).to(bias).requires_grad_()
    res = r(n, M).to(BF16).requires_grad_() if residual else None
    xl = (x if lead is None else x.view(*lead, K)).clone().requires_grad_()
    wl = w.clone().requires_grad_()
    y = lce.linear_blocks(xl, wl, b, residual=None if res is None else (res if lead is None else res.view(*lead, M)))
    assert y.shape == (*xl.shape[:-1], M)
    leaves = [t for t in (xl, wl, b, res) if t is not None]
    grads = dict(zip([k for k, t in (("x", xl), ("w", wl), ("b", b), ("r", res)) if t is not None],
                     torch.autograd.grad(y, leaves, g.view(y.shape))))
    qx, sx = quantised(x, False)
    qw, sw = quantised(w, True)
    xd, wd = qx * spread(sx, n, K, False), qw * spread(sw, M, K, True)

    def product(a, c, length, got, what, more=None):
        z, size = a @ c.t(), a.abs() @ c.abs().t()
        if more is not None:
            z, size = z + more.double(), size + more.double().abs()
        within(got, z, HALF * z.abs() + (length + 8) * U * size + cut_off(a, c), what)

    more = None if b is None else b.detach().double().expand(n, M)
    if res is not None:
        more = res.detach().double() + (0 if more is None else more)
    product(xd, wd, K, y.detach().view(n, M), "y", more)
    gq, gs = quantised(g, False)
    product(gq * spread(gs, n, M, False), wd.t().contiguous(), M, grads["x"].view(n, K), "grad_x")
    gq, gs = quantised(g.t(), False)
    xq, xs = quantised(x.t(), True)
    product(gq * spread(gs, M, n, False), xq * spread(xs, K, n, True), n, grads["w"], "grad_weight")
    if b is not None:
        s = g.double().sum(0)
        half = torch.finfo(bias).eps / 2
        within(grads["b"], s, half * s.abs() + (n + 8) * U * g.double().abs().sum(0), "grad_bias")
    if res is not None:
        assert torch.equal(grads["r"], g)


@pytest.mark.parametrize("n,K,M", [(1, 1, 1), (1, 300, 130), (7, 129, 1000), (40, 1001, 77), (128, 256, 384),
                                   (300, 515, 1030), (517, 1001, 2051), (1030, 1024, 2048)])
def test_training(n, K, M):
    check_training(n, K, M, n + K, bias=BF16 if n % 2 else F32, residual=n % 3 == 0)


def test_training_with_leading_dimensions_and_expanded_gradients():
    check_training(24, 160, 96, 9, lead=(2, 3, 4), bias=F32)
    x = normal(1)(6, 64).to(BF16).requires_grad_()
    w = normal(2)(32, 64).to(BF16)
    y = lce.linear_blocks(x, w)
    y.float().sum().backward()   # an upstream gradient of one value, expanded
    got = x.grad.clone()
    x.grad = None
    lce.linear_blocks(x, w).backward(torch.ones(6, 32, dtype=BF16, device=DEV))
    assert torch.equal(got, x.grad)


def test_training_without_tokens_and_without_gradients():
    x = torch.empty(0, 40, dtype=BF16, device=DEV, requires_grad=True)
    w, b = (normal(1)(24, 40).to(BF16).requires_grad_(), torch.ones(24, device=DEV, requires_grad=True))
    y = lce.linear_blocks(x, w, b)
    gx, gw, gb = torch.autograd.grad(y, (x, w, b), torch.empty(0, 24, dtype=BF16, device=DEV))
    assert y.shape == (0, 24) and gx.shape == (0, 40) and not bool(gw.any()) and not bool(gb.any())
    full = normal(2)(5, 40).to(BF16)
    with torch.no_grad():
        assert not lce.linear_blocks(full, w, b).requires_grad
    (only,) = torch.autograd.grad(lce.linear_blocks(full, w.detach(), b), (b,), torch.ones(5, 24, dtype=BF16, device=DEV))
    assert torch.equal(only, torch.full((24,), 5.0, device=DEV))


def test_gradients_against_differences():
    """Along the direction of the gradient, where the roundings average out: the quantised products are
    linear in their inputs up to a relative rounding of 2^-4 of each of K values, which for the sum's
    difference over steps of a tenth leaves (K = 512 values and 64 x 96 outputs) well under 5%."""
    r = normal(21)
    x, w = r(64, 512).to(BF16), (r(96, 512) / math.sqrt(512)).to(BF16)
    g = r(64, 96).to(BF16)
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    gx, gw = torch.autograd.grad(lce.linear_blocks(xl, wl), (xl, wl), g)
    for leaf, grad in ((0, gx), (1, gw)):
        t = (x, w)[leaf].double()
        d = grad.double() * (0.1 * t.norm() / grad.double().norm())
        ends = [[x, w] for _ in range(2)]
        for k, sign in ((0, 1), (1, -1)):
            ends[k][leaf] = (t + sign * d).to(BF16)
        step = (ends[0][leaf].double() - ends[1][leaf].double())
        up, down = (lce.linear_blocks(*e).double() for e in ends)
        found, told = float(((up - down) * g.double()).sum()), float((step * grad.double()).sum())
        assert abs(found - told) <= 0.05 * abs(told), (found, told)


def test_captured_training_step_replays():
    r = normal(31)
    x, w = r(200, 256).to(BF16), (r(384, 256) / 16).to(BF16)
    g = r(200, 384).to(BF16)
    xs = x.clone().requires_grad_()
    ws = w.clone().requires_grad_()

    def step():
        y = lce.linear_blocks(xs, ws)
        return (y, *torch.autograd.grad(y, (xs, ws), g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        with torch.no_grad():
            xs.copy_(r(200, 256).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in held]
        xe, we = xs.detach().clone().requires_grad_(), w.clone().requires_grad_()
        y = lce.linear_blocks(xe, we)
        want = (y.detach(), *torch.autograd.grad(y, (xe, we), g))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del y


def test_same_bits_again():
    x, sx, w, sw = operands(700, 4096, 500, 8, False)
    a = lce.lce_linear_blocks(x, sx, w, sw).out
    assert torch.equal(a, lce.lce_linear_blocks(x, sx, w, sw).out)


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 values, its transpose and the products that read and write as much."""
    r = normal(41)
    n, K = 70001, 61504
    x = torch.empty(n, K, dtype=BF16, device=DEV)
    for i in range(0, n, 10000):
        x[i:i + 10000] = r(min(10000, n - i), 1).to(BF16) * r(1, K).to(BF16)
    got = lce.lce_quantize_blocks(x, blocks="row", transposed="tile")
    for rows in (slice(0, 128), slice(69888, n)):   # whole blocks of rows
        qv, qs = quantised(x[rows], False)
        assert torch.equal(got.scale[rows].double(), qs) and torch.equal(got.values[rows].double(), qv)
        for cols in (slice(0, 256), slice(61440, K)):
            qv, qs = quantised(x[rows, cols].t(), True)
            at = slice(cols.start // 128, -(-cols.stop // 128)), slice(rows.start // 128, -(-rows.stop // 128))
            assert torch.equal(got.scale_t[at].double(), qs) and torch.equal(got.values_t[cols, rows].double(), qv)
    # as the weight: [K, n] in tiles, against few rows of x
    few = lce.lce_quantize_blocks(r(3, n))
    out = lce.lce_linear_blocks(few.values, few.scale, got.values_t, got.scale_t).out
    for cols in (slice(0, 128), slice(61440, K)):
        at = slice(cols.start // 128, -(-cols.stop // 128))
        a, b = stands_for(few.values, few.scale, False), stands_for(got.values_t[cols], got.scale_t[at], True)
        z = a @ b.t()
        within(out[:, cols], z, HALF * z.abs() + (n + 8) * U * (a.abs() @ b.abs().t()) + cut_off(a, b), "weight past 2^32")
    # as x, and an output of more than 2^32 values
    M = 61457
    w = lce.lce_quantize_blocks(r(M, 128), blocks="tile")
    narrow = torch.as_strided(got.values, (n, 128), got.values.stride()), got.scale[:, :1]
    out = lce.lce_linear_blocks(*narrow, w.values, w.scale).out
    for rows in (slice(0, 64), slice(n - 64, n)):
        a = stands_for(narrow[0][rows], narrow[1][rows], False)
        b = stands_for(w.values, w.scale, True)
        z = a @ b.t()
        within(out[rows], z, HALF * z.abs() + 136 * U * (a.abs() @ b.abs().t()) + cut_off(a, b), "output past 2^32")


def test_calls_at_once_with_their_own_workspaces():
    """Two streams, each with split products, and two captured graphs that share one workspace in turn."""
    cases = [operands(34, 1286, 72, s, True) for s in (1, 2)]
    want = [lce.lce_linear_blocks(*c).out for c in cases]
    assert lce.lce_linear_blocks_workspace_bytes(34, 1286, 72) > 0
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[lce.lce_linear_blocks(*c, stream=st).out for c, st in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))
    ws = torch.empty(lce.lce_linear_blocks_workspace_bytes(34, 1286, 72), dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.empty_like(w) for w in want], [torch.cuda.CUDAGraph() for _ in cases]
    for g, c, o in zip(graphs, cases, outs):
        with torch.cuda.graph(g):
            lce.lce_linear_blocks(*c, out=o, workspace=ws)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for o in outs:
            o.zero_()


def test_rows_behind_the_last_are_left():
    x, sx, w, sw = operands(40, 300, 72, 3, True)
    out = torch.full((60, 80), 7.0, dtype=BF16, device=DEV)
    lce.lce_linear_blocks(x, sx, w, sw, out=out[:40, :72])
    assert bool((out[40:] == 7).all()) and bool((out[:, 72:] == 7).all())
    assert torch.equal(out[:40, :72], lce.lce_linear_blocks(x, sx, w, sw).out)


def test_no_rows():
    x = torch.empty(0, 300, device=DEV)
    got = lce.lce_quantize_blocks(x, blocks="row", transposed="tile")
    assert got.values.shape == (0, 300) and got.scale.shape == (0, 3) and got.values_t.shape == (300, 0) and got.scale_t.shape == (3, 0)
    w = lce.lce_quantize_blocks(normal(1)(40, 300), blocks="tile")
    assert lce.lce_linear_blocks(got.values, got.scale, w.values, w.scale).out.shape == (0, 40)
    assert lce.lce_orthogonalise(torch.empty(0, 8, 8, device=DEV)).shape == (0, 8, 8)


@pytest.mark.parametrize("n,K", [(1, 130), (130, 1), (1, 1)])
def test_single_rows_and_columns_with_odd_strides(n, K):
    """A single row or column may have any stride; the operands that come of it are read as they lie."""
    x = torch.as_strided(normal(6)(4000), (n, K), (1 if n == 1 else 7 + K, 1 if K > 1 else 3))
    got = check_quantiser(x, "row", "tile")
    w = lce.lce_quantize_blocks(normal(7)(20, K), blocks="tile")
    check_product(got.values, got.scale, w.values, w.scale)
    wide = torch.zeros(n, 256, dtype=torch.uint8, device=DEV).view(E4M3)[:, :K]
    wide.view(torch.uint8).copy_(got.values.view(torch.uint8))
    assert torch.equal(lce.lce_linear_blocks(wide, got.scale, w.values, w.scale).out,
                       lce.lce_linear_blocks(got.values, got.scale, w.values, w.scale).out)
