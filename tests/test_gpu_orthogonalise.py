"""The orthogonalised update on the GPU against its definition in 64 bits.

Tolerances.  The same recursion with the kernel's roundings put in (X as fp16 and what that leaves in e4m3,
the operand the former; the diagonals of A and B kept, the rest in fp16), in 64 bits otherwise, is off from the definition by some
`dev` that the matrix's own spectrum decides.  The kernel rounds at the same places, so its deviation is of
the same size; sums in another order and values next to a rounding's border change which way single
roundings go, not how large they are.  It is held to three times dev in the 2-norm, and each
value to three times the largest of dev's.  (Not to eight times its root mean square, the bound first
tried, which holds for independent normal values only.  The deviation lies along the few singular
directions that the steps amplify most, sum_k d_k u_k v_k^T.  The product of two normal values passes t
times its root mean square with probability about sqrt(2 / (pi t)) e^-t: one of 530 thousand is expected
to pass 11.6, where e^-11.6 sqrt(0.055) 5.3e5 = 1.1, and 9.3 was met.)  All this besides the
output's own rounding: half a step of bf16, 2^-8, for each value, whose 2-norm is at most 2^-8 / sqrt(3)
of the result's where the roundings fall evenly (a tenth more is allowed for, and for few values the
bound itself)."""
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
BF16, F32 = torch.bfloat16, torch.float32
ABC = (3.4445, -4.7750, 2.0315)


def defined(G, steps=5, abc=ABC, eps=1e-7):
    a, b, c = abc
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    X = X / (X.norm() + eps)
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    return X.t() if tall else X


def rounded(G, steps=5, abc=ABC, eps=1e-7):
    """The definition with the kernel's roundings."""
    a, b, c = abc
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    X = X / (X.norm() + eps)
    S = 2.0 ** round(0.5 * math.log2(X.shape[1]))

    def half(v, s):
        return (v * s).half().double() / s

    for _ in range(steps):
        hi = half(X, S)
        up = 2.0 ** 19 / S
        X = hi + ((X - hi) * S * up).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() / up / S
        A = hi @ hi.t()
        D = A.diagonal().clone()
        O = half(A - torch.diag(D), 1024.0)
        B = b * O + c * (O @ O + (D[:, None] + D[None, :]) * O)
        E = b * D + c * ((O @ O).diagonal() + D * D)
        X = (a + E)[:, None] * X + half(B - torch.diag(B.diagonal()), 256.0) @ hi
    return X.t() if tall else X


def check(G, got, what="", **kw):
    want, model = defined(G, **kw), rounded(G, **kw)
    off = got.double() - want
    dev = float((model - want).norm())
    size = want.numel()
    assert got.dtype == BF16 and got.shape == G.shape
    each = want.abs() * 2.0 ** -8 + 3 * max(float((model - want).abs().max()), 2.0 ** -22)
    assert bool((off.abs() <= each).all()), f"{what}: worst by {float((off.abs() - each).max()):.3g}"
    share = 1.1 / math.sqrt(3) if size >= 4096 else 1.0
    limit = math.hypot(2.0 ** -8 * share * float(want.norm()), 3 * dev)
    assert float(off.norm()) <= limit, f"{what}: {float(off.norm()):.3g} of {limit:.3g}"


def matrix(r, c, seed, kind="noise"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    G = torch.randn(r, c, generator=g, device=DEV)
    if kind == "signal":   # a few strong directions over noise
        k = max(1, min(r, c) // 16)
        G = 0.2 * G + torch.randn(r, k, generator=g, device=DEV) @ torch.randn(k, c, generator=g, device=DEV)
    return 1e-3 * G


SIZES = [(1, 1), (1, 300), (300, 1), (2, 3), (5, 64), (64, 64), (65, 64), (63, 65), (100, 257), (513, 130), (256, 1024),
         (130, 4100), (1003, 517), (512, 4096), (700, 9000), (1500, 1400), (2305, 2049)]


@pytest.mark.parametrize("r,c", SIZES)
@pytest.mark.parametrize("kind", ["noise", "signal"])
def test_against_the_definition(r, c, kind):
    for dtype in (BF16, F32):
        G = matrix(r, c, r + c, kind).to(dtype)
        check(G, lce.lce_orthogonalise(G), f"{dtype}")


@pytest.mark.parametrize("batch,r,c", [(1, 70, 90), (3, 100, 40), (16, 64, 128), (5, 257, 300), (70, 33, 20)])
def test_batches(batch, r, c):
    G = torch.stack([matrix(r, c, 7 * k, "signal") * 10.0 ** k for k in range(min(batch, 5))] * -(-batch // 5))[:batch]
    got = lce.lce_orthogonalise(G)
    for k in range(batch):
        check(G[k], got[k], f"matrix {k}")


@pytest.mark.parametrize("batch,r,c", blocks_plans.ORTHO_COVER)
def test_every_kernel(batch, r, c):
    G = torch.stack([matrix(r, c, 5 * k, "signal" if k % 2 else "noise") for k in range(batch)])
    got = lce.lce_orthogonalise(G)
    for k in range(batch):
        check(G[k], got[k], f"matrix {k}")


@pytest.mark.parametrize("r,c", [(64, 4000), (1, 5000), (40, 70), (33, 65), (2900, 17), (64, 64), (32, 256), (48, 20000)])
def test_up_to_64_rows(r, c):
    for kind in ("noise", "signal"):
        G = matrix(r, c, 3 * r + c, kind)
        check(G, lce.lce_orthogonalise(G), kind)


def test_offsets_past_32_bits():
    G = torch.empty(33000, 128, 1024, dtype=BF16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    for part in G.split(3000):
        part.normal_(generator=g)
    got = lce.lce_orthogonalise(G)
    for k in (0, 16383, 16384, 32767, 32768, 32999):
        check(G[k], got[k], f"matrix {k}")


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, (1.5, -0.5, 0.0)), (8, ABC), (3, (2.0, -1.5, 0.5)), (12, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(steps, abc):
    G = matrix(200, 300, 3)
    check(G, lce.lce_orthogonalise(G, steps=steps, coefficients=abc), steps=steps, abc=abc)


def test_strides_and_given_output():
    hold = torch.randn(3, 120, 400, device=DEV)
    G = hold[:, 7:110, 5:322]
    place = torch.zeros(3, 130, 350, dtype=BF16, device=DEV)
    out = place[:, 3:106, 9:326]
    got = lce.lce_orthogonalise(G, out=out)
    assert got is out
    for k in range(3):
        check(G[k], out[k])
    outside = torch.ones_like(place, dtype=torch.bool)
    outside[:, 3:106, 9:326] = False
    assert not bool(place[outside].any())   # around the output, as it was
    expanded = hold[:1, :50, :60].expand(4, 50, 60)   # one matrix for the whole batch
    got = lce.lce_orthogonalise(expanded)
    for k in range(4):
        assert torch.equal(got[k], got[0])
    flat = torch.as_strided(torch.zeros(60 * 200, dtype=BF16, device=DEV), (4, 50, 50), (50, 200, 1))   # side by side
    lce.lce_orthogonalise(hold[0, :50, :50].expand(4, 50, 50), out=flat)
    check(hold[0, :50, :50], flat[2])


def test_zeros_and_values_that_are_no_numbers():
    G = torch.stack([matrix(90, 70, k) for k in range(5)])
    clean = lce.lce_orthogonalise(G)
    G[1] = 0
    G[2, 5, 6] = math.nan
    G[3, 8, 1] = -math.inf
    got = lce.lce_orthogonalise(G)
    assert not bool(got[1].any()) and bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[3]).all())
    assert torch.equal(got[0], clean[0]) and torch.equal(got[4], clean[4])


@pytest.mark.parametrize("scale", [1e-40, 1e-30, 1e-12, 1e30, 5e37])
def test_scale_of_the_gradient(scale):
    G = matrix(80, 100, 4).double() * scale * 1e3
    G = G.float()
    check(G, lce.lce_orthogonalise(G, eps=0.0), eps=0.0)


def test_singular_values():
    G = torch.randn(300, 500, device=DEV)
    s = torch.linalg.svdvals(lce.lce_orthogonalise(G).double())
    assert 0.65 < float(s.min()) and float(s.max()) < 1.25, (float(s.min()), float(s.max()))


def test_single_entries_and_orthogonal_rows():
    G = torch.zeros(70, 200, device=DEV)
    G[3, 150] = 2.0
    check(G, lce.lce_orthogonalise(G))
    check(torch.eye(130, 130, device=DEV), lce.lce_orthogonalise(torch.eye(130, device=DEV)))
    same = torch.ones(100, 65, device=DEV)   # one direction
    check(same, lce.lce_orthogonalise(same))


def test_same_bits_and_another_stream():
    G = matrix(600, 900, 8, "signal")
    want = lce.lce_orthogonalise(G)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = lce.lce_orthogonalise(G, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_captured_and_replayed():
    G = matrix(300, 200, 9)
    out = torch.empty(300, 200, dtype=BF16, device=DEV)
    lce.lce_orthogonalise(G, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lce.lce_orthogonalise(G, out=out)
    for k in range(3):
        G.copy_(matrix(300, 200, 20 + k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lce.lce_orthogonalise(G))


def test_training_step_with_an_orthogonalised_update():
    """The operators as they are used together: a product with its gradients in 8 bits, the momentum's
    orthogonalised update, and the updated weight quantised for serving."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(256, 192, generator=g, device=DEV).to(BF16)
    w = (torch.randn(320, 192, generator=g, device=DEV) / 14).to(BF16).requires_grad_()
    b = torch.zeros(320, device=DEV, requires_grad=True)
    labels = torch.randint(0, 320, (256,), generator=g, device=DEV)
    momentum = torch.zeros(320, 192, device=DEV)
    for _ in range(2):
        y = lce.linear_blocks(x, w, b)
        loss = lce.cross_entropy(y, labels)[0]   # its gradient replaces y
        gw, gb = torch.autograd.grad(loss, (w, b))
        momentum.mul_(0.95).add_(gw.float())
        update = lce.lce_orthogonalise(momentum)
        check(momentum, update)
        with torch.no_grad():
            w.add_(update, alpha=-0.02)
    held = lce.lce_quantize_blocks(w.detach(), blocks="tile")
    q = lce.lce_quantize_blocks(x)
    served = lce.lce_linear_blocks(q.values, q.scale, held.values, held.scale, bias=b.detach()).out
    assert torch.equal(served, lce.linear_blocks(x, w, b).detach())   # the training form's own forward
