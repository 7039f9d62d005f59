"""What the orthogonalised update keeps beyond fp16, on the GPU.

Gradients of few directions show it.  The other singular values are 0 and stay 0 by the definition; whatever the
roundings put there grows by 3.4445 a step, 485 times in five steps and 19800 times in eight.  Coefficients under which
values grow show that no step leaves fp16's range.

Tolerances.  ``ortho_model.rounded`` has the kernel's roundings (fp32 sums among them, in another order than the
kernel's) and is off from the definition by some dev; the kernel's deviation is of the same size and held to three
times that, besides the output's own rounding to bf16: 2^-8 of each value at most, and 2^-8 / sqrt(3) of the whole in the
Frobenius norm where the roundings fall evenly (a tenth more allowed for)."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import blocks_plans  # noqa: E402
import ortho_model as model  # noqa: E402
import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("r,c,rank", [(64, 64, 1), (40, 500, 1), (33, 20, 2), (256, 256, 1), (130, 300, 4), (300, 130, 4),
                                      (512, 1024, 1), (1024, 512, 16), (600, 700, 4), (1100, 2100, 2)])
def test_few_directions(r, c, rank, steps):
    G = model.matrix(r, c, r + c, rank, device=DEV)
    got = lce.lce_orthogonalise(G, steps=steps).double()
    want, like = model.defined(G, steps), model.rounded(G, steps)
    size = float(want.norm())
    dev = float((like - want).norm())
    limit = math.hypot(1.1 * 2.0 ** -8 / math.sqrt(3) * size, 3 * dev)
    off = float((got - want).norm())
    assert off <= limit, f"off by {off / size:.2e} of the result, limit {limit / size:.2e}"


@pytest.mark.parametrize("case", model.CASES)
def test_every_rounding_is_as_fine_as_stated(case):
    """The output's deviation from the model, along what a coarser rounding would change: 1 with that rounding, 0
    without."""
    G, steps = model.case_matrix(case).to(DEV), case[4]
    got = lce.lce_orthogonalise(G, steps=steps).double()
    for mutation in model.MUTATIONS:
        share = model.share_of(got, G, steps, mutation)
        if share is None:   # the product takes fp16's X alone
            assert mutation == "B X without the rest" and not model.takes_rest(min(G.shape), steps, model.ABC)
        else:
            assert abs(share) < 0.5, f"{share:.2f} of what {mutation!r} would change"


# (gradient, steps, coefficients), and the most that singular values make of X, A and B before the last step: 12, 144, 0;
# 16, 256, 0; 16, 256, 3.6e3; 150, 2.3e4, 0; 1, 1, 2e6; 6, 36, 1.4e3 (twice); 238, 5.7e4, 0; 238, 5.7e4, 2.2e6
GROWTH = [("ones 2 3", 2, (12.0, 0.0, 0.0)), ("ones 2 2", 3, (4.0, 0.0, 0.0)), ("ones 100 70", 2, (2.0, 14.0, 0.0)),
          ("directions 200 300", 5, (3.5, 0.0, 0.0)), ("directions 70 90", 1, (1e6, 1e6, 1e6)), ("directions 70 90", 2, (3.0, 2.0, 1.0)),
          ("noise 70 90", 2, (3.0, 2.0, 1.0)), ("noise 300 90", 4, (6.2, 0.0, 0.0)), ("diagonal 130 200", 2, (200.0, 38.0, 0.0))]


def growing(kind):
    name, r, c = kind.split()
    r, c = int(r), int(c)
    if name == "ones":
        return torch.ones(r, c, device=DEV)
    if name == "diagonal":   # one entry far above the others
        G = 1e-3 * torch.eye(r, c, device=DEV)
        G[3, 5] = 1.0
        return G
    return model.matrix(r, c, 9, 2 if name == "directions" else 0, device=DEV)


@pytest.mark.parametrize("kind,steps,abc", GROWTH)
def test_values_that_grow(kind, steps, abc):
    """Each value off by half a step of bf16 and three times the largest of the model's deviations; by 2^-20 of it
    besides, for a value next to the middle of a step that fp32's roundings move (two of each step's, 2^-24 each)."""
    G = growing(kind)
    got = lce.lce_orthogonalise(G, steps=steps, coefficients=abc).double()
    want, like = model.defined(G, steps, abc), model.rounded(G, steps, abc)
    limit = want.abs() * (2.0 ** -8 + 2.0 ** -20) + 3 * (like - want).abs().max()
    off = (got - want).abs()
    assert bool((off <= limit).all()), f"worst {float(off.max()):.3g} of {float(want.abs().max()):.3g}, limit {float(limit.max()):.3g}"


@pytest.mark.parametrize("steps", [2, 8])
@pytest.mark.parametrize("batch,r,c", blocks_plans.ORTHO_COVER)
def test_every_kernel_without_and_with_the_rest(batch, r, c, steps):
    """Two steps take fp16's X alone in B X from 65 rows on, eight the rest too."""
    assert not model.takes_rest(65, 2, model.ABC) and model.takes_rest(2007, 8, model.ABC)
    G = torch.stack([model.matrix(r, c, k, 3 * (k % 2), device=DEV) for k in range(batch)])
    got = lce.lce_orthogonalise(G, steps=steps).double()
    for k in {0, 1 % batch, batch - 1}:
        want, like = model.defined(G[k], steps), model.rounded(G[k], steps)
        limit = math.hypot(1.1 * 2.0 ** -8 / math.sqrt(3) * float(want.norm()), 3 * float((like - want).norm()))
        off = float((got[k] - want).norm())
        assert off <= limit, f"matrix {k}: {off:.3g} of {limit:.3g}"


@pytest.mark.parametrize("norm", [1e-7, 1e-9, 1e-12, 1e-14])
@pytest.mark.parametrize("r,c", [(60, 90), (300, 200)])
def test_gradients_next_to_eps_and_far_below(r, c, norm):
    G = model.matrix(r, c, 4, device=DEV)
    G = G * (norm / float(G.norm()))
    got = lce.lce_orthogonalise(G, eps=1e-7).double()
    want, like = model.defined(G), model.rounded(G)
    limit = want.abs() * (2.0 ** -8 + 2.0 ** -20) + 3 * (like - want).abs().max()
    assert bool(((got - want).abs() <= limit).all())
    if norm >= 1e-12:   # X's steps of 2^-38 are far below its values of norm / eps / sqrt(r c), 4e-8 at the least
        assert float((like - want).norm()) <= 2e-3 * float(want.norm())
