"""What the orthogonalised update keeps beyond fp16, on the GPU.

Gradients of few directions show it.  The other singular values are 0 and stay 0 by the definition; whatever the
roundings put there grows by 3.4445 a step, 485 times in five steps and 19800 times in eight.

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
@pytest.mark.parametrize("mutation", model.MUTATIONS)
def test_every_rounding_is_as_fine_as_stated(case, mutation):
    """The output's deviation from the model, along what a coarser rounding would change: 1 with that rounding, 0
    without."""
    G = model.case_matrix(case).to(DEV)
    share = model.share_of(lce.lce_orthogonalise(G, steps=case[4]).double(), G, case[4], mutation)
    if share is None:
        pytest.skip("the product does not take the rest at this size")
    assert abs(share) < 0.5, f"{share:.2f} of what {mutation!r} would change"
