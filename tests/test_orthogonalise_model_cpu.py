"""What include/lce.h says of the orthogonalised update's error holds of the definition with the kernel's roundings, and
the GPU tests' comparison with it would notice each of them made coarser."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

import ortho_model as model  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FROBENIUS, SPECTRAL, SMALL = 1.4e-3, 1.9e-3, 6e-3   # of the result; from 64 rows on, and below in either norm
KINDS = ["noise", "uneven", "1", "2", "4", "16", "falling"]


def gradient(kind, r, c, seed):
    if kind in ("noise", "uneven"):
        return model.matrix(r, c, seed, uneven=kind == "uneven")
    if kind == "falling":   # singular values 1, 1/2, 1/3, ...
        u, s, v = torch.linalg.svd(model.matrix(r, c, seed).double(), full_matrices=False)
        return ((u / torch.arange(1, len(s) + 1)) @ v).float()
    return model.matrix(r, c, seed, int(kind))


def errors(G, steps=5):
    want = model.defined(G, steps)
    off = model.rounded(G, steps) - want
    return float(off.norm() / want.norm()), float(torch.linalg.matrix_norm(off, 2) / torch.linalg.matrix_norm(want, 2))


def test_header_states_these_numbers():
    with open(os.path.join(ROOT, "include", "lce.h")) as f:
        text = re.sub(r"\s+\*?\s*", " ", f.read())
    assert ("up to 1.4e-3 of it (Frobenius norm; 2-norm 1.9e-3) before it is rounded to bf16, matrices of few directions included, "
            "and by up to 6e-3 below 64 rows") in text


@pytest.mark.parametrize("kind", KINDS)
def test_stated_error_from_64_rows_on(kind):
    for r, c in ((64, 64), (65, 66), (64, 1024), (200, 90), (256, 256), (300, 800), (484, 500), (485, 500), (512, 1024)):
        frobenius, spectral = errors(gradient(kind, r, c, r + c))
        assert frobenius <= FROBENIUS and spectral <= SPECTRAL, (r, c, frobenius, spectral)


@pytest.mark.parametrize("kind", KINDS)
def test_stated_error_below(kind):
    for r, c in ((1, 300), (2, 3), (3, 6), (5, 8), (16, 16), (33, 20), (48, 51), (63, 252)):
        if kind.isdigit() and int(kind) >= min(r, c):
            continue
        for seed in range(5):
            assert max(errors(gradient(kind, r, c, seed))) <= SMALL, (r, c, seed)


@pytest.mark.parametrize("steps", [8, 10])
@pytest.mark.parametrize("r,c", [(64, 64), (64, 1024), (256, 256), (512, 600)])
def test_more_steps_are_as_exact_as_products_in_32_bits(r, c, steps):
    """Of gradients of few directions, besides what five steps may be off by (with a third more for the roundings that
    differ, of which there are as many)."""
    for rank in (1, 2, 8):
        G = model.matrix(r, c, 5, rank)
        want = model.defined(G, steps)
        plain = float((model.defined(G, steps, dtype=torch.float32) - want).norm() / want.norm())
        assert errors(G, steps)[0] <= 4 / 3 * plain + FROBENIUS, (rank, plain)


@pytest.mark.parametrize("case", model.CASES)
def test_a_coarser_rounding_is_noticed(case):
    """Of an output in bf16, as test_gpu_orthogonalise_precision.py compares it: nearer to the model that it came from
    than to the other, for each."""
    G, steps = model.case_matrix(case), case[4]
    like = model.rounded(G, steps).bfloat16().double()
    for mutation in model.MUTATIONS:
        share = model.share_of(like, G, steps, mutation)
        if share is None:
            assert mutation == "B X without the rest" and not model.takes_rest(min(G.shape), steps, model.ABC)
            continue
        other = model.share_of(model.rounded(G, steps, mutation=mutation).bfloat16().double(), G, steps, mutation)
        assert abs(share) < 0.25 and abs(other - 1) < 0.25, (mutation, share, other)
