"""The powers of two that fp16 holds the orthogonalised update's values times, and the coefficients that are refused."""
import shutil

import pytest

torch = pytest.importorskip("torch")

import blocks_plans  # noqa: E402
import ortho_model as model  # noqa: E402
import vocabulary_cross_entropy_row_amd as lce  # noqa: E402


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    return model.load(str(tmp_path_factory.mktemp("scales")))


@pytest.fixture(scope="module")
def chosen(plans):
    return plans[0]


COEFFICIENTS = [model.ABC, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (3.0, -3.2, 1.2), (4.0, 0.0, 0.0), (12.0, 0.0, 0.0), (0.0, 1.0, 0.0),
                (0.0, 0.0, 1.0), (1.0, 0.0, -3.0), (-2.0, 5.0, -2.5), (2.0, 14.0, 0.0), (3.0, 2.0, 1.0), (1e6, 1e6, 1e6), (0.0, 0.0, 0.0)]


@pytest.mark.parametrize("steps", [1, 2, 3, 5, 8, 100])
def test_kernel_and_model_choose_alike(chosen, steps):
    for abc in COEFFICIENTS:
        abc = tuple(torch.tensor(abc).float().tolist())
        for r in (1, 64, 65, 484, 485, 5000):
            got = chosen(r, steps, abc)
            if got is not None:
                assert got == (*model.scales(steps, abc), model.takes_rest(r, steps, abc)), (abc, r)


@pytest.mark.parametrize("seed", range(40))
def test_nothing_overflows(chosen, seed):
    """Matrices with singular values anywhere from 0 to 1, one of them the largest, under random coefficients."""
    g = torch.Generator().manual_seed(seed)
    abc = tuple((torch.randn(3, generator=g) * torch.tensor([3.0, 4.0, 2.0])).tolist())
    steps = 1 + seed % 4
    got = chosen(500, steps, abc)
    if got is None:
        assert max(value for value, _, _ in model.values(steps, abc)) > 250
        return
    x, o, b, _ = got
    for value, gram, poly in model.values(steps, abc):
        assert value * x < 65504 and gram * o < 65504 and poly * b < 65504


def call(steps, abc, batch=0):
    status = lce.lib().lce_orthogonalise(None, 70, 7000, lce.LCE_BF16, batch, 100, 70, steps, *abc, 1e-7, None, 70, 7000, None, 0, None)
    return status, lce.lce_last_error()


@pytest.mark.parametrize("steps,abc", [(3, (20.0, 0.0, 0.0)), (100, (1.2, 0.0, 0.0)), (3, (3.0, 2.0, 1.0)), (4, (0.0, 0.0, 5.0)), (1, (0.0, 1e31, 0.0)),
                                       (1, (1e31, 0.0, 0.0)), (100, (3e38, 3e38, 3e38)), (2, (300.0, 0.0, 0.0)), (2, (-300.0, 0.0, 0.0))])
def test_growth_past_the_limit_is_refused(steps, abc):
    for batch in (0, 1):
        status, message = call(steps, abc, batch)
        assert status == lce.LCE_ERR_UNSUPPORTED and "singular values past 256" in message, message


@pytest.mark.parametrize("steps,abc", [(100, model.ABC), (100, (1.5, -0.5, 0.0)), (100, (2.0, -1.5, 0.5)), (2, (250.0, 0.0, 0.0)), (1, (1e30, -1e30, 1e30)),
                                       (100, (1.0, 0.0, 0.0)), (3, (15.0, 0.0, 0.0)), (50, (0.0, 0.0, 0.0))])
def test_other_coefficients_are_not(steps, abc):
    assert call(steps, abc)[0] == lce.LCE_OK


def test_sizes_of_the_gpu_test_take_every_kernel(plans):
    """B X without the rest (two steps) and with it (eight) in every shape of tile."""
    sizes = [size for size in blocks_plans.ORTHO_COVER if min(size[1:]) > 64]
    for rest in (False, True):
        assert {plans[1](*size, rest) for size in sizes} == set(range(len(blocks_plans.ORTHO_SHAPES)))
    for size in sizes:
        assert [plans[0](min(size[1:]), steps, model.ABC)[3] for steps in (2, 8)] == [False, True]
