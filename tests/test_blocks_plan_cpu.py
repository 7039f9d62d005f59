"""The sizes that the GPU tests of the block-scaled product and of the orthogonalised update run take every
kernel that a size can."""
import shutil

import pytest

import blocks_plans

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    return blocks_plans.load(str(tmp_path_factory.mktemp("plans")))


@pytest.mark.parametrize("e8m0", [True, False])
def test_every_product_has_a_size(plans, e8m0):
    taken, whole = set(), set()
    for n, K, M in blocks_plans.COVER[e8m0]:
        shape, splits = plans[0](n, K, M, e8m0)
        taken.add((shape, K % 128 != 0, splits > 1))
        if "x" in shape:   # ends inside a tile both ways
            f, t = map(int, shape.split("x"))
            assert n % t and M % f, (n, K, M, shape)
            whole.add((shape, n > t and M > f))
        else:
            assert M % 16
    tiles = {(s, cut, split) for s in blocks_plans.SHAPES[:4] for cut in (False, True) for split in (False, True)}
    rows = {(s, cut, False) for s in blocks_plans.SHAPES[4:] for cut in (False, True)}
    assert taken == tiles | rows
    assert all((s, True) in whole for s in blocks_plans.SHAPES[:4])   # and has whole tiles before


def test_product_plans_are_within_their_limits(plans):
    for n in (1, 16, 17, 32, 33, 700, 9000):
        for K in (16, 400, 4096, 20000):
            for M in (1, 300, 8192, 202048):
                for e8m0 in (False, True):
                    shape, splits = plans[0](n, K, M, e8m0)
                    assert 1 <= splits <= 16 and (splits == 1 or -(-K // 128) // splits >= 3)
                    assert splits == 1 or shape not in blocks_plans.SHAPES[4:]
                    assert (shape != "16 tokens" or n <= 16) and (shape != "32 tokens" or 16 < n <= 32)


def test_every_update_has_a_size(plans):
    taken = {(k, *p) for size in blocks_plans.ORTHO_COVER for k, p in enumerate(plans[1](*size))}
    shapes = set(blocks_plans.ORTHO_SHAPES)
    tiles = shapes - {"32"}
    assert taken == {(k, s, False) for k in range(3) for s in (shapes if k else tiles)} | {(0, s, True) for s in tiles}
