"""The sizes that the GPU tests of the matrix product run take every kernel that a size can: each shape of
tile with whole and cut last steps of K, in one launch and split along K."""
import shutil

import pytest

import linear_plan

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return linear_plan.load(str(tmp_path_factory.mktemp("plan")))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_every_kernel_has_a_size(plan, dtype):
    taken, whole = set(), set()
    for n, K, M in linear_plan.COVER[dtype]:
        shape, splits = plan(n, K, M, dtype == "e4m3")
        taken.add((shape, K * (2 if dtype == "bf16" else 1) % 128 != 0, splits > 1))
        if "x" in shape:   # ends inside a tile both ways
            f, t = map(int, shape.split("x"))
            assert n % t and M % f, (n, K, M, shape)
            whole.add((shape, n > t and M > f))
    tiles = {(s, tail, split) for s in linear_plan.SHAPES[:4] for tail in (False, True) for split in (False, True)}
    rows = {(s, tail, False) for s in linear_plan.SHAPES[4:] for tail in (False, True)}
    assert taken == tiles | rows
    assert all((s, True) in whole for s in linear_plan.SHAPES[:4])   # and has whole tiles before


def test_plans_are_within_their_limits(plan):
    for n in (1, 16, 17, 32, 33, 700, 9000):
        for K in (16, 400, 4096, 20000):
            for M in (1, 300, 8192, 202048):
                for e4m3 in (False, True):
                    shape, splits = plan(n, K, M, e4m3)
                    assert 1 <= splits <= 16 and (splits == 1 or -(-K * (2 - e4m3) // 128) // splits >= 3)
                    assert splits == 1 or shape not in linear_plan.SHAPES[4:]
                    assert (shape != "16 tokens" or n <= 16) and (shape != "32 tokens" or 16 < n <= 32)
