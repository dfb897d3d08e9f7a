"""Which way a product with 8-bit weights is taken (no GPU)."""
import random

import pytest

from base8_plan import plan

KINDS = {256: (256, 1), 128: (128, 2), 96: (128, 2), 64: (64, 4), 48: (64, 4), 32: (32, 4)}    # columns: accumulator, k-blocks


def shapes(count=4000):
    r = random.Random(0)
    for _ in range(count):
        yield r.random() < 0.5, int(2 ** r.uniform(0, 22)), int(2 ** r.uniform(0, 22)), r.choice([152, 148, 20, 1]), r.choice([76, 74, 10, 0])


def test_every_plan_is_a_kernel_that_there_is():
    for back, m, n, sms, pairs in shapes():
        cg, bn, w, deep = plan(back, m, n, sms, pairs)
        assert (w, deep) == KINDS[bn] and cg in (1, 2)
        assert not (back and bn in (96, 48))                    # a copied piece is a whole swizzle span
        assert cg == 1 or (bn == 256 and pairs > 0 and m > 128)


def test_without_the_kernels_of_256_columns():
    for back, m, n, sms, pairs in shapes():
        cg, bn, w, deep = plan(back, m, n, sms, pairs, wide=False)
        assert cg == 1 and bn <= 128 and (w, deep) == KINDS[bn] and not (back and bn in (96, 48))


@pytest.mark.parametrize("m", [1, 33, 128])
@pytest.mark.parametrize("n,columns", [(4864, 32), (7000, 48), (9728, 64), (9800, 96), (12000, 96), (14592, 96), (14600, 128), (38912, 256)])
def test_few_rows_take_the_narrowest_tiles_that_one_round_holds(m, n, columns):
    assert plan(False, m, n)[:2] == (1, columns)
