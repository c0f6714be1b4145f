"""The choice of kernels on a device of fewer CUs (a partition of the card): a CU of it has the work that one of
a larger device has on as many times the columns, so it is given the same kernel."""
import random

import pytest

from gated_plan import FORMS, plan


def pairs(form, cus, rows):
    """(launch on `cus` CUs, launch on 256 of as many times the columns) of drawn products."""
    r = random.Random(cus)
    for _ in range(300):
        M, n, K = r.randint(*rows), int(2 ** r.uniform(0, 5)), int(2 ** r.uniform(5, 13)) // 16 * 16
        N = 256 * n  # (whole tiles and widths, so that their numbers are in the CUs' ratio)
        small, large = plan(*form, M, N, K, cus=cus), plan(*form, M, N * (256 // cus), K)
        if len(small) == len(large) == 1 and small[0].splits == large[0].splits == 1:
            yield (M, N, K), small[0].kernel, large[0].kernel


@pytest.mark.parametrize("cus", [32, 64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_widths_of_few_rows(form, cus):
    n = 0
    for shape, small, large in pairs(form, cus, (1, 64)):
        if small.startswith("few_rows") and large.startswith("few_rows"):
            assert small == large, shape
            n += 1
    assert n >= 20


@pytest.mark.parametrize("cus", [32, 64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_tiles(form, cus):
    """(few rows too, where tiles are given to them; splits and second launches pass the memory that all CUs share)"""
    n = 0
    for rows in ((1, 64), (65, 600)):
        for shape, small, large in pairs(form, cus, rows):
            if not small.startswith("few_rows") and not large.startswith("few_rows"):
                assert small == large, shape
                n += 1
    assert n >= 20
