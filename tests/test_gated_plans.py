"""Which kernels the gated and 8-bit integer operators run on, on the host: that the shapes of
tests/gated_plan.py reach every one of them, and that the launches of a call make up its product."""
import ctypes
import random

import pytest

import dense_blas3_gemm_amd as d
from gated_plan import FORMS, SHAPES, every_instance, instances, plan


@pytest.mark.parametrize("form", FORMS)
def test_every_kernel_has_a_shape(form):
    reached = set().union(*(instances(form, s) for s in SHAPES))
    assert reached == every_instance(form)


def test_launches_make_up_the_product():
    r = random.Random(0)
    for form in FORMS * 60:
        M, N, K = (max(1, int(2 ** r.uniform(0, e))) for e in (14, 14, 13))
        if r.random() < 0.5:
            N, K = (N + 15) // 16 * 16, (K + 15) // 16 * 16
        p = plan(*form, M, N, K, sums=r.random() < 0.5 and form[0] == "dgated", pad=r.choice([0, 1, 16]))
        assert sum(x.rows * x.cols for x in p) == M * N
        assert all(x.rows == M or x.cols == N // 16 * 16 or x.cols == N // 8 * 8 or x.cols == N for x in p)


def test_generic_launches_end():
    """2^32 threads are no launch: 8 columns to 256 threads of the kernel for few elements, 64 on tiles."""
    for op, kind in (("gated", "bf16"), ("dgated", "e4m3"), ("i8", "i8"), ("gated", "i8")):
        for M, N in ((1, 2 ** 27), (8, 2 ** 27 + 3), (1, 2 ** 31 - 1), (40, 2 ** 30 + 1), (3, 2 ** 26)):
            for tB in (0, 1):
                p = plan(op, kind, tB, M, N, 1)
                assert sum(x.cols for x in p) == N
                assert all(x.kernel.startswith("simt") and -(-x.cols // (8 if "thin" in x.kernel else 64)) * 256 < 2 ** 32
                           for x in p)
    # partial column sums, two sets of them, in 64 MiB
    for N in (2 ** 23 - 8, 2 ** 23, 2 ** 23 + 1, 2 ** 31 - 1):
        p = plan("dgated", "bf16", 0, 100, N, 1, sums=True)
        assert sum(x.cols for x in p) == N and all(2 * x.cols * 4 <= 64 << 20 for x in p)


def test_rows_in_blocks():
    """Offsets into A of 32 bits, and partial column sums that the workspace holds."""
    p = plan("i8", "i8", 1, 320000, 72, 16, pad=8176)
    assert len({x.rows for x in p}) > 1 and sum(x.rows * x.cols for x in p) == 320000 * 72
    assert all((x.rows + 256) * 8192 < 2 ** 31 for x in p)
    p = plan("dgated", "bf16", 1, 100100, 8203, 16, sums=True)
    assert sum(x.rows * x.cols for x in p) == 100100 * 8203 and p[-1] == ("simt_thin", 1, 100100, 3)
    assert len([x for x in p if x.cols == 8200]) > 1


def test_what_cannot_be():
    fn = d.load_library().dbgemm_gated_plan
    plan("i8", "i8", 0, 1, 1, 1)  # (sets the argument types)
    text = ctypes.create_string_buffer(8)
    assert fn(0, 2, 0, 1, 8, 16, 16, 8, 8, 0, 256, text, 8) == 1 and len(text.value) < 8
    assert fn(0, 2, 0, 0, 8, 16, 16, 8, 8, 0, 256, text, 8) == 1
    assert fn(0, 2, 0, 1, 8, 16, 16, 8, 8, 0, 256, None, 8) == 1
