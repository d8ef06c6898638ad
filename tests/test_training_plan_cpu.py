"""The sizes that the GPU tests of the grouped products run reach every kernel their
plans choose, and each what it is there for."""
import pytest

pytest.importorskip("dense_fp16_gemm_02_amd")

import grouped_cases as cases  # noqa: E402


@pytest.mark.parametrize("case", cases.GROUPED, ids=str)
def test_cases_take_their_plans(case):
    assert cases.plans(*case[:4]) == case[4:]


@pytest.mark.parametrize("case", cases.LONG, ids=str)
def test_long_cases_take_their_plans(case):
    assert cases.plans(*case[:4])[2] == case[4]


def test_every_kernel_is_run():
    seen = {name.split()[-1] for case in cases.GROUPED for name in case[4:]} | {case[4] for case in cases.LONG}
    assert seen == cases.KERNELS
    words = {w for case in cases.GROUPED for name in case[4:] for w in name.split()}
    assert {"pack_a", "pack_b"} <= words


def test_no_other_kernel_is_planned():
    """Over the sizes of a grid, aligned and not."""
    seen = set()
    for M in (1, 3, 17, 70, 300, 1000, 3000, 9000, 30000, 200000):
        for E in (1, 2, 8, 60, 300):
            for N in (8, 72, 200, 1000, 4096, 14336):
                for K in (8, 72, 200, 1000, 4096, 14336):
                    seen.update(name.split()[-1] for name in cases.plans(M, E, N, K))
    assert seen <= cases.KERNELS and len(seen) >= 25
