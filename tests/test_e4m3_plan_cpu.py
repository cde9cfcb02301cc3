"""The choice of a kernel for an 8-bit product, on the host: the sizes that
stand for each kernel reach it, and every kernel that a call can reach stands
among them (the GPU tests compare each with 64 bits)."""
import pytest

import e4m3_cases as cases


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    return cases.Planner(str(tmp_path_factory.mktemp("plan")))


def test_names_are_the_planners(planner):
    assert [n for n, _ in planner.kernels()] == [*cases.TILES, *cases.SKINNY]


def test_cases_reach_their_kernels(planner):
    plans = planner.plans([(m, n, k, al, ws) for _, m, n, k, al, ws, _ in cases.CASES])
    for case, (kernel, splits, _) in zip(cases.CASES, plans):
        assert (kernel, splits) == (case[0], case[6]), case


def test_every_kernel_has_its_cases(planner):
    """Aligned and not, whole and split, with a last slice that is cut inside 16
    codes and fewer slices than stages."""
    for name, reg in planner.kernels():
        for aligned in (True, False) if reg else (True,):
            mine = [c for c in cases.CASES if c[0] == name and c[4] == aligned]
            assert mine, (name, aligned)
            if name in cases.SKINNY:
                continue
            ks = [c[3] for c in mine if c[6] == 1]
            assert any(c[6] > 1 for c in mine), (name, aligned, "no K split")
            assert any(k % 16 for k in ks), (name, aligned, "no ragged K")
            whole = cases.STAGES[name] * cases.SLICE[name]
            assert min(ks) <= cases.SLICE[name] and max(ks) > whole, (name, aligned, "slices")


def test_tiles_for_unaligned_rows(planner):
    """Rows that are not 16-byte aligned never get a kernel without a form for them."""
    reg = dict(planner.kernels())
    sizes = [(m, n, k, False, ws) for m in (1, 20, 64, 65, 1000, 5000, 20000) for n in (1, 100, 4100, 20000)
             for k in (1, 200, 4000) for ws in (False, True)]
    for s, (kernel, _, _) in zip(sizes, planner.plans(sizes)):
        assert reg[kernel], s
