"""Calls of the operators for long contexts that lie beside those of the other files: page
selections that take every page, errors in each of its kernels, factors at the ends of the
exponents, borders between many scores."""
import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from rag_kv_cache_layer_gb300 import _lib as L
from test_gpu_paged import ints

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("n", [4, 10, 16])
def test_select_records_errors_whether_or_not_pages_are_scored(dt, n):
    """Sequences of ten pages, fewer picks than those, as many and more: where every page fits,
    only the last of the selection's kernels runs."""
    bounds, q = torch.zeros(20, 2, 64, dtype=dt, device="cuda"), torch.ones(3, 64, dtype=dt, device="cuda")
    table = ints([list(range(10)), list(range(10, 20))])

    def run(offsets, lens, **kw):
        picks = torch.full((3, 1, n), -5, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, ints(offsets), ints(lens), table, bounds, 8, 1, 1, 64, picks, **kw)
        torch.cuda.synchronize()
        return R.device_status(), picks[:, 0].tolist()
    bad, old = L.CB_ERR_DEVICE_INDEX, [-5] * n
    ok = {4: [0, 1, 2, 9], 10: list(range(10)), 16: list(range(10)) + [-1] * 6}[n]
    assert run([0, 1, 2], [80, 80]) == (0, [ok, ok, old])                   # padding behind the last row
    assert run([0, 1, 2], [80, 0]) == (0, [ok, [-1] * n, old])
    assert run([0, 1, 2], [80, 81]) == (bad, [ok, old, old])                # past the table
    assert run([0, 1, 2], [80, -1]) == (bad, [ok, old, old])
    assert run([0, 1, 2], [79, 80], max_kv_len=79) == (bad, [ok, old, old])
    assert run([0, 1, 9], [80, 80]) == (bad, [ok, old, old])
    assert run([0, 2, 1], [80, 80]) == (bad, [ok, ok, old])
    assert run([-1, 1, 2], [80, 80]) == (bad, [old, ok, old])
    # a page outside the pool is looked at where pages are scored
    table[0, 1] = 20
    assert run([0, 1, 2], [80, 80]) == ((bad, [[0, 2, 3, 9], ok, old]) if n == 4 else (0, [ok, ok, old]))
    table[0, 1] = -1
    assert run([0, 1, 2], [80, 80]) == ((bad, [[0, 2, 3, 9], ok, old]) if n == 4 else (0, [ok, ok, old]))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pages", [60, 9000])
def test_select_keeps_the_newest_pages_where_scores_are_not_finite(dt, pages):
    for what in ("q nan", "q inf", "bounds nan", "bounds inf", "overflow"):
        gen = torch.Generator(device="cuda").manual_seed(pages)
        bounds = torch.randn(pages, 1, 64, generator=gen, device="cuda").to(dt).repeat(1, 2, 1)
        q = torch.randn(1, 128, generator=gen, device="cuda").to(dt)
        if what[0] == "q":
            q[0, 5] = float(what[2:])
        elif what == "overflow":
            bounds, q = bounds * 3e38, q * 3e38
        else:
            bounds[::3, 1, 7] = float(what[7:])
        table = torch.randperm(pages, generator=gen, device="cuda").int()[None]
        picks = torch.full((1, 1, 20), -5, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, ints([0, 1]), ints([8 * pages]), table, bounds, 8, 2, 1, 64, picks, n_first=2, n_last=3)
        torch.cuda.synchronize()
        got = [j for j in picks.flatten().tolist() if j >= 0]
        assert {0, 1, *range(pages - 3, pages)} <= set(got) and len(set(got)) == len(got), (what, got)
        assert got == sorted(got) and got[-1] == pages - 1
    assert R.device_status() == 0
