"""Batch plans over arrays that a decode loop keeps, for more requests than one block of threads counts:
the lengths are read and written in place while kernels before and after the sums count and push the
pages of ended requests."""
import numpy as np
import pytest

from tests.test_gpu_attn import L  # noqa: F401
from tests.test_gpu_cache8 import run_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1024, 1025, 2500])
@pytest.mark.parametrize("wild", [False, True])
def test_plans_in_place(L, n, wild):
    rng = np.random.default_rng(n)
    cached = rng.integers(0, 300, n)
    # (with pages missing in the rows, requests either end or begin: a row in a missing page is an error)
    cached[rng.random(n) < 0.5] = 0
    new = np.where(rng.random(n) < 0.4, -1, np.where(cached == 0, rng.integers(0, 40, n), 0 if wild else rng.integers(0, 9, n)))
    shared = np.minimum(rng.integers(0, 4, n), -(-cached // 16))
    need = sum(max(-(-(c + x) // 16) - -(-c // 16), 0) for c, x in zip(cached, np.maximum(new, 0)))
    got = run_plan(L, rng, n, 16, 25, int(np.maximum(new, 0).sum()) + 3, cached, new, shared, wild=wild, in_place=True,
                   spare=need + 2)
    assert int(got.n_free[0]) >= 2


def test_rows_of_a_plan_without_a_number_of_rows(L):
    """T left out: the rows of the plan that is given, else none, which is reported."""
    import torch
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    table, free = torch.full((1, 3), -1, dtype=torch.int32, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")
    ws = L.batch_plan_workspace(1)
    got = L.batch_plan_t(table, one - 1, one * 4, free, one * 5, 16, 5, ws, out=L.BatchPlan.empty(1, 4))
    assert L.get_error_t(ws) == 0 and got.kv_len.tolist() == [4] and got.slots.tolist() == [64, 65, 66, 67]
    got = L.batch_plan_t(table, one - 1, one * 4, free, one * 5, 16, 5, ws)
    assert L.get_error_t(ws) == L.DEVERR_BAD_LEN and got.kv_len.tolist() == [0] and got.slots.numel() == 0
