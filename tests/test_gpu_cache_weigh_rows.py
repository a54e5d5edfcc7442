"""Weights of keys under numbers of rows that do not fill an instance, with scores of every form, against 64 bits."""
import pytest
import torch

from cache_more_case import More
from test_gpu_cache_scores import slopes_of
from test_gpu_cache_weigh import weigh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("queries, new", [(1, 1), (3, 1), (4, 1), (7, 1), (9, 1), (5, 3), (4, 5), (11, 3), (13, 5)])
def test_rows_beside_none(queries, new, pool):
    case = More(141, [200, 1, 0, 77], queries=queries, new=new, dim=64, pool=pool, block=32)
    for cap, slopes, window in ((0.0, None, 0), (5.0, None, 33), (0.0, "powers", 0), (5.0, "mixed", 2 ** 31 - 1)):
        weigh(case, cap=cap, slopes=slopes_of(case, slopes), window=window, add=window == 0)


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("queries, new", [(8, 1), (4, 4), (3, 1), (8, 8), (16, 9)])
def test_rows_whose_sum_is_none_give_nothing_whatever_they_hold(queries, new, pool):
    """Rows that a batch pads with: an lse of -infinity, and queries that may be anything."""
    case = More(142, [200, 90], queries=queries, new=new, dim=64, pool=pool, block=32)
    for cap in (0.0, 5.0):
        _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, cap=cap)
        good = lse.clone()
        lse[0, -1, 1], lse[1, 0, 0], lse[1, -1, queries - 1] = (-float("inf"),) * 3
        old = torch.rand((2, 1, 200), device="cuda")
        want = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone(), cap=cap)
        assert torch.isfinite(want).all()
        more = case.cache.weigh(0, case.q, good, case.dlen, case.dtable, old.clone(), cap=cap)
        assert ((more - want)[:, 0].sum(-1) - torch.tensor([1.0, 2.0], device="cuda")).abs().max() < 2.0 ** -8
        for odd in (float("nan"), float("inf"), -float("inf")):
            q = case.q.clone()
            q[0, -1, 1], q[1, 0, 0, ::2], q[1, -1, queries - 1, 5] = odd, odd, odd
            got = case.cache.weigh(0, q, lse, case.dlen, case.dtable, old.clone(), cap=cap)
            assert torch.equal(got, want)
        case.cache.check()
    if pool in ("bf16", "f16"):
        # a key that is no number reaches nothing through such rows alone
        case.dev[0, 0, int(case.table[0, 0]), 7, 0] = float("nan")
        lse[:] = -float("inf")
        assert torch.equal(case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone()), old)
