"""Weights of keys under numbers of rows that do not fill an instance, with scores of every form, against 64 bits."""
import pytest

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
