"""Windows of the decode cache's attention: as large as an int32, and what lies below their start.

The pools, the 64-bit form and the derived tolerances are those of ``test_gpu_cache.Case``.
"""
import pytest

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(heads=1, queries=8, dim=128, pool="e4m3"),
                                dict(dim=576, queries=16), dict(dim=576, queries=16, block=5)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 4096])
def test_the_largest_windows_hide_nothing(kw, window):
    """Requests shorter than the newest tokens, where a 32-bit difference would not hold."""
    Case(81, [1, 2, 3, 4, 0, 300], new=4, **kw).attend(scale=0.1, window=window)
