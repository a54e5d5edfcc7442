"""Windows of the decode cache's attention: as large as an int32, and what lies below their start.

The pools, the 64-bit form and the derived tolerances are those of ``test_gpu_cache.Case``.
"""
import pytest
import torch

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(heads=1, queries=8, dim=128, pool="e4m3"),
                                dict(dim=576, queries=16), dict(dim=576, queries=16, block=5)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 4096])
def test_the_largest_windows_hide_nothing(kw, window):
    """Requests shorter than the newest tokens, where a 32-bit difference would not hold."""
    Case(81, [1, 2, 3, 4, 0, 300], new=4, **kw).attend(scale=0.1, window=window)


def _evict(case, window):
    """What no newest token sees below the window: NaN in the pool, and -1 in the table for blocks of
    which nothing is seen."""
    B, table = case.B, case.table
    for r, n in enumerate(case.lengths):
        first = max(0, n - case.new + 1 - window)
        for k in range(-(-first // B)):
            held = min(B, first - k * B)
            case.dev[:, :, int(table[r, k]), :held] = 0x7F if case.pool_type == "e4m3" else float("nan")
            if held == B:
                table[r, k] = -1
    case.dtable.copy_(torch.from_numpy(table))


BELOW = [
    # lengths, kw, window
    ([90], dict(heads=1, queries=8, dim=128), 50),
    ([90, 260, 31, 0, 64], dict(heads=2, queries=8, dim=128), 1),
    ([90, 260, 31, 0, 64], dict(heads=2, queries=8, dim=128, new=4, block=8), 47),
    ([700, 333], dict(heads=1, queries=4, dim=64, pool="f16", block=1), 129),
    ([700, 333], dict(heads=1, queries=4, dim=64, pool="f16", block=5, new=2), 64),
    ([77, 200], dict(heads=2, queries=32, dim=256, block=64), 33),
    ([500, 130], dict(heads=1, queries=8, dim=128, new=4, block=32), 63),
    ([260, 33, 1], dict(heads=2, queries=8, dim=128, pool="e4m3", block=32), 100),
    ([260, 33, 1], dict(heads=2, queries=48, dim=256, pool="e4m3", block=3, new=2), 17),
    ([9000, 20, 4100], dict(heads=2, queries=8, dim=64, block=16), 3001),
    ([90], dict(dim=576, queries=16), 50),
    ([90, 260, 31, 0, 64], dict(dim=576, queries=16, block=8), 1),
    ([90, 260, 31, 0, 64], dict(dim=576, queries=8, new=3, block=16), 45),
    ([90, 260, 31, 0, 64], dict(dim=576, queries=8, new=3, block=5), 45),
    ([500, 129], dict(dim=576, queries=128, block=64), 97),
    ([500, 129], dict(dim=576, queries=40, pool="f16", block=128), 96),
    ([400, 300], dict(dim=576, queries=32, block=24, new=2), 33),
    ([9000, 20, 4100], dict(dim=576, queries=16, block=32), 3001),
]


@pytest.mark.parametrize("lengths, kw, window", BELOW)
def test_what_lies_below_a_window_is_neither_read_nor_looked_up(lengths, kw, window):
    """NaN next to the first key that is seen, in the same block and tile, and blocks that are gone
    from the table: results are those of the window alone and nothing is flagged."""
    case = Case(82, lengths, **kw)
    _evict(case, window)
    case.attend(scale=0.1, window=window)
