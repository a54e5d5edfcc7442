"""Waits at the ends of the latents' kernel, for parts of every number of tiles."""
import pytest

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [32, 5])
def test_no_wait_runs_out_whatever_a_parts_tiles_are(block):
    """160 requests of t tiles each: parts of about 2 t tiles, so that every barrier ends in every phase.
    A wait that runs out is flagged, and check() raises."""
    for t in list(range(1, 13)) + [27]:
        case = Case(101, [32 * t - (r % 3 == 1) for r in range(160)], dim=576, queries=4, block=block)
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1)
        case.cache.check()
        case.check(out[:3], lse[:3], 0.1, 0, first=3)
        one = case.cache.attend(0, case.q[:1], case.dlen[:1], case.dtable[:1], scale=0.1)
        case.cache.check()
        case.check(one[0], one[1], 0.1, 0, first=1)
