"""Calls on weights, evictions and reads that the cache refuses, and that leave everything as it was."""
import pytest
import torch

from test_gpu_cache_evict import Pool

pytestmark = pytest.mark.gpu


def test_a_table_without_blocks_is_no_eviction_in_place():
    case = Pool(131, [100, 90], 40)
    w = case.weights()
    before = w.clone()
    for into in (case.dtables[1][:, :0], torch.empty((2, 0), dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError, match="without blocks"):
            case.cache.evict(0, w, case.dlen, case.dtables[0], 40, 10, into=into)
    case.cache.check()
    assert torch.equal(case.dev, case.first) and torch.equal(w, before)
    # of no requests nothing is asked
    case.cache.evict(0, w[:0], case.dlen[:0], case.dtables[0][:0], 40, 10, into=case.dtables[1][:0])
    case.cache.check()
