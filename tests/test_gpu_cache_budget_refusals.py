"""Calls on weights, evictions and reads that the cache refuses, and that leave everything as it was."""
import pytest
import torch

from prefill_decode_paged_gb300 import KVRelayoutError
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


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "e2m1"])
def test_read_into_rows_that_overlap(pool):
    case = Pool(132, [30], 10, pool=pool)
    one = torch.zeros(5, dtype=torch.int32, device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    whole = torch.full((5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    other = whole.clone()
    for bad in (whole[:, :1].expand(5, 2, 64), whole[:1].expand(5, 2, 64), whole[:1, :1].expand(5, 2, 64)):
        for kw in (dict(k=bad, v=other), dict(k=other, v=bad)):
            with pytest.raises(KVRelayoutError, match="OVERLAP"):
                case.cache.read(0, one, pos, case.dtables[0], **kw)
    case.cache.check()
    assert (whole == 7.0).all() and (other == 7.0).all()
    # keys and values side by side, heads before tokens
    want = case.cache.read(0, one, pos, case.dtables[0])
    both = torch.zeros((5, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    turned = torch.zeros((2, 2, 5, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(k=both[:, 0], v=both[:, 1]), dict(k=turned[0].transpose(0, 1), v=turned[1].transpose(0, 1))):
        for a, b in zip(case.cache.read(0, one, pos, case.dtables[0], **kw), want):
            assert torch.equal(a.contiguous().view(torch.int16), b.view(torch.int16))
    case.cache.check()


def test_arguments_of_another_form_are_refused_as_such():
    """A tensor that does not fit is a ValueError, what the library refuses a KVRelayoutError, and neither is torch's own."""
    case = Pool(133, [30], 10)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    for bad in (pos.view(2, 3), pos[0], pos.long(), pos[::2], pos.cpu()):
        with pytest.raises(ValueError, match="positions"):
            case.cache.read(0, pos, bad, case.dtables[0])
    with pytest.raises(ValueError, match="requests"):
        case.cache.read(0, pos[:5], pos, case.dtables[0])
    w = case.weights()
    for keep in (0, -1, -2 ** 31):
        with pytest.raises(KVRelayoutError, match="INVALID"):
            case.cache.evict(0, w, case.dlen, case.dtables[0], keep)
    assert torch.equal(case.dev, case.first)
