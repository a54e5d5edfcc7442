"""Block tables that are views of others: one row for all requests, rows that overlap, slices."""
import pytest
import torch

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu


def _views(row, R):
    """Tables of R rows whose entries are all in ``row``'s own tensor, and none beside it: the pool holds NaN
    in blocks that no request owns, and the entries beside a view's are no blocks."""
    width = row.numel()
    room = torch.full((R, 3 * width + 5), -7, dtype=torch.int32, device="cuda")
    room[:, width:2 * width] = row
    long = torch.cat([row, torch.full((1000,), -7, dtype=torch.int32, device="cuda")])
    return {"expanded": long[:width].expand(R, width), "sliced": room[:, width:2 * width],
            "every other row": room.repeat_interleave(2, 0)[::2, width:2 * width]}


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(heads=1, queries=8, dim=128, pool="e4m3"),
                                dict(dim=576, queries=16), dict(dim=576, queries=16, block=5)])
def test_requests_that_share_a_row(kw):
    one = Case(91, [700], max_requests=6, **kw)
    lengths, R = [700, 1, 0, 333, 699, 64], 6
    case = Case(91, [700], max_requests=R, **kw)
    case.lengths, case.table = lengths, case.table.repeat(R, 0)
    case.q = torch.randn((R,) + case.q.shape[1:], device="cuda").to(case.q.dtype)
    case.dlen = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    results = []
    for name, t in _views(one.dtable[0], R).items():
        case.dtable = t
        results.append(case.attend(scale=0.1))
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])


def test_rows_that_overlap():
    """Request r's blocks are those from entry r on of one list: a stride of one entry."""
    case = Case(92, [160], heads=2, queries=8, dim=64, block=16, max_requests=5)
    line = torch.full((1 << 12,), -7, dtype=torch.int32, device="cuda")
    line[:10] = case.dtable[0, :10]
    case.dtable = line.as_strided((5, 6), (1, 1))
    case.table = case.dtable.cpu().numpy()
    case.lengths = [96, 90, 1, 50, 96]
    case.dlen = torch.tensor(case.lengths, dtype=torch.int32, device="cuda")
    case.q = torch.randn((5,) + case.q.shape[1:], device="cuda").to(case.q.dtype)
    case.attend()


def test_append_through_a_shared_row():
    from prefill_decode_paged_gb300 import KVCache
    pool = torch.zeros((1, 2, 8, 4, 2, 32), dtype=torch.bfloat16, device="cuda")
    cache = KVCache(pool, num_layers=1, num_components=2, kv_heads=2, head_dim=32, block=4, num_blocks=8, dtype=1)
    row = torch.full((1 << 12,), 7, dtype=torch.int32, device="cuda")       # block 7 beside the row
    row[:3] = torch.tensor([5, 0, 2], dtype=torch.int32)
    k = torch.randn((6, 2, 32), device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    pos = [0, 11, 3, 8, 5, 6]
    cache.append(0, k, 2 * k, torch.arange(6, **i32), torch.tensor(pos, **i32), row[:3].expand(6, 3))
    cache.check()
    expect = torch.zeros_like(pool)
    for t, p in enumerate(pos):
        b = [5, 0, 2][p // 4]
        expect[0, 0, b, p % 4], expect[0, 1, b, p % 4] = k[t], 2 * k[t]
    assert torch.equal(pool, expect)
