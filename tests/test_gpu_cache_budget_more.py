"""More of the calls that a decode under a budget may make: bad blocks among whole tiles, windows that begin with a
tile, most requests, one scale a plane, latents' positions of rotation, tables with rows apart."""
import numpy as np
import pytest
import torch

import cache_more_ref as ref
from cache_more_case import More
from prefill_decode_paged_gb300 import KVCache, KVRelayoutError, rotary_table
from test_gpu_cache_evict import Pool
from test_gpu_cache_weigh import check as check_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool, new", [("e2m1", 1), ("e2m1", 5), ("e4m3", 1), ("e4m3", 5), ("bf16", 5)])
@pytest.mark.parametrize("block", [32, 64, 96])
def test_bad_blocks_among_whole_tiles(pool, new, block):
    """Blocks of whole tiles, one of them out of range: its keys and values count as zeros, the rest as ever."""
    case = More(121, [300, 70, 200], heads=2, queries=16, dim=128, block=block, new=new, pool=pool)
    table = case.dtable.clone()
    for r, k, bad in ((0, 1, case.N), (2, 0, -1), (1, 0, 2 ** 31 - 1)):
        table[r, k] = bad
        case.wide[0, :, case.table[r, k]] = 0.0
    out, lse = case.cache.attend(0, case.q, case.dlen, table, scale=0.1, cap=6.0)
    with pytest.raises(KVRelayoutError, match="block id"):
        case.cache.check()
    case.check_scored(out, lse, 0.1, cap=6.0)
    old = torch.rand((3, 2, 300), device="cuda")
    w = case.cache.weigh(0, case.q, lse, case.dlen, table, old.clone(), scale=0.1, cap=6.0)
    with pytest.raises(KVRelayoutError, match="block id"):
        case.cache.check()
    check_weights(case, w, old, lse, 0.1, cap=6.0)


@pytest.mark.parametrize("pool", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("new, window", [(1, 64), (1, 96), (5, 60), (5, 92), (5, 200)])
def test_windows_that_begin_with_a_tile(pool, new, window):
    """Lengths and windows by which the first key seen is a multiple of 32, or one away from it."""
    lengths = [window + 32 * k + new - 1 + d for k in (1, 4) for d in (-1, 0, 1)]
    case = More(122, lengths, heads=1, queries=8, dim=128, block=32, new=new, pool=pool)
    out, lse = case.attend_scored(window=window, scale=0.1)
    old = torch.rand((len(lengths), 1, max(lengths)), device="cuda")
    for add in (True, False):
        w = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone(), add=add, scale=0.1, window=window)
        case.cache.check()
        check_weights(case, w, old, lse, 0.1, window, add=add)


def test_most_requests_of_one_call():
    lengths = [(7 * r) % 5 for r in range(2048)]
    for pool in ("bf16", "e2m1"):
        case = More(123, lengths, heads=1, queries=1, dim=64, block=4, pool=pool)
        _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
        old = torch.rand((2048, 1, 5), device="cuda")
        w = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
        case.cache.check()
        check_weights(case, w, old, lse, 0.125)
    Pool(124, lengths, 2, heads=1, dim=16, block=4).evict(1, False)
    Pool(125, lengths, 2, heads=1, dim=64, block=4, pool="e2m1").evict(1, True)
    torch.cuda.empty_cache()


def test_one_scale_a_plane():
    """A 4-bit pool with scales [L][C], appended, read and attended."""
    N, B, H, D, n = 6, 16, 2, 64, 80
    scales = np.array([[0.7, 2.5]], dtype=np.float32)
    pool = torch.zeros(2 * N * B * H * D * 9 // 16, dtype=torch.uint8, device="cuda")
    gen = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((n, H, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((1, 4, D), generator=gen, device="cuda").bfloat16()
    req, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.tensor([[5, 0, 3, 1, 2, 4]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    with KVCache(pool, num_layers=1, num_components=2, kv_heads=H, head_dim=D, block=B, num_blocks=N, dtype=5,
                 scales=scales, query_heads=4) as cache:
        cache.append(0, k, v, req, pos, table)
        got = cache.read(0, req, pos, table, dtype=torch.float16)
        out, lse = cache.attend(0, q, lens, table)
        cache.check()
    wide = []
    for x, s, g in zip((k, v), scales[0], got):
        c, b = ref.quantize(x.float().cpu().numpy(), s)
        wide.append(ref.values(c, b) * np.float64(s))
        want = torch.from_numpy((ref.values(c, b).astype(np.float32) * s)).to(torch.float16)
        assert torch.equal(g.cpu(), want)
    want = ref.attend(q.double().cpu().numpy()[:, None], lambda r, g, j: (wide[0][j, g // 2], wide[1][j, g // 2]), [n],
                      D ** -0.5)
    off = np.abs(out.double().cpu().numpy()[:, None] - want["out"])
    # one rounding of the output, the weights as f16, and fp32 scores
    assert (off <= 2.0 ** -8 * np.abs(want["out"]) + (2.0 ** -10 + 2 * want["off"][..., None] + n * 2.0 ** -22) *
            want["size"] + 2.0 ** -35 * want["total"]).all()


@pytest.mark.parametrize("tokens", [3, 700])
def test_latents_positions_of_rotation(tokens):
    """576-element rows whose last 64 are turned by other positions than their places."""
    gen = torch.Generator("cuda").manual_seed(6)
    k, q = torch.randn((tokens, 1, 576), generator=gen, device="cuda").bfloat16(), \
        torch.randn((tokens, 16, 64), generator=gen, device="cuda").bfloat16()
    at, angles = (torch.randperm(1000, generator=gen, device="cuda")[:tokens].to(torch.int32) for _ in range(2))
    req = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    table = torch.arange(63, dtype=torch.int32, device="cuda")[None].contiguous()
    kw = dict(rotary=torch.from_numpy(rotary_table(1000, 64)).cuda(), q=q, interleaved=True, rotate_last=True)
    pools = [torch.zeros((1, 1, 63, 16, 1, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    geometry = dict(num_layers=1, num_components=1, kv_heads=1, head_dim=576, block=16, num_blocks=63, dtype=1)
    with KVCache(pools[0], **geometry) as one, KVCache(pools[1], **geometry) as two:
        a = one.append(0, k, None, req, angles, table, **kw)
        b = two.append(0, k, None, req, at, table, angles=angles, **kw)
        one.check()
        two.check()
        x, none = two.read(0, req, at, table)
    assert torch.equal(a, b) and none is None
    assert torch.equal(pools[0].view(-1, 576)[angles.long()], pools[1].view(-1, 576)[at.long()])
    assert torch.equal(x[:, 0], pools[1].view(-1, 576)[at.long()])


def test_tables_whose_rows_are_apart_or_overlap():
    case = More(126, [90, 33], heads=2, queries=4, dim=64, pool="e2m1")
    room = torch.full((2, 40), -9, dtype=torch.int32, device="cuda")
    table = room[:, 3:3 + case.dtable.shape[1]]
    table.copy_(case.dtable)
    out, lse = case.cache.attend(0, case.q, case.dlen, table)
    w = case.cache.weigh(0, case.q, lse, case.dlen, table, torch.zeros((2, 2, 90), device="cuda"))
    case.cache.check()
    case.check_scored(out, lse, 0.125)
    check_weights(case, w, torch.zeros((2, 2, 90), device="cuda"), lse, 0.125)
    kept, slots = case.cache.evict(0, w.clone(), case.dlen, table, 40, 8)
    case.cache.check()
    req = torch.tensor([0] * 40 + [1] * 33, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(40), torch.arange(33)]).to(torch.int32).cuda()
    keys, _ = case.cache.read(0, req, pos, table)
    for r, n in enumerate((40, 33)):
        for h in range(2):
            j = ref.kept_slots(w[r, h].cpu().numpy(), case.lengths[r], 40, 8)
            assert slots[r, h, :n].tolist() == j
            want = case.wide[0, 0, case.table[r, np.array(j) // 16], np.array(j) % 16, h]
            got = keys[40 * r:40 * r + n, h].double().cpu().numpy()
            assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want)).all()
    assert (room[:, :3] == -9).all() and (room[:, 3 + table.shape[1]:] == -9).all()
