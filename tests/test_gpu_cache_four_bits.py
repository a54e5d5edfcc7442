"""Pools of 4 bits on the GPU: append and read bit for bit by the header's definition, attention against 64 bits."""
import numpy as np
import pytest
import torch

import cache_more_ref as ref
from cache_more_case import More, torch_type
from prefill_decode_paged_gb300 import KVCache, KVRelayoutError, rotary_table

pytestmark = pytest.mark.gpu


def _pool(N, B, H, D, fill=0):
    return torch.full((2 * N * B * H * (D // 2 + D // 16),), fill, dtype=torch.uint8, device="cuda")


def _views(pool, N, B, H, D):
    n = 2 * N * B * H * (D // 2)
    host = pool.cpu().numpy()
    return host[:n].reshape(2, N, B, H, D // 2), host[n:].reshape(2, N, B, H, D // 16)


def _tokens(rng, tokens, R, width, B):
    """Distinct slots of random requests."""
    flat = rng.permutation(R * width * B)[:tokens]
    return (flat // (width * B)).astype(np.int32), (flat % (width * B)).astype(np.int32)


APPEND = [
    # heads, queries, dim, rotated, interleaved, last, type, block, tokens
    (1, 0, 64, 0, False, False, "bf16", 1, 1), (2, 4, 64, 64, False, False, "bf16", 16, 3),
    (8, 32, 128, 128, False, False, "bf16", 32, 1), (8, 32, 128, 128, True, False, "f16", 32, 70),
    (3, 6, 192, 96, False, True, "bf16", 5, 40), (3, 3, 192, 96, True, True, "f16", 24, 40),
    (2, 4, 256, 64, False, False, "f16", 16, 33), (1, 16, 256, 256, False, False, "bf16", 7, 500),
    (4, 8, 128, 32, True, False, "bf16", 16, 2000), (2, 64, 128, 64, False, True, "bf16", 16, 9),
]


@pytest.mark.parametrize("heads, queries, dim, rotated, interleaved, last, kind, block, tokens", APPEND)
def test_append_is_the_definition_bit_for_bit(heads, queries, dim, rotated, interleaved, last, kind, block, tokens):
    rng = np.random.default_rng(41)
    R, width = 5, max(2, -(-tokens // (4 * block)))
    N = R * width + 2
    table = rng.permutation(N)[:R * width].reshape(R, width).astype(np.int32)
    requests, positions = _tokens(rng, tokens, R, width, block)
    angles = rng.integers(0, 999, tokens).astype(np.int32)
    rows = 1000
    spread = np.exp(rng.standard_normal((tokens, heads, 1)) * 2)
    k, v = (torch.from_numpy(rng.standard_normal((tokens, heads, dim)) * spread).to(torch_type(kind)).cuda()
            for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((tokens, queries, dim))).to(torch_type(kind)).cuda() if queries else None
    rot = rotary_table(rows, rotated) if rotated else None
    scales = rng.uniform(0.3, 3.0, (1, 2, heads)).astype(np.float32)
    pool = _pool(N, block, heads, dim, 0x5A)
    with KVCache(pool, num_layers=1, num_components=2, kv_heads=heads, head_dim=dim, block=block, num_blocks=N,
                 dtype=5, scales=scales, per_head=True) as cache:
        dev = [torch.from_numpy(x).cuda() for x in (requests, positions, table, angles)]
        kw = dict(rotary=None if rot is None else torch.from_numpy(rot).cuda(), interleaved=interleaved,
                  rotate_last=last, q=q, angles=dev[3])
        q_out = cache.append(0, k, v, *dev[:3], **kw)
        got_k, got_v = cache.read(0, *dev[:3], dtype=torch_type(kind))
        cache.check()
    codes, block_scales = _views(pool, N, block, heads, dim)
    want_c, want_s = np.full_like(codes, 0x5A), np.full_like(block_scales, 0x5A)
    at = table[requests, positions // block], positions % block
    back = []
    for comp, x in enumerate((k, v)):
        x = x.float().cpu().numpy()
        if comp == 0 and rot is not None:
            x = ref.rotate32(x, angles, rot, rotated, interleaved, last)
        both = []
        for h in range(heads):
            c, s = ref.quantize(x[:, h], scales[0, comp, h])
            want_c[comp][at[0], at[1], h], want_s[comp][at[0], at[1], h] = c, s
            # code * block scale is exact in fp32, its product with s one rounding, to 16 bits another
            both.append(ref.values(c, s).astype(np.float32) * scales[0, comp, h])
        back.append(torch.from_numpy(np.stack(both, 1)).to(torch_type(kind)))
    np.testing.assert_array_equal(block_scales, want_s)
    np.testing.assert_array_equal(codes, want_c)
    assert torch.equal(got_k.cpu(), back[0]) and torch.equal(got_v.cpu(), back[1])
    # the values themselves: half a step of the code, and half a step of the block scale where it clips 6
    x = v.double().cpu().numpy()
    top = np.abs(x).reshape(tokens, heads, -1, 16).max(-1).repeat(16, -1)
    s64 = scales[0, 1].astype(np.float64)[:, None]
    # b is within r = max(2^-4 t, 2^-10) of t = top / (6 s), half a step of a normal or a subnormal number. Between
    # 4 and 6 codes are at most 1 from a value: b <= t + r. Beyond 6 b it is clipped: by at most 6 r, which is
    # 0.375 t, or 6 * 2^-10 where b is subnormal. Groups of a top beyond 6 * 448 s are out of range
    off = np.abs(back[1].double().numpy() - x) - 1.01 * (top / 6 * (1 + 2.0 ** -4) + 6 * 2.0 ** -10 * s64) - 0.01 * top
    assert (off[top <= 2688 * s64] <= 0).all() and (top <= 2688 * s64).mean() > 0.9
    if q is not None:
        turned = ref.rotate32(q.float().cpu().numpy(), angles, rot, rotated, interleaved, last)
        assert torch.equal(q_out.cpu(), torch.from_numpy(turned).to(torch_type(kind)))


def test_numbers_at_the_ends_of_the_range():
    """Zeros, values below the least block scale, beyond the largest, on every border, infinite and NaN."""
    rng = np.random.default_rng(42)
    grid = ref.decode_e2m1(np.arange(8))
    borders = (grid[:-1] + grid[1:]) / 2
    rows = [np.zeros(64), np.full(64, 2.0 ** -14), np.full(64, 3e38), np.full(64, -3e38)]
    for b in (2.0 ** -9, 0.25, 1.0, 1.125, 1.875, 7.0, 448.0):   # a 6 b makes b the block scale
        row = np.concatenate([borders, -borders, [6.0, 0.0]] * 4) * b
        rows.append(row)
    for one in (np.inf, -np.inf, np.nan):
        row = rng.standard_normal(64)
        row[20] = one
        rows.append(row)
    k = torch.from_numpy(np.stack(rows)).float().bfloat16()[:, None, :].contiguous()
    T = len(rows)
    pool = _pool(T, 1, 1, 64)
    with KVCache(pool, num_layers=1, num_components=2, kv_heads=1, head_dim=64, block=1, num_blocks=T,
                 dtype=5) as cache:
        table = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
        requests = torch.arange(T, dtype=torch.int32, device="cuda")
        cache.append(0, k.cuda(), k.cuda(), requests, torch.zeros_like(requests), table)
        got, _ = cache.read(0, requests, torch.zeros_like(requests), table)
        cache.check()
    codes, scales = _views(pool, T, 1, 1, 64)
    c, s = ref.quantize(k.float().numpy())
    np.testing.assert_array_equal(scales[0, :, 0, 0], s[:, 0])
    nan = np.repeat(s[:, 0] == 0x7F, 8, -1)
    np.testing.assert_array_equal(codes[0, :, 0, 0][~nan], c[:, 0][~nan])
    want = ref.values(c, s)[:, 0]
    np.testing.assert_array_equal(got[:, 0].double().cpu().numpy(), want)
    assert np.isnan(want[-1, 16:32]).all() and np.isfinite(np.delete(want[-1], range(16, 32))).all()
    assert want[-3, 20] == 2688 and want[-2, 20] == -2688 and (want[2] == 2688).all()


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
def test_read_of_every_pool(pool):
    lengths = [70, 1, 33]
    case = More(43, lengths, heads=3, queries=3, dim=64, block=7, pool=pool, layers=2, layer=1)
    req = np.repeat(np.arange(3), lengths).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
    pos[5] = -1                                                  # padding
    dev = torch.from_numpy(req).cuda(), torch.from_numpy(pos).cuda(), case.dtable
    types = [torch.bfloat16, torch.float16] if pool in ("e4m3", "e2m1") else [torch_type(pool)]
    for dtype in types:
        room = torch.full((len(req), 5, 64), 7.0, dtype=dtype, device="cuda")
        k, v = case.cache.read(1, *dev, k=room[:, 1:4], dtype=dtype)
        case.cache.check()
        for got, comp in ((k, 0), (v, 1)):
            for t in range(len(req)):
                want = np.zeros((3, 64)) if pos[t] < 0 else \
                    case.wide[1, comp, case.table[req[t], pos[t] // 7], pos[t] % 7]
                # exact up to the product with the plane's scale: one fp32 rounding, one to 16 bits
                want = torch.from_numpy(want.astype(np.float32)).to(dtype)
                assert torch.equal(got[t].cpu(), want)
        assert (room[:, 0] == 7).all() and (room[:, 4] == 7).all()
    # what is out of range gives zeros, and says so
    bad = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3, -1, 0], [0, 0, 0, 10 ** 6])]
    k, v = case.cache.read(1, *bad, case.dtable, dtype=types[0])
    assert k[0].any() and not k[1:].any() and not v[1:].any()
    with pytest.raises(KVRelayoutError, match="request index, position"):
        case.cache.check()
    case.dtable[0, 0] = case.N
    k, _ = case.cache.read(1, bad[0][:1].contiguous(), bad[1][:1].contiguous(), case.dtable, dtype=types[0])
    assert not k.any()
    with pytest.raises(KVRelayoutError, match="block id"):
        case.cache.check()


def test_read_of_latents():
    case = More(44, [40, 3], dim=576, queries=16)
    req = torch.tensor([0] * 40 + [1] * 3, dtype=torch.int32, device="cuda")
    pos = torch.tensor(list(range(40)) + list(range(3)), dtype=torch.int32, device="cuda")
    k, v = case.cache.read(0, req, pos, case.dtable)
    case.cache.check()
    assert v is None
    for t in range(43):
        want = case.host[0, 0, case.table[int(req[t]), int(pos[t]) // 16], int(pos[t]) % 16]
        assert torch.equal(k[t].cpu(), want)


ATTEND = [
    ([1], {}, 0), ([0], {}, 0), ([2, 0, 1, 17], dict(new=3), 0),
    ([100], dict(heads=2, queries=2, dim=64, qtype="f16", block=32), 0),
    ([300, 5, 64], dict(heads=2, queries=8, block=16), 0), ([300, 5, 64], dict(heads=2, queries=8, block=5), 0),
    ([129, 128, 127], dict(heads=3, queries=15, dim=192, block=24), 0),
    ([77, 200], dict(heads=1, queries=16, dim=256, block=64), 0),
    ([77, 200], dict(heads=1, queries=40, dim=256, block=1), 0), ([500], dict(heads=1, queries=33, block=8), 0),
    ([31, 65], dict(heads=2, queries=32, dim=64), 0), ([90, 1, 0, 260], dict(heads=2, queries=16, new=4, block=32), 0),
    ([90, 1, 0, 260], dict(heads=2, queries=16, new=4, block=32, qtype="f16"), 50),
    ([90, 3, 700], dict(heads=1, queries=8, dim=64, new=2, block=7), 333), ([700, 30], dict(queries=4, new=9), 64),
    ([260, 33, 1], dict(heads=2, queries=48, dim=256), 100), ([6000], dict(heads=2, queries=4, block=64), 0),
    ([3000, 1, 0, 2000, 17, 900], dict(queries=16, dim=64, new=2), 0),
    ([97 * k % 701 for k in range(128)], dict(heads=1, queries=2, dim=64), 0),
    ([97 * k % 701 for k in range(129)], dict(heads=3, queries=3, dim=64), 0),
    ([200], dict(heads=1, queries=8, new=200), 0), ([2000] * 9, dict(heads=2, queries=4, dim=64, scaled=False), 0),
]


@pytest.mark.parametrize("lengths, kw, window", ATTEND)
def test_attend(lengths, kw, window):
    More(45, lengths, pool="e2m1", **kw).attend_scored(window=window)


def test_most_requests_of_one_call():
    More(46, [(7 * r) % 5 for r in range(2048)], heads=1, queries=1, dim=64, block=4, pool="e2m1").attend_scored()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_strided_pools_and_layers(dim):
    """Heads before tokens, rows apart from each other's ends, layers in tensors of their own."""
    from prefill_decode_paged_gb300.kv_relayout import layout_of_views

    def padded(case):
        L, C, N, B, H, half = case.codes.shape
        gap = 64 if dim % 128 == 0 else 32
        views, more = [], []
        for layer in range(L):
            per = []
            for c in range(C):
                t = torch.zeros((N, H, B, half + gap), dtype=torch.uint8, device="cuda")
                s = torch.full((N, H, B, (half + gap) // 8), 0x7F, dtype=torch.uint8, device="cuda")
                v, w = t[..., :half].transpose(1, 2), s[..., :half // 8].transpose(1, 2)
                v.copy_(torch.from_numpy(case.codes[layer, c]))
                w.copy_(torch.from_numpy(case.block_scales[layer, c]))
                per.append(v)
                more.append(w)
            views.append(per)
        return views, layout_of_views([views]), more

    for layer in (0, 1):
        case = More(47, [90, 33], heads=3, queries=6, dim=dim, layers=2, layer=layer, layout=padded, pool="e2m1")
        case.attend_scored(scale=0.11)
        req = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        pos = torch.tensor([89, 32], dtype=torch.int32, device="cuda")
        k = torch.randn((2, 3, dim), device="cuda").bfloat16()
        before = [v.clone() for per in case.dev for v in per]
        case.cache.append(layer, k, 2 * k, req, pos, case.dtable)
        a, b = case.cache.read(layer, req, pos, case.dtable)
        case.cache.check()
        scale = torch.from_numpy(case.scales[layer]).cuda()
        for got, x, comp in ((a, k, 0), (b, 2 * k, 1)):
            want = [ref.quantize(x[:, h].float().cpu().numpy(), case.scales[layer, comp, h]) for h in range(3)]
            want = torch.stack([torch.from_numpy(ref.values(*w)).float() for w in want], 1).cuda()
            assert torch.equal(got, (want * scale[comp][:, None]).bfloat16())
        for i, (v, old) in enumerate(zip([v for per in case.dev for v in per], before)):
            same = (v == old).all(-1).all(-1)
            for r, p in ((0, 89), (1, 32)):
                same[int(case.table[r, p // 16]), p % 16] = True
            assert same.all()


def test_offsets_beyond_32_bits():
    """Blocks 1.5 GB apart, so that the last lie past 4 GB."""
    stride, N, B, D = 3 << 29, 5, 16, 64
    big = torch.empty(N * stride, dtype=torch.uint8, device="cuda")
    more = torch.empty(N * stride // 8, dtype=torch.uint8, device="cuda")
    small = More(48, [80], heads=1, queries=4, dim=D, block=B, pool="e2m1", scaled=False)
    order = [4, 2, 0, 3, 1]
    views, scales = [], []
    for c in range(2):
        v = big[c << 20:].as_strided((N, B, 1, D // 2), (stride, D // 2, D // 2, 1), c << 20)
        s = more[c << 17:].as_strided((N, B, 1, D // 16), (stride // 8, D // 16, D // 16, 1), c << 17)
        for k in range(5):
            v[order[k]] = torch.from_numpy(small.codes[0, c, small.table[0, k]])
            s[order[k]] = torch.from_numpy(small.block_scales[0, c, small.table[0, k]])
        views.append(v)
        scales.append(s)
    cache = KVCache(None, num_layers=1, num_components=2, kv_heads=1, head_dim=D, block=B, num_blocks=N, dtype=5,
                    query_heads=4, block_scales=scales,
                    layout=dict(bases=views, block_stride=stride, token_stride=D // 2, head_stride=D // 2,
                                shape=(N, B, 1, D // 2), elem_bytes=1))
    table = torch.tensor([order], dtype=torch.int32, device="cuda")
    out, lse = cache.attend(0, small.q, small.dlen, table)
    cache.check()
    small.check_scored(out, lse, D ** -0.5)
    k = torch.randn((1, 1, D), device="cuda").bfloat16()
    zero, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda")
    cache.append(0, k, 2 * k, zero, pos, table)
    a, b = cache.read(0, zero, pos, table)
    cache.check()
    c, s = ref.quantize(k.float().cpu().numpy())
    assert torch.equal(a.cpu(), torch.from_numpy(ref.values(c, s)).bfloat16()) and torch.equal(b, 2 * a)
    np.testing.assert_array_equal(views[0][4, 5].cpu().numpy(), c[0])
    cache.close()
    del big, more, views, scales, v, s
    torch.cuda.empty_cache()


def test_bad_lengths_and_blocks_are_flagged_and_not_read():
    case = More(49, [50, 90, 20], heads=2, queries=8, dim=64, pool="e2m1")
    case.attend_scored(scale=0.1)
    for bad in (-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        lens = case.dlen.clone()
        lens[1] = bad
        table = torch.zeros_like(case.dtable)
        table[0], table[2] = case.dtable[0].clamp(min=0), case.dtable[2].clamp(min=0)
        out, lse = case.cache.attend(0, case.q, lens, table, scale=0.1)
        with pytest.raises(KVRelayoutError, match="length"):
            case.cache.check()
    table = case.dtable.clone()
    table[1, 2] = case.N                                          # its keys and values count as zeros
    out, lse = case.cache.attend(0, case.q, case.dlen, table, scale=0.1)
    with pytest.raises(KVRelayoutError, match="block id"):
        case.cache.check()
    case.wide[0, :, case.table[1, 2]] = 0.0
    case.check_scored(out, lse, 0.1)


def test_a_nan_block_scale_reaches_its_own_rows_only():
    case = More(50, [40, 40], heads=2, queries=4, dim=64, pool="e2m1")
    n = case.codes.size
    flat = np.ravel_multi_index((0, 0, case.table[0, 1], 3, 0, 2), case.block_scales.shape)
    case.dev[n + int(flat)] = 0x7F                                # a key of request 0, head 0
    out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 0, :2].float()).all() and torch.isnan(lse[0, 0, :2]).all()
    assert torch.isfinite(out[0, 0, 2:].float()).all() and torch.isfinite(out[1].float()).all()


def test_the_same_bits_again_captured_and_on_another_stream():
    case = More(51, [3000, 1200, 40], heads=2, queries=8, dim=64, pool="e2m1")
    first, lse = case.attend_scored(scale=0.1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, l2 = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1, stream=side)
    side.synchronize()
    assert torch.equal(out, first) and torch.equal(l2, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, l2 = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(l2, lse)
    case.lengths = [700, 0, 33]
    case.dlen.copy_(torch.tensor(case.lengths, dtype=torch.int32))
    graph.replay()
    case.cache.check()
    case.check_scored(out, l2, 0.1)


def test_padding_and_bad_tokens_write_nothing():
    pool = _pool(4, 2, 1, 64, 0x33)
    before = pool.clone()
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    k = torch.randn((6, 1, 64), device="cuda").bfloat16()
    req = torch.tensor([0, 2, -1, 0, 1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([-5, 0, 0, 4, 2, 1], dtype=torch.int32, device="cuda")
    angles = torch.tensor([0, 0, 0, 0, 0, 8], dtype=torch.int32, device="cuda")
    rot = torch.from_numpy(rotary_table(8, 64)).cuda()
    with KVCache(pool, num_layers=1, num_components=2, kv_heads=1, head_dim=64, block=2, num_blocks=4,
                 dtype=5) as cache:
        cache.append(0, k, k, req, pos, table, rotary=rot, angles=angles)
        with pytest.raises(KVRelayoutError, match="request index, position, block id"):
            cache.check()
    assert torch.equal(pool, before)


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("tokens", [3, 700])
def test_angles_of_their_own_in_other_pools(pool, tokens):
    """The rows of a call whose positions are the angles, at other places."""
    dt = torch.float16 if pool == "f16" else torch.bfloat16
    D, H = 64, 2
    gen = torch.Generator("cuda").manual_seed(5)
    k, v, q = (torch.randn((tokens, H, D), generator=gen, device="cuda").to(dt) for _ in range(3))
    at = torch.randperm(1000, generator=gen, device="cuda")[:tokens].to(torch.int32)
    angles = torch.randperm(1000, generator=gen, device="cuda")[:tokens].to(torch.int32)
    req = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    table = torch.arange(63, dtype=torch.int32, device="cuda")[None].contiguous()
    rot = torch.from_numpy(rotary_table(1000, D)).cuda()
    kw = dict(num_layers=1, num_components=2, kv_heads=H, head_dim=D, block=16, num_blocks=63,
              dtype={"bf16": 1, "f16": 3, "e4m3": 2}[pool], scales=np.ones((1, 2)) if pool == "e4m3" else None)
    a, b = (torch.zeros((1, 2, 63, 16, H, D), dtype=torch.uint8 if pool == "e4m3" else dt, device="cuda")
            for _ in range(2))
    with KVCache(a, **kw) as one, KVCache(b, **kw) as two:
        qa = one.append(0, k, v, req, angles, table, rotary=rot, q=q)
        qb = two.append(0, k, v, req, at, table, rotary=rot, q=q, angles=angles)
        one.check()
        two.check()
    assert torch.equal(qa, qb)
    fa, fb = a.view(2, -1, H, D), b.view(2, -1, H, D)
    assert torch.equal(fa[:, angles.long()], fb[:, at.long()])


def test_hand_off_of_a_four_bit_pool_as_two_bit_copies():
    """Codes, then block scales, by the relayout: rows of D / 2 and (all heads of a token) H D / 16 bytes."""
    from prefill_decode_paged_gb300 import RelayoutPlan
    import workloads as wl
    H, D, n = 4, 128, 75
    w = wl.custom("four", 3, num_layers=1, num_components=2, kv_heads=H, head_dim=D // 2, elem_bytes=1, src_tp=1,
                  dst_tp=1, src_block=16, dst_block=32, seq_lens=[n])
    case = More(52, [n], heads=H, queries=8, dim=D, pool="e2m1", scaled=False)
    Ns, Nd = case.N, w.dst_num_blocks
    codes = case.codes.size
    dst = _pool(Nd, 32, H, D)
    tables = dict(seq_lens=np.array([n]), src_off=np.array([0, 5]), src_bt=case.table[0, :5].copy(),
                  dst_off=w.dst_off, dst_bt=w.dst_bt)
    both = dict(num_layers=1, num_components=2, elem_bytes=1, src_tp=1, dst_tp=1, src_block=16, dst_block=32,
                src_num_blocks=Ns, dst_num_blocks=Nd, **tables)
    split = 2 * Nd * 32 * H * D // 2
    with RelayoutPlan([case.dev[:codes]], [dst[:split]], kv_heads=H, head_dim=D // 2, **both) as plan:
        plan.run_all()
    with RelayoutPlan([case.dev[codes:]], [dst[split:]], kv_heads=1, head_dim=H * D // 16, **both) as plan:
        plan.run_all()
    table = torch.from_numpy(w.dst_bt[None, :3].astype(np.int32).copy()).cuda()
    with KVCache(dst, num_layers=1, num_components=2, kv_heads=H, head_dim=D, block=32, num_blocks=Nd, dtype=5,
                 query_heads=8) as cache:
        out, lse = cache.attend(0, case.q, case.dlen, table, scale=0.1)
        cache.check()
    case.check_scored(out, lse, 0.1)
