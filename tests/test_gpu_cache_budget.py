"""The cache's further calls as a decode under a memory budget makes them, one after another; and where they meet
streams of few SMs, many heads, host threads and graphs."""
import threading

import numpy as np
import pytest
import torch

import cache_more_ref as ref
from cache_more_case import More
from prefill_decode_paged_gb300 import KVCache, KVRelayoutError, SmStream, rotary_table
from test_gpu_cache_weigh import check as check_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "e2m1"])
def test_a_decode_under_a_budget(pool):
    """Prompts appended; then steps of append, attention, weights, and every 8 steps an eviction: one step one graph.
    Everything is followed in numpy: what is cached in which slot, each step's attention and weights."""
    R, H, Q, D, B, keep, recent, steps = 3, 2, 4, 64, 8, 40, 12, 17
    prompts, cap = [33, 40, 5], 20.0
    gen = torch.Generator("cuda").manual_seed(12)
    room = keep + 8 + 8                                          # tokens a request holds at most
    width = -(-room // B)
    N = R * width + 1
    rows = 2 * N * B * H
    dtype = {"bf16": 1, "e4m3": 2, "e2m1": 5}[pool]
    raw = torch.zeros(rows * D * 2 if pool == "bf16" else rows * D if pool == "e4m3" else rows * D * 9 // 16,
                      dtype=torch.uint8, device="cuda")
    table = torch.randperm(N, generator=gen, device="cuda")[:R * width].to(torch.int32).view(R, width).contiguous()
    angles = torch.from_numpy(rotary_table(200, D)).cuda()
    cache = KVCache(raw, num_layers=1, num_components=2, kv_heads=H, head_dim=D, block=B, num_blocks=N, dtype=dtype,
                    scales=np.full((1, 2), 0.05) if pool == "e4m3" else None, query_heads=Q, max_requests=R)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    # the prompts, as whole
    req = torch.repeat_interleave(torch.arange(R), torch.tensor(prompts)).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in prompts]).to(torch.int32).cuda()
    cache.append(0, randn(sum(prompts), H, D), randn(sum(prompts), H, D), req, pos, table, rotary=angles)
    weights = torch.zeros((R, H, room), device="cuda")
    k, v, q = randn(R, H, D), randn(R, H, D), randn(R, Q, D)
    turned, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((R, Q), device="cuda")
    slots = torch.empty((R, H, keep), dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    places, true = lengths.clone(), lengths.clone()              # slot and position of the next token
    requests = torch.arange(R, dtype=torch.int32, device="cuda")

    def step():
        lengths.add_(1)
        cache.append(0, k, v, requests, places, table, rotary=angles, q=q, q_out=turned, angles=true)
        cache.attend(0, turned, lengths, table, out=out, lse=lse, cap=cap)
        cache.weigh(0, turned, lse, lengths, table, weights, cap=cap)
        places.add_(1)
        true.add_(1)

    def evict():
        cache.evict(0, weights, lengths, table, keep, recent, slots=slots)
        lengths.clamp_(max=keep)
        places.copy_(lengths)

    graphs = []
    state = [t.clone() for t in (raw, weights, lengths, places, true)]
    for body in (step, evict):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            body()
        graphs.append(g)
    for t, s in zip((raw, weights, lengths, places, true), state):
        assert torch.equal(t, s)                                 # (capture runs nothing)

    def everything(n):
        """All cached rows, read back: [R] of (keys, values) [n][H][D] float64."""
        r = torch.cat([torch.full((int(x),), i) for i, x in enumerate(n)]).to(torch.int32).cuda()
        p = torch.cat([torch.arange(int(x)) for x in n]).to(torch.int32).cuda()
        a, b = cache.read(0, r, p, table)
        sizes = [int(x) for x in n]
        return [(x.double().cpu().numpy(), y.double().cpu().numpy())
                for x, y in zip(torch.split(a, sizes), torch.split(b, sizes))]

    want_w = np.zeros((R, H, room))
    n = np.array(prompts)
    for s in range(steps):
        for t in (k, v, q):
            t.copy_(randn(*t.shape))
        before = everything(n)
        graphs[0].replay()
        n = n + 1
        held = everything(n)
        assert lengths.tolist() == list(n)
        for r in range(R):
            for a, b in zip(before[r], held[r]):
                assert np.array_equal(a, b[:-1])                 # what was there stays
            p = prompts[r] + s                                   # the token's own position
            turn = ref.rotate32(k.float().cpu().numpy()[r:r + 1], [p], angles.cpu().numpy(), D, False, False)[0]
            # bf16: rounded once (fused products: 2^-24 of |a| + |b| besides); codes: half a step
            step_of = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -4 + 2.0 ** -8, "e2m1": 0.5}[pool]
            size = np.abs(turn).max()
            assert (np.abs(held[r][0][-1] - turn) <= step_of * np.abs(turn) + 0.18 * size * (pool == "e2m1") +
                    2.0 ** -10).all()
        q64 = turned.double().cpu().numpy()
        for r in range(R):
            for g in range(Q):
                key, val = held[r][0][:, g // 2], held[r][1][:, g // 2]
                x = cap * np.tanh(key @ q64[r, g] * D ** -0.5 / cap)
                z = np.log(np.exp(x - x.max()).sum()) + x.max()
                pr = np.exp(x - z)
                # read back as bf16: scales of 0.05 cost up to 2^-8 of each value (and score)
                tol = 2.0 ** -8 + (2.0 ** -6 * np.abs(key) @ np.abs(q64[r, g]) * D ** -0.5).max() * (pool == "e4m3")
                assert np.abs(out[r, g].double().cpu().numpy() - pr @ val).max() <= \
                    (tol + 2.0 ** -8) * np.abs(val).max() + 2.0 ** -8
                want_w[r, g // 2, :n[r]] += np.exp(x - float(lse[r, g]))
        got = weights.double().cpu().numpy()
        bound = 2.0 ** -14 if pool != "e4m3" else 0.2
        assert np.abs(got - want_w).max() <= bound * (s + 1) and not got[np.arange(room)[None, None] >= n[:, None, None].repeat(H, 1)].any()
        want_w = got                                             # (from here on by what the weights are)
        if s % 8 == 7:
            graphs[1].replay()
            after = everything(np.minimum(n, keep))
            for r in range(R):
                for h in range(H):
                    j = ref.kept_slots(got[r, h].astype(np.float32), int(n[r]), keep, recent)
                    assert slots[r, h, :len(j)].tolist() == j
                    for a, b in zip(held[r], after[r]):
                        assert np.array_equal(a[j, h], b[:, h])
                    w = np.zeros(room)
                    w[:len(j)] = got[r, h, j]
                    want_w[r, h] = w
            n = np.minimum(n, keep)
            assert np.array_equal(weights.double().cpu().numpy(), want_w)
    cache.check()
    assert (n >= keep).sum() >= 2
    cache.close()


@pytest.mark.parametrize("sms", [8, 16])
def test_streams_of_few_sms(sms):
    """Grids and clusters that fit a part of the device."""
    case = More(111, [2500, 100, 0], heads=2, queries=8, dim=64, pool="e2m1")
    torch.cuda.synchronize()
    with SmStream(sms) as s:
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1, cap=4.0, stream=s.handle)
        old = torch.zeros((3, 2, 2500), device="cuda")
        torch.cuda.synchronize()
        w = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone(), scale=0.1, cap=4.0, stream=s.handle)
        torch.cuda.synchronize()
        case.cache.check()
        case.check_scored(out, lse, 0.1, cap=4.0)
        check_weights(case, w, old, lse, 0.1, cap=4.0)
        kept, slots = case.cache.evict(0, w.clone(), case.dlen, case.dtable, 1500, 100, stream=s.handle)
        torch.cuda.synchronize()
        case.cache.check()
    for r, n in enumerate(case.lengths):
        for h in range(2):
            j = ref.kept_slots(w[r, h].cpu().numpy(), n, 1500, 100)
            assert slots[r, h, :len(j)].tolist() == j
            assert torch.equal(kept[r, h, :len(j)], w[r, h, j])


@pytest.mark.parametrize("pool", ["bf16", "e2m1"])
def test_more_heads_than_blocks(pool):
    """700 heads: more than an SM's share of them all."""
    case = More(112, [5, 0, 40], heads=700, queries=700, dim=64, block=4, pool=pool)
    out, lse = case.attend_scored(cap=3.0)
    old = torch.rand((3, 700, 41), device="cuda")
    w = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone(), cap=3.0)
    case.cache.check()
    check_weights(case, w, old, lse, 64 ** -0.5, cap=3.0)
    case = More(113, [300, 33], heads=40, queries=40, dim=128, pool=pool)
    out, lse = case.attend_scored()
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, torch.zeros((2, 40, 300), device="cuda"))
    check_weights(case, got, torch.zeros((2, 40, 300), device="cuda"), lse, 128 ** -0.5)


def test_block_tables_of_one_row_for_all():
    """Requests that share all their blocks, by a table whose rows are one."""
    case = More(114, [90], heads=2, queries=4, dim=64, pool="e2m1")
    table = case.dtable.expand(3, case.dtable.shape[1])
    lens = torch.tensor([90, 17, 0], dtype=torch.int32, device="cuda")
    q = case.q.expand(3, 1, 4, 64).contiguous()
    cache = KVCache(case.dev, num_layers=1, num_components=2, kv_heads=2, head_dim=64, block=16, num_blocks=case.N,
                    dtype=5, scales=case.scales, per_head=True, query_heads=4, max_requests=3)
    out, lse = cache.attend(0, q, lens, table, cap=5.0)
    w = cache.weigh(0, q, lse, lens, table, torch.zeros((3, 2, 90), device="cuda"), cap=5.0)
    cache.check()
    case.lengths, case.table = [90, 17, 0], np.repeat(case.table, 3, 0)
    case.q = q
    case.check_scored(out, lse, 64 ** -0.5, cap=5.0)
    check_weights(case, w, torch.zeros((3, 2, 90), device="cuda"), lse, 64 ** -0.5, cap=5.0)
    # evicted into blocks of their own
    fresh = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    free = [b for b in range(case.N) if b not in case.table[0, :6]]
    fresh[0, 0], fresh[1, 0] = free[0], free[1]
    kept, slots = cache.evict(0, w, lens, table, 16, 4, into=fresh[:, :1].contiguous(), out=torch.zeros_like(w))
    cache.check()
    req = torch.tensor([0] * 16 + [1] * 16, dtype=torch.int32, device="cuda")
    pos = torch.arange(16, dtype=torch.int32, device="cuda").repeat(2)
    k, v = cache.read(0, req, pos, fresh)
    for r in range(2):
        for h in range(2):
            j = ref.kept_slots(w[r, h].cpu().numpy(), case.lengths[r], 16, 4)
            assert slots[r, h].tolist() == j
            a, b = cache.read(0, torch.zeros(16, dtype=torch.int32, device="cuda"),
                              torch.tensor(j, dtype=torch.int32, device="cuda"), table)
            assert torch.equal(k[16 * r:16 * r + 16, h], a[:, h]) and torch.equal(v[16 * r:16 * r + 16, h], b[:, h])
    cache.close()


def test_host_threads_with_streams_of_their_own():
    """Weights and evictions use no workspace: threads need no order."""
    case = More(115, [700, 300], heads=2, queries=4, dim=64)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    old = torch.zeros((2, 2, 700), device="cuda")
    want = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    wanted, _ = case.cache.evict(0, want.clone(), torch.zeros_like(case.dlen), case.dtable, 100)
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                w = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, torch.zeros_like(old))
                if not torch.equal(w, want):
                    wrong.append("weigh")
                # (lengths of zero: nothing moves, nothing is written)
                e, _ = case.cache.evict(0, w, torch.zeros_like(case.dlen), case.dtable, 100)
                if not torch.equal(e, wanted):
                    wrong.append("evict")

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    case.cache.check()
    assert not wrong


def test_calls_of_a_closed_or_appending_cache():
    case = More(116, [20], heads=2, queries=8, dim=64)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    append_only = KVCache(case.dev, num_layers=1, num_components=2, kv_heads=2, head_dim=64, block=16,
                          num_blocks=case.N, dtype=1)
    w = torch.rand((1, 2, 20), device="cuda")
    with pytest.raises((KVRelayoutError, ValueError)):
        append_only.weigh(0, case.q, lse, case.dlen, case.dtable, w)
    kept, slots = append_only.evict(0, w.clone(), case.dlen, case.dtable, 10)
    append_only.check()
    for h in range(2):
        assert slots[0, h].tolist() == ref.kept_slots(w[0, h].cpu().numpy(), 20, 10, 0)
    append_only.close()
    for call in (lambda: append_only.evict(0, w, case.dlen, case.dtable, 10),
                 lambda: append_only.read(0, case.dlen, case.dlen, case.dtable)):
        with pytest.raises(RuntimeError, match="closed"):
            call()
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    k, v = case.cache.read(0, empty, empty, case.dtable)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    got, slots = case.cache.evict(0, w[:0], empty, case.dtable[:0], 10)
    assert got.shape == (0, 2, 20) and slots.shape == (0, 2, 10)
    assert case.cache.weigh(0, case.q[:0], lse[:0], empty, case.dtable[:0], w[:0]).shape == (0, 2, 20)
    case.cache.check()
