"""Host threads that evict with one cache: on one stream beside calls that write the same weights, and each on its own."""
import threading

import pytest
import torch

from cache_more_case import More
from prefill_decode_paged_gb300 import KVCache
from test_gpu_cache_evict import Pool

pytestmark = pytest.mark.gpu


def run(bodies):
    wrong = []

    def guarded(body):
        try:
            body()
        except Exception as e:                                   # (a thread's own failure would be lost)
            wrong.append(repr(e))
    threads = [threading.Thread(target=guarded, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_weights_of_another_thread_do_not_come_between_choice_and_move():
    """Threads write either of two patterns of weights, again and again, another evicts by them, on one stream:
    each eviction's slots and weights are those of the one pattern or of the other."""
    R, H, keep, recent, times = 2, 2, 150, 10, 1500
    case = More(121, [700, 333], heads=H, queries=4, dim=64)
    stream = torch.cuda.Stream()
    need = -(-keep // 16)
    # the same pool with blocks for what stays behind the requests' own
    pool = torch.zeros((1, 2, case.N + R * need, 16, H, 64), dtype=torch.bfloat16, device="cuda")
    pool[:, :, :case.N] = case.dev.view(1, 2, case.N, 16, H, 64)
    into = torch.arange(case.N, case.N + R * need, dtype=torch.int32, device="cuda").view(R, need)
    cache = KVCache(pool, num_layers=1, num_components=2, kv_heads=H, head_dim=64, block=16, num_blocks=case.N + R * need,
                    dtype=1, query_heads=4, max_requests=R)
    queries = [case.q, case.q.flip(-1).contiguous()]
    sums = [cache.attend(0, q, case.dlen, case.dtable)[1] for q in queries]
    weights = torch.zeros((R, H, 700), device="cuda")
    want = []
    for q, lse in zip(queries, sums):
        cache.weigh(0, q, lse, case.dlen, case.dtable, weights, add=False)
        want.append(cache.evict(0, weights, case.dlen, case.dtable, keep, recent, into=into, out=torch.zeros_like(weights)))
    assert not torch.equal(want[0][1], want[1][1])
    outs = torch.zeros((times, R, H, 700), device="cuda")
    slots = torch.full((times, R, H, keep), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    done = threading.Event()

    def write():
        k = 0
        while not done.is_set():
            cache.weigh(0, queries[k & 1], sums[k & 1], case.dlen, case.dtable, weights, add=False, stream=stream)
            k += 1

    def evict():
        try:
            for k in range(times):
                cache.evict(0, weights, case.dlen, case.dtable, keep, recent, into=into, out=outs[k], slots=slots[k],
                            stream=stream)
        finally:
            done.set()

    run([write] * 4 + [evict])
    cache.check()
    of = [((outs == w).flatten(1).all(1), (slots == s).flatten(1).all(1)) for w, s in want]
    mixed = sum(int((of[a][0] & of[b][1]).sum()) for a, b in ((0, 1), (1, 0)))
    whole = sum(int((w & s).sum()) for w, s in of)
    assert (mixed, whole) == (0, times)
    cache.close()


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_threads_evict_requests_of_their_own(kind):
    """Four threads, four streams, one cache: each evicts its own request, in place or into blocks of its own."""
    lengths, keep, recent = [900, 333, 520, 128], 128, 16
    case = Pool(122, lengths, keep, pool=kind)
    w = case.weights()
    out, slots = torch.zeros_like(w), torch.full((4, 2, keep), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def body(r):
        def go():
            s = torch.cuda.Stream()
            for _ in range(25):                                  # (the same each time: rows go to other blocks)
                case.cache.evict(0, w[r:r + 1], case.dlen[r:r + 1], case.dtables[0][r:r + 1], keep, recent,
                                 into=case.dtables[1][r:r + 1], out=out[r:r + 1], slots=slots[r:r + 1], stream=s)
            s.synchronize()
        return go

    run([body(r) for r in range(4)])
    case.cache.check()
    case.check(w, out, slots, recent, True, torch.zeros_like(w))
    case.dev.copy_(case.first)
    slots.fill_(-1)
    state = w.clone()
    torch.cuda.synchronize()

    def in_place(r):
        def go():
            s = torch.cuda.Stream()
            case.cache.evict(0, state[r:r + 1], case.dlen[r:r + 1], case.dtables[0][r:r + 1], keep, recent,
                             slots=slots[r:r + 1], stream=s)
            s.synchronize()
        return go

    run([in_place(r) for r in range(4)])
    case.cache.check()
    case.check(w, state, slots, recent, False, w)
