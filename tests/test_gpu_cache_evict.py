"""Eviction by weights on the GPU: what stays, where it goes, and what is left alone, bit for bit."""
import numpy as np
import pytest
import torch

import cache_more_ref as ref
from cache_more_case import More
from prefill_decode_paged_gb300 import KVCache, KVRelayoutError

pytestmark = pytest.mark.gpu

BYTES = {"bf16": 2, "f16": 2, "e4m3": 1}


class Pool:
    """Random bytes in every slot, tables of scattered blocks for the requests and for what stays."""

    def __init__(self, seed, lengths, keep, *, heads=2, dim=64, block=16, pool="bf16", layers=1, layer=0, extra=0):
        self.rng = rng = np.random.default_rng(seed)
        self.lengths, self.keep, self.H, self.D, self.B, self.kind = lengths, keep, heads, dim, block, pool
        self.layer = layer
        need = [max(1, -(-n // block)) for n in lengths]
        more = [max(1, -(-min(n, keep) // block)) for n in lengths]
        self.N = sum(need) + sum(more) + 2
        order = rng.permutation(self.N).astype(np.int32)
        self.tables, at = [], 0
        for counts in (need, more):
            t = np.full((len(lengths), max(counts) + 1), -3, dtype=np.int32)
            for r, k in enumerate(counts):
                t[r, :k] = order[at:at + k]
                at += k
            self.tables.append(t)
        rows = layers * 2 * self.N * block * heads
        self.row = dim // 2 + dim // 16 if pool == "e2m1" else dim * BYTES[pool]
        self.first = torch.from_numpy(rng.integers(0, 256, rows * self.row).astype(np.uint8)).cuda()
        self.dev = self.first.clone()
        self.shape = (layers, 2, self.N, block, heads)
        self.cache = KVCache(self.dev, num_layers=layers, num_components=2, kv_heads=heads, head_dim=dim, block=block,
                             num_blocks=self.N, dtype={"bf16": 1, "f16": 3, "e4m3": 2, "e2m1": 5}[pool],
                             scales=np.ones((layers, 2)) if pool == "e4m3" else None)
        self.dlen = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.dtables = [torch.from_numpy(t).cuda() for t in self.tables]
        self.S = max(lengths + [0]) + extra

    def parts(self, flat):
        """The pool's rows: [L][2][N][B][H][bytes], one array or (4 bits) codes and block scales."""
        host = flat.cpu().numpy()
        if self.kind != "e2m1":
            return [host.reshape(self.shape + (self.row,))]
        n = int(np.prod(self.shape)) * (self.D // 2)
        return [host[:n].reshape(self.shape + (self.D // 2,)), host[n:].reshape(self.shape + (self.D // 16,))]

    def weights(self, kind="exp"):
        shape = len(self.lengths), self.H, self.S
        rng = self.rng
        if kind == "exp":
            w = np.exp(3 * rng.standard_normal(shape))
        elif kind == "few":                                      # many equal ones
            w = rng.integers(0, 4, shape) * 0.25
        elif kind == "zero":
            w = np.zeros(shape)
        elif kind == "close":                                    # that differ in the last bits alone
            w = 1 + rng.integers(0, 2000, shape) * 2.0 ** -23
        elif kind == "odd":                                      # of both signs, both zeros, infinite, NaN
            w = rng.choice([-np.inf, -2.5, -0.0, 0.0, 1e-40, 1.0, 3.4e38, np.inf, np.nan], shape) * 1.0
        else:                                                    # falling, rising
            w = np.broadcast_to(np.arange(self.S), shape) * (1.0 if kind == "rising" else -1.0)
        return torch.from_numpy(w.astype(np.float32)).cuda()

    def check(self, weights, out, slots, recent, into, old_out, old_slots=-1, keep=None):
        keep = keep or self.keep
        host, got_w, got_s = (t.cpu().numpy() for t in (weights, out, slots))
        want_w = old_out.cpu().numpy().copy()
        want_s = np.full_like(got_s, old_slots)
        first, dest = self.parts(self.first), self.tables[1 if into else 0]
        want = [p.copy() for p in first]
        for r, n in enumerate(self.lengths):
            for h in range(self.H):
                j = np.array(ref.kept_slots(host[r, h], n, keep, recent), dtype=np.int64)
                i = np.arange(len(j))
                assert len(j) == min(n, keep)
                want_s[r, h, :len(j)] = j
                want_w[r, h, :n] = 0
                want_w[r, h, :len(j)] = host[r, h, j]
                a, b = self.tables[0][r, j // self.B], dest[r, i // self.B]
                for p, f in zip(want, first):
                    p[self.layer][:, b, i % self.B, h] = f[self.layer][:, a, j % self.B, h]
        np.testing.assert_array_equal(got_s, want_s)
        np.testing.assert_array_equal(got_w, want_w)
        for p, q in zip(self.parts(self.dev), want):
            np.testing.assert_array_equal(p, q)

    def evict(self, recent, into, kind="exp", apart=None, **kw):
        w = self.weights(kind)
        apart = into if apart is None else apart
        given = w.clone()
        out = torch.full_like(w, 9.0) if apart else given
        old = out.clone()
        got, slots = self.cache.evict(self.layer, given, self.dlen, self.dtables[0], self.keep, recent,
                                      into=self.dtables[1] if into else None, out=out if apart else None, **kw)
        self.cache.check()
        assert got is out
        if apart:
            assert torch.equal(given.view(torch.int32), w.view(torch.int32))
        self.check(w, got, slots, recent, into, old)


CASES = [
    # lengths, keep, recent, kw
    ([5], 3, 1, {}), ([1, 0, 2], 1, 0, {}), ([1, 0, 2], 1, 1, {}), ([40, 7, 0, 33], 32, 8, dict(block=5)),
    ([300, 5, 64, 129], 64, 0, dict(heads=3, block=24)), ([300, 5, 64, 129], 64, 64, {}), ([300, 65], 64, 63, {}),
    ([700, 1000, 999], 998, 100, dict(heads=1, block=1)), ([700], 10 ** 6, 10, {}), ([2500, 100], 2000, 1, dict(dim=128)),
    ([520] * 33, 512, 32, dict(heads=5, dim=64)), ([9000], 4097, 1024, dict(heads=2)), ([600, 1200], 300, 7, dict(dim=192)),
    ([400], 399, 0, dict(dim=256, block=32)),
]


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("lengths, keep, recent, kw", CASES)
def test_what_stays_and_where_it_goes(lengths, keep, recent, kw, pool, into):
    Pool(91, lengths, keep, pool=pool, **kw).evict(recent, into)


@pytest.mark.parametrize("kind", ["few", "zero", "close", "odd", "falling", "rising"])
@pytest.mark.parametrize("into", [False, True])
def test_ties_and_odd_weights(kind, into):
    Pool(92, [3000, 77, 1, 513], 500, heads=2, dim=16, extra=5).evict(60, into, kind)
    Pool(92, [600], 599, heads=1, dim=16).evict(0, into, kind)


@pytest.mark.parametrize("kind", ["exp", "few", "close"])
def test_more_weights_than_a_block_holds(kind):
    """Shares of a head's weights beyond what shared memory holds, and heads of one block each."""
    Pool(93, [70000, 9], 30000, heads=1, dim=16, block=64).evict(5000, False, kind)
    Pool(94, [9001] * 3 + [5000] * 40, 4000, heads=8, dim=16, block=64).evict(100, True, kind)


def test_weights_and_rows_need_not_both_be_in_place():
    Pool(95, [900, 33], 128).evict(16, False, apart=True)
    Pool(96, [900, 33], 128).evict(16, True, apart=False)


@pytest.mark.parametrize("dim", [16, 48, 80, 96, 160])
def test_head_sizes(dim):
    for pool in ("bf16", "e4m3"):
        for into in (False, True):
            Pool(97, [333, 90], 50, dim=dim, heads=3, pool=pool, block=7).evict(5, into)


def test_layers_and_strided_weights():
    case = Pool(98, [200, 90], 60, heads=3, layers=3, layer=1, extra=4)
    room = torch.full((3, 5, 2, 300), 7.0, device="cuda")
    w = case.weights()
    rows = room[:, 1:3, 1, 20:20 + case.S].transpose(0, 1)       # [2][3][S] of a wider tensor
    rows.copy_(w)
    before = room.clone()
    out, slots = case.cache.evict(1, rows, case.dlen, case.dtables[0], 60, 10)
    case.cache.check()
    case.check(w, out, slots, 10, False, w)
    rows.copy_(w)
    assert torch.equal(room, before)


def test_again_and_again_as_a_decode_does():
    """64 tokens more each time, with weights of their own: each time by the slots that the last left."""
    case = Pool(99, [400, 320], 256, heads=2, dim=64, extra=0)   # (blocks for 320 at least)
    w = case.weights()
    state = w.clone()
    for step in range(4):
        out, slots = case.cache.evict(0, state, case.dlen, case.dtables[0], 256, 32)
        case.cache.check()
        case.check(w, out, slots, 32, False, w)
        # what is there now is the next one's start
        case.first.copy_(case.dev)
        state[:, :, 256:320] = torch.rand((2, 2, 64), device="cuda")
        w = state.clone()
        case.lengths = [320, 320]
        case.dlen.copy_(torch.tensor(case.lengths, dtype=torch.int32))


def test_captured_and_on_another_stream():
    case = Pool(100, [900, 33, 500], 128, heads=2)
    w = case.weights()
    out, slots = torch.full_like(w, 9.0), torch.full((3, 2, 128), -1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        case.cache.evict(0, w, case.dlen, case.dtables[0], 128, 16, into=case.dtables[1], out=out, slots=slots)
    graph.replay()
    case.cache.check()
    case.check(w, out, slots, 16, True, torch.full_like(w, 9.0))
    case.dev.copy_(case.first)
    case.lengths = [130, 20, 900]
    case.tables[0][2], case.tables[0][0] = case.tables[0][0].copy(), case.tables[0][2].copy()
    case.dtables[0].copy_(torch.from_numpy(case.tables[0]))
    case.dlen.copy_(torch.tensor(case.lengths, dtype=torch.int32))
    out.fill_(9.0)
    slots.fill_(-1)
    graph.replay()
    case.cache.check()
    case.check(w, out, slots, 16, True, torch.full_like(w, 9.0))
    case.dev.copy_(case.first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = case.cache.evict(0, w.clone(), case.dlen, case.dtables[0], 128, 16, stream=side)
    side.synchronize()
    case.check(w, a, b, 16, False, w)


def test_bad_lengths_and_blocks_are_flagged_and_not_moved():
    for bad in (-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        case = Pool(101, [100, 90], 40)
        w = case.weights()
        lens = case.dlen.clone()
        lens[1] = bad
        out, slots = case.cache.evict(0, w.clone(), lens, case.dtables[0], 40, 10)
        with pytest.raises(KVRelayoutError, match="length|block id"):
            case.cache.check()
        if bad < 0:
            case.lengths = [100, 0]
            case.check(w, out, slots, 10, False, w)
    case = Pool(102, [100], 40, heads=1)
    w = case.weights()
    case.dtables[0][0, 3] = case.N                               # slots 48 .. 63
    out, slots = case.cache.evict(0, w.clone(), case.dlen, case.dtables[0], 40, 0, into=case.dtables[1],
                                  out=torch.zeros_like(w))
    with pytest.raises(KVRelayoutError, match="block id"):
        case.cache.check()
    got, first = case.parts(case.dev)[0], case.parts(case.first)[0]
    for i, j in enumerate(ref.kept_slots(w[0, 0].cpu().numpy(), 100, 40, 0)):
        b = case.tables[1][0, i // 16]
        src = first[0, :, b, i % 16, 0] if 48 <= j < 64 else first[0, :, case.tables[0][0, j // 16], j % 16, 0]
        np.testing.assert_array_equal(got[0, :, b, i % 16, 0], src)
    # a table that holds fewer tokens than stay
    case = Pool(103, [100], 40, heads=1)
    short = case.dtables[1][:, :2].contiguous()
    case.cache.evict(0, case.weights(), case.dlen, case.dtables[0], 40, 0, into=short, out=torch.zeros_like(w))
    with pytest.raises(KVRelayoutError, match="length"):
        case.cache.check()


def test_offsets_beyond_32_bits():
    """Blocks 1.5 GB apart."""
    stride, N, B, D = 3 << 29, 5, 16, 64
    for into in (False, True):
        big = torch.empty(N * stride, dtype=torch.uint8, device="cuda")
        order = [4, 2, 0, 3, 1]
        rng = np.random.default_rng(4)
        host = rng.integers(0, 256, (2, N, B, 2 * D)).astype(np.uint8)
        views = []
        for c in range(2):
            v = big.as_strided((N, B, 1, 2 * D), (stride, 2 * D, 2 * D, 1), c << 20)
            v.copy_(torch.from_numpy(host[c])[:, :, None])
            views.append(v)
        cache = KVCache(None, num_layers=1, num_components=2, kv_heads=1, head_dim=D, block=B, num_blocks=N, dtype=1,
                        layout=dict(bases=views, block_stride=stride, token_stride=2 * D, head_stride=2 * D,
                                    shape=(N, B, 1, D), elem_bytes=2))
        table = torch.tensor([order[:3]], dtype=torch.int32, device="cuda")
        other = torch.tensor([order[3:]], dtype=torch.int32, device="cuda")
        w = torch.rand((1, 1, 48), device="cuda")
        lens = torch.tensor([48], dtype=torch.int32, device="cuda")
        _, slots = cache.evict(0, w.clone(), lens, table, 30, 4, into=other if into else None,
                               out=torch.zeros_like(w) if into else None)
        cache.check()
        want = ref.kept_slots(w[0, 0].cpu().numpy(), 48, 30, 4)
        assert slots[0, 0].tolist() == want
        dest = order[3:] if into else order[:3]
        for i, j in enumerate(want):
            for c in range(2):
                np.testing.assert_array_equal(views[c][dest[i // B], i % B, 0].cpu().numpy(), host[c, order[j // B], j % B])
        cache.close()
        del big, views, v
        torch.cuda.empty_cache()


def test_refusals():
    case = Pool(104, [100, 90], 40)
    w = case.weights()
    args = case.dlen, case.dtables[0]
    for keep, recent in ((0, 0), (5, 6), (5, -1), (-1, 0)):
        with pytest.raises((KVRelayoutError, RuntimeError), match="INVALID|negative"):
            case.cache.evict(0, w, *args, keep, recent)
    for bad in (w[0], w[:, :1], w.double(), w.cpu(), torch.zeros((2, 2, 200), device="cuda")[..., ::2]):
        with pytest.raises(ValueError, match="weights"):
            case.cache.evict(0, bad, *args, 40)
    with pytest.raises(ValueError, match="out"):
        case.cache.evict(0, w, *args, 40, out=w[..., :50])
    with pytest.raises(ValueError, match="slots"):
        case.cache.evict(0, w, *args, 40, slots=torch.zeros((2, 2, 39), dtype=torch.int32, device="cuda"))
    with pytest.raises(KVRelayoutError, match="OVERLAP"):
        case.cache.evict(0, w, *args, 40, out=torch.zeros_like(w[:, :1]).expand(2, 2, w.shape[2]))
    with pytest.raises(KVRelayoutError, match="INVALID"):
        case.cache.evict(0, w, *args, 40, into=case.dtables[0][:, :3])
    with pytest.raises(ValueError, match="gradient"):
        case.cache.evict(0, w.clone().requires_grad_(), *args, 40)
    with pytest.raises(KVRelayoutError, match="LAYER"):
        case.cache.evict(1, w, *args, 40)
    latent = More(105, [20], dim=576, queries=16)
    with pytest.raises(KVRelayoutError, match="UNSUPPORTED"):
        latent.cache.evict(0, torch.zeros((1, 1, 20), device="cuda"), latent.dlen, latent.dtable, 10)
    assert torch.equal(case.dev, case.first)
