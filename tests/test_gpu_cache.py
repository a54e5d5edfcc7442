"""The decode cache on the GPU against its definitions in 64 bits.

Tolerances. An output is rounded once to its 16-bit type (u: half a unit in the last place, relative).
Before that it differs from sum_j p_j v_j by (e_p + 2 d) sum_j p_j |v_j|: e_p for the rounding of P
(two 16-bit numbers: 2^-15; one f16: 2^-10; one bf16: 2^-8) and d for the error of a logit, in units
of the logit: products of 16-bit numbers summed in fp32 by the tensor cores, taken as 2^-21 a step of
16 elements of the largest sum of |q||k| scale, and 2^-20 for the exponential. Sums over keys add
2^-22 a key at most. lse has d, and two fp32 roundings of its own size.
"""
import math

import numpy as np
import pytest

import cache_ref

pytestmark = pytest.mark.gpu

UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = {"bf16": 1, "f16": 3, "e4m3": 2}


def torch_type(t):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.uint8}[t]


class Case:
    """A pool with NaN everywhere but at the requests' own positions, its table and its cache."""

    def __init__(self, seed, lengths, *, heads=1, queries=8, dim=128, block=16, new=1, pool="bf16",
                 qtype=None, layers=1, layer=0, spread=1.0, per_head=True, layout=None,
                 max_requests=None):
        import torch
        from prefill_decode_paged_gb300 import KVCache
        self.rng = rng = np.random.default_rng(seed)
        self.lengths, self.H, self.Q, self.D, self.B = lengths, heads, queries, dim, block
        self.latent = dim == 576
        self.comps, self.V = (1, 512) if self.latent else (2, dim)
        self.new, self.pool_type, self.qtype = new, pool, qtype or ("bf16" if pool == "e4m3" else pool)
        self.layer = layer
        R = len(lengths)
        need = [max(1, -(-n // block)) for n in lengths]
        self.N = sum(need) + 3
        order = rng.permutation(self.N)
        width = max(need) + 1
        table = np.full((R, width), -7, dtype=np.int32)     # what is not used is not a block
        at = 0
        for r, k in enumerate(need):
            table[r, :k] = order[at:at + k]
            at += k
        self.table = table
        shape = (layers, self.comps, self.N, block, heads, dim)
        self.scales = None
        if pool == "e4m3":
            self.scales = rng.uniform(0.01, 0.1, (layers, self.comps, heads)).astype(np.float32)
            codes = np.full(shape, 0x7F, dtype=np.uint8)
            fine = rng.integers(0, 254, shape).astype(np.uint8)
            fine = fine + (fine >= 0x7F)
            fill = np.where(np.abs(cache_ref.decode_e4m3(fine)) <= 32, fine, fine & 0x9F)
            values = torch.from_numpy(codes)
            fill = torch.from_numpy(fill.astype(np.uint8))
        else:
            values = torch.full(shape, float("nan"), dtype=torch_type(pool))
            fill = torch.from_numpy(rng.standard_normal(shape) * spread).to(torch_type(pool))
        for r, n in enumerate(lengths):
            for k in range(need[r]):
                t = min(block, n - k * block)
                if t > 0:
                    values[:, :, table[r, k], :t] = fill[:, :, table[r, k], :t]
        self.host = values
        if pool == "e4m3":
            self.wide = cache_ref.decode_e4m3(values.numpy()) * self.scales.astype(np.float64)[:, :, None, None, :, None]
        else:
            self.wide = values.double().numpy()
        geometry = dict(num_layers=layers, num_components=self.comps, kv_heads=heads, head_dim=dim,
                        block=block, num_blocks=self.N, dtype=TYPES[pool], scales=self.scales,
                        per_head=per_head, query_heads=queries,
                        max_requests=max_requests or R, max_new=new)
        self.dev = values.cuda()
        if layout is None:
            self.cache = KVCache(self.dev, **geometry)
        else:
            self.dev, lay = layout(self)
            self.cache = KVCache(None, layout=lay, **geometry)
        q = rng.standard_normal((R, new, queries, dim)) * 1.5
        self.q = torch.from_numpy(q).to(torch_type(self.qtype)).cuda()
        self.dtable = torch.from_numpy(table).cuda()
        self.dlen = torch.tensor(lengths, dtype=torch.int32).cuda()

    def rows_of(self, r, g, j):
        h = g // (self.Q // self.H)
        b = self.table[r, j // self.B]
        k = self.wide[self.layer, 0, b, j % self.B, h]
        return k, k[:, :self.V] if self.latent else self.wide[self.layer, 1, b, j % self.B, h]

    def check(self, out, lse, scale, window, first=None):
        """All requests, or the first few (``out`` and ``lse`` of those)."""
        ref, rlse, size, logit = cache_ref.attend(self.q[:first].double().cpu().numpy(), self.rows_of,
                                                  self.lengths[:first], scale, window)
        n = max(self.lengths + [1])
        d = (self.D / 16 + 1) * 2.0 ** -21 * logit + 2.0 ** -20
        if self.pool_type == "e4m3":
            d = d + 2.0 ** -14 * logit * 2.0 ** -10         # q's elements under 2^-14 of its largest
        e_p = {"e4m3": 2.0 ** -10, "bf16": 2.0 ** -15, "f16": 2.0 ** -15}[self.pool_type]
        if self.latent:
            e_p = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10}[self.pool_type]
        tol = UNIT[self.qtype] * np.abs(ref) + \
            (e_p + 2 * d[..., None] + n * 2.0 ** -22) * size + \
            (2.0 ** -24 if self.qtype == "f16" else 0)
        got = out.double().cpu().numpy().reshape(ref.shape)
        assert np.isfinite(got).all()
        off = np.abs(got - ref) - tol
        assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
        if lse is not None:
            got = lse.double().cpu().numpy().reshape(rlse.shape)
            none = np.isinf(rlse)
            np.testing.assert_array_equal(got[none], rlse[none])
            ref_rows = ref[none]
            assert not ref_rows.any()
            bound = 2 * d + (np.abs(np.where(none, 0, rlse)) + 24) * 2.0 ** -22 + n * 2.0 ** -22
            assert (np.abs(got[~none] - rlse[~none]) <= bound[~none]).all()

    def attend(self, scale=None, window=0, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        out, lse = self.cache.attend(self.layer, self.q, self.dlen, self.dtable, scale=scale,
                                     window=window, **kw)
        self.cache.check()
        self.check(out, lse, scale, window)
        return out, lse


ATTEND = [
    # lengths, kw, window
    ([1], {}, 0), ([0], {}, 0), ([2, 0, 1, 17], dict(new=3), 0),
    ([100], dict(heads=2, queries=2, dim=64, pool="f16", block=32), 0),
    ([300, 5, 64], dict(heads=2, queries=8, dim=128, block=16), 0),
    ([300, 5, 64], dict(heads=2, queries=8, dim=128, block=5), 0),
    ([129, 128, 127], dict(heads=3, queries=15, dim=96, block=24), 0),
    ([77, 200], dict(heads=1, queries=16, dim=256, block=64), 0),
    ([77, 200], dict(heads=1, queries=40, dim=256, block=1), 0),
    ([500], dict(heads=1, queries=33, dim=128, block=8), 0),
    ([31, 65], dict(heads=2, queries=32, dim=16, block=16, pool="f16"), 0),
    ([31, 65], dict(heads=1, queries=4, dim=80, block=48), 0),
    ([90, 1, 0, 260], dict(heads=2, queries=16, dim=128, new=4, block=32), 0),
    ([90, 1, 0, 260], dict(heads=2, queries=16, dim=128, new=4, block=32), 50),
    ([90, 3, 700], dict(heads=1, queries=8, dim=128, new=2, block=32), 1),
    ([90, 3, 700], dict(heads=1, queries=8, dim=64, new=2, block=7), 333),
    ([700, 30], dict(heads=1, queries=4, dim=128, new=9), 64),
    ([260, 33, 1], dict(heads=2, queries=8, dim=128, pool="e4m3", block=32), 0),
    ([260, 33, 1], dict(heads=2, queries=8, dim=64, pool="e4m3", block=16), 0),
    ([260, 33, 1], dict(heads=2, queries=48, dim=256, pool="e4m3", block=16), 100),
    ([130], dict(heads=1, queries=8, dim=96, pool="e4m3", qtype="f16", block=3, new=2), 0),
    ([140, 60], dict(heads=2, queries=6, dim=160, pool="e4m3", per_head=True), 0),
]


@pytest.mark.parametrize("lengths, kw, window", ATTEND)
def test_attend(lengths, kw, window):
    Case(3, lengths, **kw).attend(window=window)


LATENT = [
    ([1], dict(queries=16), 0), ([0, 40], dict(queries=16), 0), ([31, 32, 33, 64, 65], dict(queries=128), 0),
    ([500, 3], dict(queries=16, new=2, block=64), 0), ([300], dict(queries=80, new=2), 0),
    ([257, 0, 1, 90], dict(queries=8, new=3, block=8), 0), ([200, 70], dict(queries=32, block=5), 0),
    ([200, 70], dict(queries=32, block=24), 40), ([400, 31], dict(queries=16, new=4, block=32), 100),
    ([300, 100], dict(queries=40, pool="f16", block=128), 0), ([90], dict(queries=1, block=1), 0),
]


@pytest.mark.parametrize("lengths, kw, window", LATENT)
def test_attend_latents(lengths, kw, window):
    Case(4, lengths, dim=576, **kw).attend(scale=192.0 ** -0.5, window=window)


def test_many_parts_of_one_request_are_joined():
    """Long enough that its keys are cut among many blocks; and few, many and mixed requests."""
    for kw in (dict(heads=1, queries=4, dim=64), dict(heads=2, queries=4, dim=64, pool="e4m3", block=64),
               dict(dim=576, queries=8, block=64)):
        c = Case(5, [6000], **kw)
        c.attend(scale=0.1)
    Case(6, [3000, 1, 0, 2000, 17, 900], heads=1, queries=16, dim=64, new=2).attend()
    Case(6, [3000, 1, 0, 2000, 17, 900], dim=576, queries=16, new=2).attend(scale=0.07)


DIVIDED = [
    ([2000] * 9, dict(heads=2, queries=4, dim=64)),
    ([4100, 3, 0, 900, 2048], dict(heads=2, queries=8, dim=128, new=2)),
    ([60000, 1, 30000], dict(heads=1, queries=2, dim=64, pool="f16", block=64)),
    ([97 * k % 701 for k in range(128)], dict(heads=1, queries=2, dim=64)),
    ([97 * k % 701 for k in range(129)], dict(heads=1, queries=2, dim=64)),
    ([97 * k % 701 for k in range(128)], dict(heads=3, queries=3, dim=64)),
    ([0] * 20 + [5000], dict(heads=2, queries=4, dim=64)),
    ([1300, 0, 40, 2500, 7, 1280], dict(dim=576, queries=16)),
    ([640] * 19, dict(dim=576, queries=16, block=64)),
    ([97 * k % 301 for k in range(75)], dict(dim=576, queries=4)),
    ([97 * k % 301 for k in range(130)], dict(dim=576, queries=4)),
    ([2100, 700], dict(dim=576, queries=100, new=2, pool="f16")),
    ([97 * k % 601 for k in range(40)], dict(dim=576, queries=64)),
]


@pytest.mark.parametrize("lengths, kw", DIVIDED)
def test_jobs_of_all_sizes_are_divided_and_joined(lengths, kw):
    """Few long jobs and many short ones: parts that end with jobs, and parts that do not."""
    Case(61, lengths, **kw).attend()


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16)])
def test_the_first_call_may_be_captured(kw):
    """Nothing is left for a first launch that a graph's capture would not allow."""
    import torch
    case = Case(67, [700, 33, 2100], **kw)
    scale = case.D ** -0.5
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=scale)
        one = case.cache.attend(0, case.q[:1], case.dlen[:1], case.dtable[:1], scale=scale)
    graph.replay()
    case.cache.check()
    case.check(out, lse, scale, 0)
    case.check(one[0], one[1], scale, 0, first=1)


def test_most_requests_of_one_call():
    import torch
    lengths = [(7 * r) % 5 for r in range(2048)]
    for kw in (dict(heads=1, queries=1, dim=16, block=4), dict(dim=576, queries=1, block=8)):
        c = Case(8, lengths, **kw)
        c.attend(scale=0.2)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kw", [dict(heads=2, queries=16, dim=128), dict(heads=2, queries=16, dim=128, pool="f16"),
                                dict(heads=1, queries=8, dim=64, pool="e4m3"), dict(dim=576, queries=16),
                                dict(dim=576, queries=16, pool="f16")])
def test_peaked_and_growing_logits(kw):
    """Keys whose logits grow along the request, by far more than 2^8 from tile to tile (the running
    maximum has to move each time), then shrink again; and a negative scale."""
    c = Case(9, [400, 170], **kw)
    n = c.wide.shape[3]
    ramp = {0: 0.02, 1: 0.2}
    for r, length in enumerate(c.lengths):
        for j in range(length):
            f = ramp[r] * (j if j < length // 2 else length - j)
            at = (slice(None), slice(None), int(c.table[r, j // n]), j % n)
            if c.pool_type == "e4m3":
                continue
            c.host[at] = (c.host[at].float() * f).to(c.host.dtype)
    c.dev.copy_(c.host)
    if c.pool_type != "e4m3":
        c.wide = c.host.double().numpy()
    for scale in (0.5, -0.5, 3.0):
        out, lse = c.cache.attend(0, c.q, c.dlen, c.dtable, scale=scale)
        c.cache.check()
        c.check(out, lse, scale, 0)


def test_infinite_logits_and_nan_keys_reach_their_own_rows_only():
    import torch
    c = Case(10, [40, 40], heads=2, queries=4, dim=64)
    b = int(c.table[0, 1])
    c.dev[0, 0, b, 3, 0] = float("nan")                        # request 0, head 0
    out, lse = c.cache.attend(0, c.q, c.dlen, c.dtable)
    torch.cuda.synchronize()
    out, lse = out.float(), lse
    assert torch.isnan(out[0, 0, :2]).all() and torch.isnan(lse[0, 0, :2]).all()
    assert torch.isfinite(out[0, 0, 2:]).all() and torch.isfinite(out[1]).all()
    c.dev[0, 0, b, 3, 0] = 0
    c.dev[0, 1, b, 3, 0] = float("inf")
    out, lse = c.cache.attend(0, c.q, c.dlen, c.dtable)
    assert torch.isinf(out[0, 0, :2].float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kw, size", [(dict(heads=2, queries=8, dim=64), 2.0 ** 105),
                                      (dict(dim=576, queries=16), 2.0 ** 95)])
def test_values_near_the_largest_stay_finite(kw, size):
    """Sums over keys may run ahead of the last maximum, but not beyond fp32."""
    import torch
    case = Case(71, [700, 2000], **kw)
    small = size ** -0.5 if case.latent else 1.0         # a latent is its own key
    dev = case.dev.double()
    dev = dev * size if case.latent else torch.stack([dev[:, 0], dev[:, 1] * size], 1)
    case.dev.copy_(dev.to(torch.bfloat16))
    case.wide = case.dev.double().cpu().numpy()
    case.q.copy_((case.q.double() * small).to(torch.bfloat16))
    scale = case.D ** -0.5 * (small if case.latent else 1.0)
    out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=scale)
    case.cache.check()
    case.check(out, lse, scale, 0)


def _padded(case):
    """Rows 48 bytes apart from each other's ends, heads before tokens, layers in tensors of their own."""
    import torch
    from prefill_decode_paged_gb300.kv_relayout import layout_of_views
    L, C, N, B, H, D = case.host.shape
    es = case.host.element_size()
    views = []
    for l in range(L):
        per = []
        for c in range(C):
            t = torch.zeros((N, H, B, D + 48 // es), dtype=case.host.dtype, device="cuda")
            v = t[..., :D].transpose(1, 2)                     # [block][token][head][dim]
            v.copy_(case.host[l, c])
            per.append(v)
        views.append(per)
    return views, layout_of_views([views])


@pytest.mark.parametrize("kw", [dict(heads=3, queries=6, dim=64), dict(heads=2, queries=2, dim=128, pool="e4m3"),
                                dict(dim=576, queries=16, block=8), dict(dim=576, queries=16, block=6)])
def test_strided_pools_and_layers(kw):
    for layer in (0, 1):
        Case(11, [90, 33], layers=2, layer=layer, layout=_padded, **kw).attend(scale=0.11)


def test_strided_queries_and_outputs():
    import torch
    for kw in (dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16)):
        c = Case(12, [70, 9], new=2, **kw)
        wide = torch.zeros((2, 2, c.Q + 3, c.D + 8), dtype=c.q.dtype, device="cuda")
        q = wide[:, :, 1:c.Q + 1, :c.D]
        q.copy_(c.q)
        room = torch.full((2, 2, c.Q, c.V + 16), 7.0, dtype=c.q.dtype, device="cuda")
        out, lse = c.cache.attend(0, q, c.dlen, c.dtable, scale=0.1, out=room[..., :c.V])
        c.cache.check()
        c.check(out, lse, 0.1, 0)
        assert (room[..., c.V:] == 7).all()
        # one new token: the token dimension may be left out; no lse
        d = Case(12, [70, 9], **kw)
        a, none = d.cache.attend(0, d.q[:, 0], d.dlen, d.dtable, scale=0.1, lse=False)
        assert none is None and a.shape == (2, d.Q, d.V)
        d.check(a, None, 0.1, 0)


def test_offsets_beyond_32_bits():
    """Blocks 1.5 GB apart, so that the last lie past 4 GB in either unit."""
    import torch
    from prefill_decode_paged_gb300 import KVCache
    stride, N, B, D = 3 << 29, 5, 16, 64
    big = torch.empty(N * stride, dtype=torch.uint8, device="cuda")
    small = Case(13, [80], heads=1, queries=4, dim=D, block=B)
    order = [4, 2, 0, 3, 1]
    views = []
    for c in range(2):
        v = big[c * (1 << 20):].view(torch.bfloat16).as_strided((N, B, 1, D), (stride // 2, D, D, 1))
        for k in range(5):
            v[order[k]] = small.dev[0, c, int(small.table[0, k])]
        views.append(v)
    cache = KVCache(None, num_layers=1, num_components=2, kv_heads=1, head_dim=D, block=B, num_blocks=N,
                    dtype=1, query_heads=4,
                    layout=dict(bases=views, block_stride=stride, token_stride=2 * D, head_stride=2 * D,
                                shape=(N, B, 1, D), elem_bytes=2))
    table = torch.tensor([order], dtype=torch.int32, device="cuda")
    out, lse = cache.attend(0, small.q, small.dlen, table)
    small.check(out, lse, D ** -0.5, 0)
    k = torch.randn((1, 1, D), device="cuda").bfloat16()
    pos = torch.tensor([16 * 3 + 5], dtype=torch.int32, device="cuda")
    cache.append(0, k, 2 * k, torch.zeros(1, dtype=torch.int32, device="cuda"), pos, table)
    cache.check()
    assert torch.equal(views[0][3, 5], k[0]) and torch.equal(views[1][3, 5], 2 * k[0])
    del big, views, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16)])
def test_results_do_not_depend_on_the_run(kw):
    """The same bits again and again, on a captured graph, on another stream, and after other
    calls of the cache in between; lengths come from the device when the graph is replayed."""
    import torch
    c = Case(14, [3000, 1200, 40], **kw)
    first, lse = c.attend(scale=0.1)
    for _ in range(5):
        again, lse2 = c.cache.attend(0, c.q, c.dlen, c.dtable, scale=0.1)
        assert torch.equal(again, first) and torch.equal(lse2, lse)
        c.cache.attend(0, c.q[:1], c.dlen[:1], c.dtable[:1], scale=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, l2 = torch.empty_like(first), torch.empty_like(lse)
    c.cache.attend(0, c.q, c.dlen, c.dtable, out=out, lse=l2, scale=0.1, stream=side)
    side.synchronize()
    assert torch.equal(out, first) and torch.equal(l2, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.cache.attend(0, c.q, c.dlen, c.dtable, out=out, lse=l2, scale=0.1)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    c.lengths = [700, 0, 33]
    c.dlen.copy_(torch.tensor(c.lengths, dtype=torch.int32))
    graph.replay()
    c.cache.check()
    c.check(out, l2, 0.1, 0)


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16)])
def test_a_stream_with_fewer_sms(kw):
    from prefill_decode_paged_gb300 import SmStream
    import torch
    c = Case(15, [2500, 100], **kw)
    torch.cuda.synchronize()
    with SmStream(16) as s:
        out, lse = c.cache.attend(0, c.q, c.dlen, c.dtable, scale=0.1, stream=s.handle)
        torch.cuda.synchronize()
        c.cache.check()
        c.check(out, lse, 0.1, 0)


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16),
                                dict(dim=576, queries=16, block=5)])
def test_bad_lengths_and_blocks_are_flagged_and_not_read(kw):
    import torch
    from prefill_decode_paged_gb300 import KVRelayoutError
    c = Case(16, [50, 90, 20], **kw)
    good, _ = c.attend(scale=0.1)
    for bad_len in (-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        lens = c.dlen.clone()
        lens[2] = bad_len
        out, lse = c.cache.attend(0, c.q, lens, c.dtable, scale=0.1)
        with pytest.raises(KVRelayoutError, match="length") as e:
            c.cache.check()
        assert e.value.name == "KVR_ERR_DEVICE_BOUNDS"
        # (another length cuts the others' keys elsewhere: the same values, not the same bits)
        c.check(out[:2], lse[:2], 0.1, 0, first=2)
    for bad_id in (-1, c.N, 2 ** 31 - 1, -2 ** 31):
        table = c.dtable.clone()
        table[1, 2] = bad_id
        out, _ = c.cache.attend(0, c.q, c.dlen, table, scale=0.1)
        with pytest.raises(KVRelayoutError, match="block id"):
            c.cache.check()
        assert torch.isfinite(out[1].float()).all()
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    c.cache.check()                                            # cleared


def test_attend_refusals():
    import torch
    from prefill_decode_paged_gb300 import KVRelayoutError
    c = Case(17, [20, 30], heads=2, queries=8, dim=64, new=2)
    call = c.cache.attend

    def status(*a, **kw):
        with pytest.raises(KVRelayoutError) as e:
            call(*a, **kw)
        return e.value.name
    assert status(1, c.q, c.dlen, c.dtable) == "KVR_ERR_LAYER_RANGE"
    assert status(-1, c.q, c.dlen, c.dtable) == "KVR_ERR_LAYER_RANGE"
    assert status(0, c.q, c.dlen, c.dtable, window=-1) == "KVR_ERR_INVALID_ARG"
    assert status(0, c.q, c.dlen, c.dtable, scale=math.inf) == "KVR_ERR_INVALID_ARG"
    assert status(0, c.q, c.dlen, c.dtable[:1]) == "KVR_ERR_INVALID_ARG"
    three = torch.cat([c.q, c.q])[:3]
    assert status(0, three, torch.cat([c.dlen, c.dlen])[:3], torch.cat([c.dtable] * 2)) == \
        "KVR_ERR_INVALID_ARG"                                  # more than max_requests
    assert status(0, torch.cat([c.q, c.q], 1), c.dlen, c.dtable) == "KVR_ERR_INVALID_ARG"
    assert status(0, c.q.half(), c.dlen, c.dtable) == "KVR_ERR_UNSUPPORTED"
    off = torch.zeros(c.q.numel() + 4, dtype=c.q.dtype, device="cuda")[4:].view(c.q.shape)
    assert status(0, off, c.dlen, c.dtable) == "KVR_ERR_ALIGNMENT"
    for a in ((c.q.cpu(), c.dlen, c.dtable), (c.q[..., :32], c.dlen, c.dtable),
              (c.q.float(), c.dlen, c.dtable), (c.q, c.dlen.long(), c.dtable), (c.q, c.dlen[:1], c.dtable),
              (c.q, c.dlen, c.dtable.long()), (c.q, c.dlen, c.dtable.t()), (c.q[0, 0], c.dlen, c.dtable)):
        with pytest.raises(ValueError):
            call(0, *a)
    with pytest.raises(ValueError):
        call(0, c.q, c.dlen, c.dtable, lse=torch.zeros(3, device="cuda"))
    empty = c.q[:0]
    out, lse = call(0, empty, c.dlen[:0], c.dtable)
    assert out.shape[0] == 0
    c.attend()
    c.cache.close()
    with pytest.raises(RuntimeError):
        call(0, c.q, c.dlen, c.dtable)


# -- append ------------------------------------------------------------------------------

APPEND = [
    # heads, queries, dim, qdim, rotated, interleaved, last, pool, type, block
    (8, 32, 128, 128, 128, False, False, "bf16", "bf16", 16),
    (2, 5, 64, 64, 32, False, True, "f16", "f16", 5),
    (2, 4, 96, 96, 48, True, False, "bf16", "bf16", 24),
    (1, 3, 256, 256, 256, True, True, "f16", "f16", 1),
    (1, 16, 576, 64, 64, True, True, "bf16", "bf16", 16),
    (1, 2, 576, 576, 64, False, True, "f16", "f16", 64),
    (3, 6, 128, 128, 64, False, False, "e4m3", "bf16", 32),
    (2, 2, 64, 64, 64, True, False, "e4m3", "f16", 8),
    (4, 0, 16, 0, 16, False, False, "bf16", "bf16", 4),
    (2, 0, 48, 0, 0, False, False, "bf16", "bf16", 16),
]


@pytest.mark.parametrize("tokens", [1, 37, 300])
@pytest.mark.parametrize("H, Q, D, QD, rot, il, last, pool, dtype, B", APPEND)
def test_append(H, Q, D, QD, rot, il, last, pool, dtype, B, tokens):
    """Rows against 64 bits, rounded once (E4M3: to a neighbour in the format, the nearer but for
    products that lie within fp32's error of the middle); everything else in the pool unchanged."""
    import torch
    from prefill_decode_paged_gb300 import KVCache, rotary_table
    rng = np.random.default_rng(tokens + D)
    C = 1 if D == 576 else 2
    R, width = 4, 300 // B + 2
    N = R * width + 2
    table = rng.permutation(N)[:R * width].reshape(R, width).astype(np.int32)
    slots = rng.permutation(R * 300)[:tokens]
    req, pos = (slots // 300).astype(np.int32), (slots % 300).astype(np.int32)
    pad = rng.random(tokens) < 0.1
    pad[0] = False
    pos[pad] = -1 - (pos[pad] % 3)
    es = 1 if pool == "e4m3" else 2
    sentinel = torch.from_numpy(rng.integers(0, 256, (2, C, N, B, H, D * es), dtype=np.uint8)).cuda()
    dev = sentinel.clone()
    pool_t = dev if es == 1 else dev.view(torch_type(pool))
    scales = rng.uniform(0.004, 0.02, (2, C)).astype(np.float32) if pool == "e4m3" else None
    cache = KVCache(pool_t, num_layers=2, num_components=C, kv_heads=H, head_dim=D, block=B,
                    num_blocks=N, dtype=TYPES[pool], scales=scales)
    tt = torch_type(dtype)
    # rows of a packed projection: strides of their own
    packed = torch.from_numpy(rng.standard_normal((tokens, 2 * H + 1, D))).to(tt).cuda()
    k, v = packed[:, :H], packed[:, H:2 * H]
    q = torch.from_numpy(rng.standard_normal((tokens, Q, QD))).to(tt).cuda() if Q else None
    angles = rotary_table(300, rot, 10000.0) if rot else None
    dangles = torch.from_numpy(angles).cuda() if rot else None
    dreq, dpos, dtab = (torch.from_numpy(x).cuda() for x in (req, pos, table))
    keep = torch.full_like(q, 5.0) if Q else None
    out = cache.append(1, k, v if C == 2 else None, dreq, dpos, dtab, rotary=dangles, interleaved=il,
                       rotate_last=last, q=q, q_out=keep)
    cache.check()
    turned = {0: k.double().cpu().numpy(), 1: v.double().cpu().numpy()}
    if rot:
        turned[0] = cache_ref.rotate(turned[0], pos, angles, rot, il, last)
    expect = sentinel.cpu().clone()
    got = dev.cpu()
    u = UNIT["f16"] if pool == "f16" else UNIT["bf16"]
    grid = cache_ref.e4m3_grid()
    for t in range(tokens):
        if pos[t] < 0:
            continue
        b, s = table[req[t], pos[t] // B], pos[t] % B
        for c in range(C):
            row = got[1, c, b, s]
            expect[1, c, b, s] = row
            ref = turned[c][t]
            if pool == "e4m3":
                x = np.clip(ref * float(np.float32(1) / scales[1, c]), -448, 448)
                y = cache_ref.decode_e4m3(row.numpy())
                near = np.abs(grid[None, None] - x[..., None]).min(-1)
                assert (np.abs(y - x) <= near + 2.0 ** -21 * (np.abs(x) + 1)).all()
            else:
                y = row.view(torch_type(pool)).double().numpy()
                # one rounding, and three fp32 operations on values of at most |a| + |b| <= 12
                assert (np.abs(y - ref) <= u * np.abs(ref) + 12 * 2.0 ** -22 + 2.0 ** -25).all()
                if c == 1 or rot == 0:
                    np.testing.assert_array_equal(y, ref)
    assert torch.equal(got, expect)                            # nothing else was written
    if Q:
        ref = cache_ref.rotate(q.double().cpu().numpy(), pos, angles, rot, il, last)
        y = out.double().cpu().numpy()
        live = pos >= 0
        assert (np.abs(y - ref)[live] <= UNIT[dtype] * np.abs(ref)[live] + 12 * 2.0 ** -22 + 2.0 ** -25).all()
        assert (y[~live] == 5.0).all()
        again = cache.append(1, k, v if C == 2 else None, dreq, dpos, dtab, rotary=dangles,
                             interleaved=il, rotate_last=last, q=q, q_out=q)
        assert again is q and torch.equal(q[torch.from_numpy(live)], out[torch.from_numpy(live)])


@pytest.mark.parametrize("H, Q, D, QD, rot, il, last, pool, dtype, B, tokens",
                         [c + (1100,) for c in APPEND] +
                         [APPEND[0] + (6000,), (8, 32, 128, 128, 64, True, False, "e4m3", "f16", 32, 6000)])
def test_append_of_many_tokens_is_that_of_few(H, Q, D, QD, rot, il, last, pool, dtype, B, tokens):
    """Bit for bit: what one call writes, calls of 150 of its tokens write."""
    import torch
    from prefill_decode_paged_gb300 import KVCache, rotary_table
    C, R = (1 if D == 576 else 2), 4
    each = tokens // R
    width = each // B + 1
    gen = torch.Generator("cuda").manual_seed(tokens + D)
    order = torch.randperm(R * width, device="cuda", generator=gen).int()
    table = order.view(R, width)
    req = torch.arange(R, device="cuda").repeat_interleave(each).int()
    pos = torch.arange(each, device="cuda").repeat(R).int()
    mixed = torch.randperm(R * each, device="cuda", generator=gen)
    req, pos = req[mixed].contiguous(), pos[mixed].contiguous()
    pos[::17] = -1
    T, tt = R * each, torch_type(dtype)
    k, v, q = (torch.randn(T, h, d, device="cuda", generator=gen).to(tt) for h, d in ((H, D), (H, D), (Q, QD)))
    angles = torch.from_numpy(rotary_table(each, rot, 10000.0)).cuda() if rot else None
    kw = dict(rotary=angles, interleaved=il, rotate_last=last)
    results = []
    for step in (T, 150):
        shape = (1, C, R * width, B, H, D)
        dev = torch.full(shape, 7, dtype=torch.uint8, device="cuda") if pool == "e4m3" else \
            torch.full(shape, 7.0, dtype=torch_type(pool), device="cuda")
        out = torch.full_like(q, 5.0) if Q else None
        with KVCache(dev, num_layers=1, num_components=C, kv_heads=H, head_dim=D, block=B,
                     num_blocks=R * width, dtype=TYPES[pool],
                     scales=np.full((1, C), 0.02, np.float32) if pool == "e4m3" else None) as cache:
            for a in range(0, T, step):
                b = min(T, a + step)
                cache.append(0, k[a:b], v[a:b] if C == 2 else None, req[a:b], pos[a:b], table,
                             q=q[a:b] if Q else None, q_out=out[a:b] if Q else None, **kw)
            cache.check()
        results.append((dev, out))
    assert torch.equal(results[0][0].view(torch.uint8), results[1][0].view(torch.uint8))
    if Q:
        assert torch.equal(results[0][1].view(torch.uint8), results[1][1].view(torch.uint8))


def test_append_nan_and_saturation_in_eight_bits():
    import torch
    from prefill_decode_paged_gb300 import KVCache
    pool = torch.zeros((1, 2, 2, 4, 1, 16), dtype=torch.uint8, device="cuda")
    cache = KVCache(pool, num_layers=1, num_components=2, kv_heads=1, head_dim=16, block=4, num_blocks=2,
                    dtype=2, scales=np.array([[0.5, 2.0]]))
    x = torch.zeros((1, 1, 16), device="cuda")
    x[0, 0, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 300.0, -300.0, 1.0, -0.0, 2.0 ** -11])
    i32 = dict(dtype=torch.int32, device="cuda")
    cache.append(0, x.bfloat16(), x.bfloat16(), torch.zeros(1, **i32), torch.tensor([5], **i32),
                 torch.tensor([[0, 1]], **i32))
    cache.check()
    k, v = pool[0, 0, 1, 1, 0, :8].tolist(), pool[0, 1, 1, 1, 0, :8].tolist()
    assert k[0] & 0x7F == 0x7F and v[0] & 0x7F == 0x7F
    assert k[1:] == [0x7E, 0xFE, 0x7E, 0xFE, 0x40, 0x80, 0x00] or k[1:] == [0x7E, 0xFE, 0x7E, 0xFE, 0x40, 0x80, 0x01]
    assert [cache_ref.decode_e4m3(c) for c in v[1:5]] == [448, -448, 144, -144] or \
        [cache_ref.decode_e4m3(c) for c in v[1:5]] == [448, -448, 152, -152]


def test_append_flags_what_is_out_of_range_and_writes_none_of_it():
    import torch
    from prefill_decode_paged_gb300 import KVCache, KVRelayoutError, rotary_table
    rng = np.random.default_rng(1)
    pool = torch.from_numpy(rng.standard_normal((1, 2, 6, 4, 2, 32))).bfloat16().cuda()
    before = pool.clone()
    cache = KVCache(pool, num_layers=1, num_components=2, kv_heads=2, head_dim=32, block=4, num_blocks=6, dtype=1)
    k = torch.ones((1, 2, 32), dtype=torch.bfloat16, device="cuda")
    angles = torch.from_numpy(rotary_table(10, 32)).cuda()
    table = torch.tensor([[0, 1, 2, 9], [3, -1, 6, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")

    def call(r, p, **kw):
        i32 = dict(dtype=torch.int32, device="cuda")
        cache.append(0, k, k, torch.tensor([r], **i32), torch.tensor([p], **i32), table, **kw)
    for r, p, kw, word in ((-1, 0, {}, "request"), (2, 0, {}, "request"), (0, 16, {}, "position"),
                           (0, 2 ** 31 - 1, {}, "position"), (0, 10, dict(rotary=angles), "position"),
                           (0, 12, {}, "block id"), (1, 4, {}, "block id"), (1, 8, {}, "block id"),
                           (1, 12, {}, "block id")):
        call(r, p, **kw)
        with pytest.raises(KVRelayoutError, match=word):
            cache.check()
        assert torch.equal(pool, before)
    call(0, -5)
    cache.check()
    assert torch.equal(pool, before)
    call(1, 3)
    cache.check()
    assert torch.equal(pool[0, 0, 3, 3], k[0])


def test_append_refusals():
    import torch
    from prefill_decode_paged_gb300 import KVCache, KVRelayoutError, rotary_table
    pool = torch.zeros((1, 2, 6, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache = KVCache(pool, num_layers=1, num_components=2, kv_heads=2, head_dim=64, block=4, num_blocks=6, dtype=1)
    k = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    rot = torch.from_numpy(rotary_table(8, 64)).cuda()

    def status(*a, **kw):
        with pytest.raises(KVRelayoutError) as e:
            cache.append(*a, **kw)
        return e.value.name
    assert status(1, k, k, n, n, table) == "KVR_ERR_LAYER_RANGE"
    assert status(0, k.half(), k.half(), n, n, table) == "KVR_ERR_UNSUPPORTED"
    assert status(0, k, k, n, n, table, q=k) == "KVR_ERR_INVALID_ARG"          # queries, no angles
    assert status(0, k, k, n, n, table, rotary=rot[:, :24].contiguous()) == "KVR_ERR_UNSUPPORTED"
    wide = torch.from_numpy(rotary_table(8, 128)).cuda()
    assert status(0, k, k, n, n, table, rotary=wide) == "KVR_ERR_UNSUPPORTED"
    assert status(0, k, k, n, n, table, rotary=rot, q=k[..., :40].contiguous()) == "KVR_ERR_UNSUPPORTED"
    off = torch.zeros(k.numel() + 4, dtype=k.dtype, device="cuda")[4:].view(k.shape)
    assert status(0, off, k, n, n, table) == "KVR_ERR_ALIGNMENT"
    assert status(0, k, off, n, n, table) == "KVR_ERR_ALIGNMENT"
    assert status(0, k, k, n, n, table, rotary=rot, q=off) == "KVR_ERR_ALIGNMENT"
    for bad in ((k, None, n, n, table), (k[..., :32], k, n, n, table), (k, k[:2], n, n, table),
                (k, k, n[:2], n, table), (k, k, n, n.long(), table), (k, k, n, n, table[0]),
                (k.cpu(), k, n, n, table)):
        with pytest.raises(ValueError):
            cache.append(0, *bad)
    with pytest.raises(ValueError):
        cache.append(0, k, k, n, n, table, rotary=rot.double())
    with pytest.raises(KVRelayoutError) as e:                 # this cache only appends
        cache.attend(0, k[:, :0], n, table)
    assert e.value.name == "KVR_ERR_UNSUPPORTED"
    assert cache.append(0, k[:0], k[:0], n[:0], n[:0], table) is None


def test_appended_rows_are_what_attention_reads():
    """Append token by token and attend at each step: the same as attending to a pool that held
    them all along."""
    import torch
    full = Case(21, [37], heads=2, queries=8, dim=64, block=8)
    empty = Case(21, [37], heads=2, queries=8, dim=64, block=8)
    empty.dev.fill_(float("nan"))
    i32 = dict(dtype=torch.int32, device="cuda")
    for p in range(37):
        b, s = int(full.table[0, p // 8]), p % 8
        empty.cache.append(0, full.dev[0, 0, b, s][None], full.dev[0, 1, b, s][None], torch.zeros(1, **i32),
                           torch.tensor([p], **i32), empty.dtable)
        n = torch.tensor([p + 1], **i32)
        a = full.cache.attend(0, full.q, n, full.dtable)
        b = empty.cache.attend(0, full.q, n, empty.dtable)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    empty.cache.check()
