"""Pools of every type with NaN everywhere but at the requests' own tokens, for the cache's further calls (tests only).

Tolerances are ``test_gpu_cache``'s: an output is rounded once (u), P before its product (e_p: two 16-bit
numbers 2^-15, one f16 2^-10), a logit is off by d (``cache_more_ref.scores``), sums over keys add 2^-22 a key."""
import numpy as np
import torch

import cache_more_ref as ref
from test_gpu_cache import Case, TYPES, UNIT, torch_type


class More(Case):
    """``Case`` with 4-bit pools among its types."""

    def __init__(self, seed, lengths, *, heads=1, queries=8, dim=128, block=16, new=1, pool="bf16", qtype=None,
                 layers=1, layer=0, per_head=True, layout=None, scaled=True, spread=1.0, max_requests=None):
        self.heads = heads
        if pool != "e2m1":
            super().__init__(seed, lengths, heads=heads, queries=queries, dim=dim, block=block, new=new, pool=pool,
                             qtype=qtype, layers=layers, layer=layer, per_head=per_head, layout=layout, spread=spread,
                             max_requests=max_requests)
            return
        from prefill_decode_paged_gb300 import KVCache
        # the queries, table and lengths of a pool of 16 bits
        super().__init__(seed, lengths, heads=heads, queries=queries, dim=dim, block=block, new=new, pool="bf16",
                         qtype=qtype, layers=layers, layer=layer, spread=spread)
        self.cache.close()
        rng = np.random.default_rng(seed + 1)
        shape = (layers, 2, self.N, block, heads, dim)
        self.pool_type = "e2m1"
        self.scales = rng.uniform(0.5, 2.0, (layers, 2, heads)).astype(np.float32) if scaled else None
        codes = rng.integers(0, 256, shape[:-1] + (dim // 2,)).astype(np.uint8)
        scales = rng.integers(0x28, 0x40, shape[:-1] + (dim // 16,)).astype(np.uint8)
        used = ~np.isnan(self.wide[..., :1])                     # the requests' own tokens
        scales = np.where(used, scales, 0x7F).astype(np.uint8)
        self.codes, self.block_scales = codes, scales
        self.settle()
        geometry = dict(num_layers=layers, num_components=2, kv_heads=heads, head_dim=dim, block=block,
                        num_blocks=self.N, dtype=5, scales=self.scales, per_head=per_head, query_heads=queries,
                        max_requests=max_requests or len(lengths), max_new=new)
        if layout is None:
            self.dev = torch.from_numpy(np.concatenate([codes.reshape(-1), scales.reshape(-1)])).cuda()
            self.cache = KVCache(self.dev, **geometry)
        else:
            self.dev, lay, more = layout(self)
            self.cache = KVCache(None, layout=lay, block_scales=more, **geometry)

    def settle(self):
        """What the codes stand for."""
        with np.errstate(invalid="ignore"):
            self.wide = ref.values(self.codes, self.block_scales)
        if self.scales is not None:
            self.wide = self.wide * self.scales.astype(np.float64)[:, :, None, None, :, None]

    def reference(self, scale, window, cap, slopes, first=None, lse_in=None, width=None):
        s = None if slopes is None else slopes.double().cpu().numpy()
        return ref.attend(self.q[:first].double().cpu().numpy(), self.rows_of, self.lengths[:first], scale, window,
                          cap, s, width, self.Q // self.H, lse_in)

    def check_scored(self, out, lse, scale, window=0, cap=0.0, slopes=None, first=None):
        want = self.reference(scale, window, cap, slopes, first)
        n, d, size = max(self.lengths + [1]), want["off"], want["size"]
        coded = self.pool_type in ("e4m3", "e2m1")
        if coded:
            # elements of q below 2^-14 of its largest become multiples of 2^-24 of it
            qs = np.abs(self.q[:first].double().cpu().numpy()).max(-1)
            d = d + 2.0 ** -24 * qs * abs(scale) * np.nan_to_num(np.abs(self.wide)).max() * self.D
        e_p = 2.0 ** -10 if coded else 2.0 ** -15
        tol = UNIT[self.qtype] * np.abs(want["out"]) + (e_p + 2 * d[..., None] + n * 2.0 ** -22) * size + \
            (2.0 ** -24 if self.qtype == "f16" else 0)
        if coded or self.pool_type == "f16":
            # P is f16 of 2^10 times a weight: spaced 2^-24 where it is smallest, so a weight is off by 2^-35 of
            # the row's largest, whatever its own size
            tol = tol + 2.0 ** -35 * want["total"]
        got = out.double().cpu().numpy().reshape(want["out"].shape)
        assert np.isfinite(got).all()
        off = np.abs(got - want["out"]) - tol
        assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
        if lse is not None:
            got, rlse = lse.double().cpu().numpy().reshape(want["lse"].shape), want["lse"]
            none = np.isinf(rlse)
            np.testing.assert_array_equal(got[none], rlse[none])
            assert not want["out"][none].any()
            bound = 2 * d + (np.abs(np.where(none, 0, rlse)) + 24) * 2.0 ** -22 + n * 2.0 ** -22
            assert (np.abs(got[~none] - rlse[~none]) <= bound[~none]).all()

    def attend_scored(self, scale=None, window=0, cap=0.0, slopes=None, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        more = dict(cap=cap, slopes=slopes) if cap or slopes is not None else {}
        out, lse = self.cache.attend(self.layer, self.q, self.dlen, self.dtable, scale=scale, window=window,
                                     **more, **kw)
        self.cache.check()
        self.check_scored(out, lse, scale, window, cap, slopes)
        return out, lse


assert TYPES and torch_type      # (re-exported to the test files)
