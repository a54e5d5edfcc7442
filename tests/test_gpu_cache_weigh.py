"""Attention weights of cached keys on the GPU, against 64 bits.

Tolerance: each exponential by its score's and its lse's error (``cache_more_ref``), their sum by one fp32 rounding
a row, and one more where it is added to what was there."""
import numpy as np
import pytest
import torch

from cache_more_case import More
from prefill_decode_paged_gb300 import KVRelayoutError
from test_gpu_cache_scores import slopes_of

pytestmark = pytest.mark.gpu


def check(case, got, old, lse, scale, window=0, cap=0.0, slopes=None, add=True, first=None):
    """``got`` and ``old`` [R][H][S]: old where nothing was cached, old + w (w) elsewhere."""
    S = got.shape[2]
    width = max(S, max(case.lengths + [1]))
    z = lse.double().cpu().numpy().reshape(lse.shape[0], case.new, case.Q)
    want = case.reference(scale, window, cap, slopes, first, z, width)
    w, off = want["weights"][..., :S], want["weights_off"][..., :S]
    if case.pool_type in ("e4m3", "e2m1"):
        # elements of q below 2^-14 of its largest become multiples of 2^-24 of it
        qs = float(case.q[:first].abs().max())
        off = off + w * 2.0 ** -24 * qs * abs(scale) * np.nan_to_num(np.abs(case.wide)).max() * case.D
    rows = case.new * case.Q // case.H
    off = off + (rows + 4) * 2.0 ** -24 * w + 2.0 ** -126
    old, got = old.double().cpu().numpy(), got.double().cpu().numpy()
    held = np.arange(S)[None, None, :] < np.array(case.lengths[:first])[:, None, None]
    base = old if add else np.zeros_like(old)
    target = np.where(held, base + w, old)
    bound = np.where(held, off + (2.0 ** -24 * np.abs(target) if add else 0), 0)
    assert np.isfinite(got).all()
    over = np.abs(got - target) - bound
    assert over.size == 0 or over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))
    return want


def weigh(case, scale=None, window=0, cap=0.0, slopes=None, add=True, extra=3):
    scale = case.D ** -0.5 if scale is None else scale
    kw = dict(scale=scale, window=window, cap=cap, slopes=slopes)
    _, lse = case.cache.attend(case.layer, case.q, case.dlen, case.dtable, **kw)
    gen = torch.Generator("cuda").manual_seed(3)
    R = len(case.lengths)
    old = torch.rand((R, case.H, max(case.lengths + [0]) + extra), generator=gen, device="cuda")
    got = case.cache.weigh(case.layer, case.q, lse, case.dlen, case.dtable, old.clone(), add=add, **kw)
    case.cache.check()
    check(case, got, old, lse, scale, window, cap, slopes, add)
    return got, lse


CASES = [
    # lengths, kw, window
    ([1], {}, 0), ([0], {}, 0), ([2, 0, 1, 17], dict(new=3), 0), ([300, 5, 64], dict(heads=2, queries=8, block=5), 0),
    ([129, 128, 127], dict(heads=3, queries=15, dim=64, block=24), 0), ([77, 200], dict(queries=16, dim=256, block=64), 0),
    ([77, 200], dict(heads=2, queries=80, dim=192, block=1), 0), ([500], dict(queries=33, block=8), 0),
    ([90, 1, 0, 260], dict(heads=2, queries=16, new=4, block=32), 50), ([90, 3, 700], dict(queries=3, new=2, block=7), 333),
    ([700, 30], dict(queries=4, dim=64, new=9), 64), ([6000], dict(heads=2, queries=4, dim=64, block=64), 0),
    ([3000, 1, 0, 2000, 17, 900], dict(queries=16, dim=64, new=2), 0), ([300, 17, 0, 64], dict(queries=2, new=40), 33),
    ([97 * k % 701 for k in range(129)], dict(heads=1, queries=2, dim=64), 0), ([200], dict(queries=8, new=200), 0),
    ([200, 130], dict(queries=8, dim=256, new=30), 0), ([2000] * 9, dict(heads=2, queries=12, dim=64), 0),
]


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("lengths, kw, window", CASES)
def test_weigh(lengths, kw, window, pool):
    case = More(71, lengths, pool=pool, **kw)
    weigh(case, window=window, add=True)
    weigh(case, window=window, add=False, extra=0)


@pytest.mark.parametrize("dim", [16, 96, 160])
def test_head_sizes_of_other_pools(dim):
    for pool in ("bf16", "f16", "e4m3"):
        weigh(More(72, [150, 33], heads=2, queries=4, dim=dim, pool=pool, block=7), window=70)


@pytest.mark.parametrize("pool", ["bf16", "e2m1"])
def test_scores_of_other_forms(pool):
    case = More(73, [300, 1, 0, 90], heads=2, queries=8, dim=64, new=2, pool=pool)
    for cap, slopes in ((3.0, None), (0.0, "mixed"), (1.0, "powers")):
        weigh(case, cap=cap, slopes=slopes_of(case, slopes), window=40)
        weigh(case, cap=cap, slopes=slopes_of(case, slopes), add=False)


def test_rows_without_a_sum_or_without_keys_give_nothing():
    case = More(74, [40, 0, 2], heads=2, queries=4, dim=64, new=3)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    assert torch.isinf(lse[1]).all() and torch.isinf(lse[2, 0]).all()
    lse[0, :, 1] = -float("inf")
    old = torch.rand((3, 2, 44), device="cuda")
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    assert torch.isfinite(got).all() and torch.equal(got[1], old[1])
    case.q[0, :, 1] = 0                                          # (what its scores are does not matter)
    again = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    assert torch.equal(got, again)


def test_nan_keys_and_sums_reach_their_own_entries_only():
    case = More(75, [70, 40], heads=2, queries=4, dim=64, new=2)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    old = torch.zeros((2, 2, 70), device="cuda")
    good = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    case.dev[0, 0, int(case.table[0, 1]), 3, 0] = float("nan")   # request 0, head 0, key 19
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    assert torch.isnan(got[0, 0, 19])
    got[0, 0, 19] = good[0, 0, 19]
    assert torch.equal(got, good)
    case.dev[0, 0, int(case.table[0, 1]), 3, 0] = 0
    lse[1, 0, 0] = float("nan")                                  # the older of request 1's new tokens
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    assert torch.isnan(got[1, 0, :39]).all() and torch.isfinite(got[1, 0, 39:]).all()
    assert torch.isfinite(got[1, 1]).all() and torch.isfinite(got[0]).all()


def test_strided_weights_queries_and_layers():
    case = More(76, [70, 9], heads=2, queries=8, dim=64, new=2, layers=2, layer=1)
    _, lse = case.cache.attend(1, case.q, case.dlen, case.dtable)
    room = torch.full((2, 3, 2, 100), 7.0, device="cuda")
    rows = room[:, :, 1, 5:85].transpose(0, 1)[:2].transpose(0, 1)          # [2][2][80] of a wider tensor
    assert not rows.is_contiguous()
    before = room.clone()
    wide = torch.zeros((2, 2, 11, 72), dtype=case.q.dtype, device="cuda")
    q = wide[:, :, 2:10, :64]
    q.copy_(case.q)
    got = case.cache.weigh(1, q, lse, case.dlen, case.dtable, rows)
    case.cache.check()
    check(case, got, before[:, :, 1, 5:85][:, :2], lse, 64 ** -0.5)
    rows.fill_(7.0)
    assert torch.equal(room, before)
    # one new token: its dimension may be left out
    one = More(77, [70, 9], heads=2, queries=8, dim=64)
    _, lse = one.cache.attend(0, one.q[:, 0], one.dlen, one.dtable)
    old = torch.zeros((2, 2, 70), device="cuda")
    got = one.cache.weigh(0, one.q[:, 0], lse, one.dlen, one.dtable, old.clone())
    check(one, got, old, lse, 64 ** -0.5)


def test_narrow_weights_bad_lengths_and_blocks_are_flagged():
    case = More(78, [50, 90, 20], heads=2, queries=8, dim=64)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    old = torch.rand((3, 2, 60), device="cuda")
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, old.clone())
    with pytest.raises(KVRelayoutError, match="length"):
        case.cache.check()
    check(case, got, old, lse, 64 ** -0.5)
    for bad in (-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        lens = case.dlen.clone()
        lens[1] = bad
        wide = torch.rand((3, 2, 200), device="cuda")
        got = case.cache.weigh(0, case.q, lse, lens, case.dtable, wide.clone())
        with pytest.raises(KVRelayoutError, match="length"):
            case.cache.check()
        top = case.dtable.shape[1] * 16                          # a length counts as the nearest in range
        assert torch.equal(got[1, :, (0 if bad < 0 else top):], wide[1, :, (0 if bad < 0 else top):])
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all()
    case.dtable[1, 2] = -1                                       # its keys count as zeros
    wide = torch.zeros((3, 2, 90), device="cuda")
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, wide.clone())
    with pytest.raises(KVRelayoutError, match="block id"):
        case.cache.check()
    want = torch.exp(-lse[1, 0].view(2, 4)).sum(-1)
    assert torch.allclose(got[1, :, 32:48], want[:, None].expand(2, 16), rtol=2.0 ** -18)


def test_the_same_bits_again_captured_and_on_another_stream():
    case = More(79, [3000, 1200, 40], heads=2, queries=8, dim=64)
    first, lse = weigh(case, add=False, extra=0)
    out = torch.zeros_like(first)
    args = 0, case.q, lse, case.dlen, case.dtable
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    case.cache.weigh(*args, out, add=False, stream=side)
    side.synchronize()
    held = torch.arange(3000, device="cuda")[None, None, :] < case.dlen[:, None, None]
    assert torch.equal(out[held.expand_as(out)], first[held.expand_as(out)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.cache.weigh(*args, out)
    old = out.clone()
    case.lengths = [700, 0, 33]
    case.dlen.copy_(torch.tensor(case.lengths, dtype=torch.int32))
    _, l2 = case.cache.attend(0, case.q, case.dlen, case.dtable)
    lse.copy_(l2)
    graph.replay()
    case.cache.check()
    check(case, out, old, lse, 64 ** -0.5)


def test_offsets_beyond_32_bits_in_the_weights():
    """Heads 1.1e9 weights apart."""
    case = More(80, [90, 33], heads=2, queries=4, dim=64)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    step = 1100 * 10 ** 6
    room = torch.empty(3 * step + 100, dtype=torch.float32, device="cuda")
    rows = room.as_strided((2, 2, 90), (2 * step, step, 1))
    rows.zero_()
    got = case.cache.weigh(0, case.q, lse, case.dlen, case.dtable, rows)
    case.cache.check()
    check(case, got, torch.zeros((2, 2, 90), device="cuda"), lse, 64 ** -0.5)
    del room, rows, got
    torch.cuda.empty_cache()


def test_refusals():
    case = More(81, [20], heads=2, queries=8, dim=64)
    _, lse = case.cache.attend(0, case.q, case.dlen, case.dtable)
    w = torch.zeros((1, 2, 20), device="cuda")
    args = case.dlen, case.dtable
    for bad in (w[0], w[:, :1], w.double(), w.cpu(), torch.zeros((1, 2, 40), device="cuda")[..., ::2]):
        with pytest.raises(ValueError, match="weights"):
            case.cache.weigh(0, case.q, lse, *args, bad)
    for bad in (lse[..., :4], lse.double(), lse.cpu()):
        with pytest.raises(ValueError, match="lse"):
            case.cache.weigh(0, case.q, bad, *args, w)
    with pytest.raises(ValueError, match="gradient"):
        case.cache.weigh(0, case.q, lse, *args, w.clone().requires_grad_())
    with pytest.raises(KVRelayoutError, match="OVERLAP"):
        case.cache.weigh(0, case.q, lse, *args, torch.zeros((1, 1, 20), device="cuda").expand(1, 2, 20))
    with pytest.raises(KVRelayoutError, match="INVALID"):
        case.cache.weigh(0, case.q, lse, *args, w, cap=-1.0)
    with pytest.raises(KVRelayoutError, match="INVALID"):
        case.cache.weigh(0, case.q, lse, *args, w, window=-1)
    with pytest.raises(KVRelayoutError, match="LAYER"):
        case.cache.weigh(1, case.q, lse, *args, w)
    latent = More(82, [20], dim=576, queries=16)
    with pytest.raises(KVRelayoutError, match="UNSUPPORTED"):
        latent.cache.weigh(0, latent.q, torch.zeros((1, 1, 16), device="cuda"), latent.dlen, latent.dtable,
                           torch.zeros((1, 1, 20), device="cuda"))
