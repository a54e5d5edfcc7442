"""Attention with scores that are capped by a tanh or biased by the distance, against 64 bits."""
import numpy as np
import pytest
import torch

from cache_more_case import More
from prefill_decode_paged_gb300 import KVRelayoutError

pytestmark = pytest.mark.gpu


def slopes_of(case, kind):
    Q = case.Q
    if kind is None:
        return None
    if kind == "powers":                                         # 2^(-8 / Q), its square, ...
        s = 2.0 ** (-8.0 * np.arange(1, Q + 1) / Q)
    else:                                                        # of both signs, some zero
        s = np.random.default_rng(7).uniform(-0.02, 0.1, Q) * (np.arange(Q) % 3 > 0)
    return torch.from_numpy(s.astype(np.float32)).cuda()


CASES = [
    # lengths, kw, window, cap, slopes
    ([1], {}, 0, 30.0, "powers"), ([0, 1], {}, 0, 5.0, None), ([2, 0, 1, 17], dict(new=3), 0, 0.0, "powers"),
    ([300, 5, 64], dict(heads=2, queries=8, block=5), 0, 2.0, None),
    ([300, 5, 64], dict(heads=2, queries=8, dim=64, block=16), 100, 50.0, "mixed"),
    ([77, 200], dict(heads=1, queries=16, dim=256, block=64), 0, 50.0, None),
    ([77, 200], dict(heads=2, queries=80, dim=256, block=1), 0, 0.5, "mixed"),
    ([500], dict(heads=1, queries=33, block=8), 0, 0.0, "powers"),
    ([90, 1, 0, 260], dict(heads=2, queries=16, new=4, block=32), 50, 20.0, "powers"),
    ([90, 3, 700], dict(heads=1, queries=3, dim=96, new=2, block=7), 333, 1.0, "mixed"),
    ([31, 65], dict(heads=4, queries=4, dim=16), 0, 3.0, "powers"),
    ([6000], dict(heads=2, queries=2, dim=64, block=64), 0, 0.0, "powers"),
    ([3000, 1, 0, 2000, 17, 900], dict(queries=16, dim=64, new=2), 0, 10.0, "mixed"),
    ([97 * k % 701 for k in range(129)], dict(heads=1, queries=2, dim=64), 0, 4.0, "powers"),
    ([300, 17, 0, 64, 40], dict(heads=1, queries=2, new=40), 33, 8.0, "powers"),
]


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("lengths, kw, window, cap, slopes", CASES)
def test_attend(lengths, kw, window, cap, slopes, pool):
    if pool == "e2m1" and kw.get("dim", 128) % 64:
        kw = dict(kw, dim=192)
    case = More(61, lengths, pool=pool, **kw)
    case.attend_scored(window=window, cap=cap, slopes=slopes_of(case, slopes))


@pytest.mark.parametrize("pool", ["bf16", "e2m1"])
def test_scores_from_far_below_the_cap_to_far_beyond_it(pool):
    """Products of 10^-4 to 10^4 caps: the series, the exponential, and both where they meet."""
    case = More(62, [400, 170], heads=2, queries=16, dim=64, pool=pool)
    case.q.copy_(case.q * torch.exp(torch.linspace(-7, 3, 16, device="cuda"))[None, None, :, None])
    for cap in (0.3, 30.0, 2.0 ** 20, 2.0 ** -30):
        for scale in (0.5, -0.5, 0.01):
            case.attend_scored(scale=scale, cap=cap)


@pytest.mark.parametrize("pool", ["bf16", "f16", "e2m1"])
def test_without_cap_and_slopes_it_is_attend(pool):
    case = More(63, [300, 1, 77], heads=2, queries=8, dim=64, pool=pool)
    zero = torch.zeros(8, device="cuda")
    a, la = case.cache.attend(0, case.q, case.dlen, case.dtable)
    b, lb = case.cache.attend(0, case.q, case.dlen, case.dtable, cap=0.0)
    c, lc = case.cache.attend(0, case.q, case.dlen, case.dtable, slopes=zero)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, c) and torch.equal(la, lc)


def test_distances_of_long_requests():
    """Slopes that leave the last few keys, over 100000: scores down to -10^5, distances that fp32 holds."""
    case = More(64, [100000], heads=1, queries=2, dim=64, block=64)
    case.attend_scored(slopes=torch.tensor([1.0, 2.0 ** -12], device="cuda"))
    case.attend_scored(slopes=torch.tensor([-2.0 ** -10, 0.0], device="cuda"))


def test_infinite_logits_are_capped_and_nan_stays():
    case = More(65, [40, 40], heads=2, queries=4, dim=64)
    b = int(case.table[0, 1])
    case.dev[0, 0, b, 3, 0] = 0
    case.dev[0, 0, b, 3, 0, 5] = float("inf")
    case.q[0, 0, :2] = case.q[0, 0, :2].abs()
    case.wide[0, 0, b, 3, 0] = 0
    out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, cap=3.0)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    case.wide[0, 0, b, 3, 0, 5] = 1e30                            # its score is the cap itself
    want = case.reference(64 ** -0.5, 0, 3.0, None)
    got = out.double().cpu().numpy()
    # (bounds by hand, as the reference's own bound grows with the key: 2^-8 of the output, 2^-12 of the sum)
    assert (np.abs(got - want["out"]) <= 2.0 ** -8 * np.abs(want["out"]) + 2.0 ** -12 * want["size"]).all()
    case.dev[0, 0, b, 3, 0, 5] = float("nan")
    out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, cap=3.0)
    assert torch.isnan(out[0, 0, :2].float()).all() and torch.isfinite(out[0, 0, 2:].float()).all()
    assert torch.isfinite(out[1].float()).all()


def test_captured_with_lengths_and_slopes_from_the_device():
    case = More(66, [3000, 1200, 40], heads=2, queries=8, dim=64)
    slopes = slopes_of(case, "powers")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, cap=5.0, slopes=slopes)
    graph.replay()
    torch.cuda.synchronize()
    case.check_scored(out, lse, 64 ** -0.5, 0, 5.0, slopes)
    case.lengths = [700, 0, 33]
    case.dlen.copy_(torch.tensor(case.lengths, dtype=torch.int32))
    slopes.mul_(3)
    graph.replay()
    case.cache.check()
    case.check_scored(out, lse, 64 ** -0.5, 0, 5.0, slopes)


def test_refusals():
    case = More(67, [20], heads=2, queries=8, dim=64)
    args = 0, case.q, case.dlen, case.dtable
    for cap in (-1.0, float("nan"), float("inf")):
        with pytest.raises(KVRelayoutError, match="INVALID"):
            case.cache.attend(*args, cap=cap)
    for cap in (1e-38, 1e35):
        with pytest.raises(KVRelayoutError, match="UNSUPPORTED"):
            case.cache.attend(*args, cap=cap)
    for slopes in (torch.zeros(7), torch.zeros(8), torch.zeros(8, device="cuda").double(),
                   torch.zeros(16, device="cuda")[::2]):
        with pytest.raises(ValueError, match="slopes"):
            case.cache.attend(*args, slopes=slopes)
    with pytest.raises(ValueError, match="gradient"):
        case.cache.attend(*args, slopes=torch.zeros(8, device="cuda", requires_grad=True))
    latent = More(68, [20], dim=576, queries=16)
    for kw in (dict(cap=1.0), dict(slopes=torch.zeros(16, device="cuda"))):
        with pytest.raises(KVRelayoutError, match="UNSUPPORTED"):
            latent.cache.attend(0, latent.q, latent.dlen, latent.dtable, **kw)


def test_every_element_type_has_its_first_call_captured():
    for pool in ("bf16", "f16", "e4m3", "e2m1"):
        case = More(69, [90], heads=1, queries=9, dim=64, pool=pool)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, cap=5.0)
        graph.replay()
        torch.cuda.synchronize()
        case.check_scored(out, lse, 64 ** -0.5, 0, 5.0)
