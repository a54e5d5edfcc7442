"""Latents under few query rows: weights enter their product as two 16-bit numbers.

The tolerance is that of ``test_gpu_cache`` with e_p = 2^-15, as over keys and values: the first number
is the one next below (at most 2^-7 of the weight away, 2^-10 in f16), the second holds what is left to 8
bits or more. One bf16 number alone is up to 2^-9 of the weight off.
"""
import numpy as np
import pytest

import cache_ref
from test_gpu_cache import Case, UNIT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", ["bf16", "f16"])
@pytest.mark.parametrize("lengths, kw", [
    ([300], dict(queries=16)), ([3000, 40, 0, 1, 777], dict(queries=16)), ([33, 1000], dict(queries=32, block=64)),
    ([500, 90], dict(queries=16, new=2, block=5)), ([6000], dict(queries=8, new=4, block=32)),
    ([200] * 90, dict(queries=1)), ([32, 64, 96, 1], dict(queries=10, new=3, block=24))])
def test_latents_keep_fifteen_bits_of_their_weights(lengths, kw, pool):
    case = Case(111, lengths, dim=576, pool=pool, **kw)
    scale = 192.0 ** -0.5
    out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=scale)
    case.cache.check()
    case.check(out, lse, scale, 0)
    ref, _, size, logit = cache_ref.attend(case.q.double().cpu().numpy(), case.rows_of, lengths, scale, 0)
    d = (case.D / 16 + 1) * 2.0 ** -21 * logit + 2.0 ** -20
    tol = UNIT[pool] * np.abs(ref) + (2.0 ** -15 + 2 * d[..., None] + max(lengths) * 2.0 ** -22) * size + \
        (2.0 ** -24 if pool == "f16" else 0)
    off = np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


def test_infinite_values_stay_infinite_and_nan_reaches_its_own_request():
    import torch
    case = Case(112, [300, 300], dim=576, queries=16, block=16)
    at = int(case.table[0, 2]), 5
    q = case.q.clone()
    q[..., 3] = 0                                       # this element does not enter the logits
    case.dev[0, 0, at[0], at[1], 0, 3] = 3.0e38
    out, lse = case.cache.attend(0, q, case.dlen, case.dtable, scale=0.05)
    assert torch.isfinite(lse).all() and torch.isfinite(out[1].float()).all()
    assert torch.isfinite(out[0].float()).all() and (out[0, 0, :, 3].float() > 1e30).all()
    case.dev[0, 0, at[0], at[1], 0, 100] = float("nan")
    out, lse = case.cache.attend(0, q, case.dlen, case.dtable, scale=0.05)
    torch.cuda.synchronize()
    assert torch.isnan(out[0].float()).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[1].float()).all() and torch.isfinite(lse[1]).all()
