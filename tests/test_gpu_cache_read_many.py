"""Rows read back by two tokens a block: odd and even numbers of tokens, and what lies behind the last."""
import pytest
import torch

from test_gpu_cache_evict import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", ["bf16", "f16", "e4m3", "e2m1"])
def test_as_many_tokens_one_by_one(pool):
    case = Pool(161, [700, 333], 40, pool=pool)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    kind = torch.float16 if pool == "f16" else torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(3)
    for T in (16 * sms - 1, 16 * sms, 16 * sms + 1, 16 * sms + 2, 5001):
        req = torch.randint(0, 2, (T,), generator=gen, device="cuda", dtype=torch.int32)
        pos = torch.randint(-20, 333, (T,), generator=gen, device="cuda", dtype=torch.int32)
        k, v = (torch.full((T + 2, 2, 64), 3.0, dtype=kind, device="cuda") for _ in range(2))
        case.cache.read(0, req, pos, case.dtables[0], k=k[:T], v=v[:T])
        assert (k[T:] == 3.0).all() and (v[T:] == 3.0).all()
        for at in range(0, T, 1000):
            some = slice(at, min(T, at + 1000))
            a, b = case.cache.read(0, req[some], pos[some], case.dtables[0], dtype=kind)
            assert torch.equal(k[some].view(torch.int16), a.view(torch.int16))
            assert torch.equal(v[some].view(torch.int16), b.view(torch.int16))
    case.cache.check()
