"""More shapes of the decode cache's calls: 8-bit logits that grow, chunks of many newest tokens, latents
past 4 GB, 8-bit latent rows. The pools, 64-bit forms and derived tolerances are ``test_gpu_cache``'s."""
import numpy as np
import pytest
import torch

import cache_ref
import test_gpu_cache as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(heads=2, queries=2, dim=64), dict(heads=1, queries=8, dim=128, block=5),
                                dict(heads=1, queries=16, dim=256, qtype="f16")])
def test_eight_bit_logits_that_outgrow_the_maximum_from_tile_to_tile(kw):
    """Keys along each head's first query, so that its logits rise by far more than 2^5 (what P may run ahead of
    the last maximum) from each 32 keys to the next, then fall again."""
    case = base.Case(121, [400, 170], pool="e4m3", **kw)
    scale, B, G = 2.0, case.B, case.Q // case.H
    q = case.q.float().cpu()
    for r, n in enumerate(case.lengths):
        for h in range(case.H):
            u = q[r, 0, h * G]
            # x_j = rise * j, then down
            per = 0.5 / (float((u * u).sum()) * scale)
            for j in range(n):
                a = per * (j if j < n // 2 else n - j)
                code = (u * a / float(case.scales[0, 0, h])).clamp(-448, 448).to(torch.float8_e4m3fn)
                case.host[0, 0, int(case.table[r, j // B]), j % B, h] = code.view(torch.uint8)
    case.dev.copy_(case.host)
    case.wide = cache_ref.decode_e4m3(case.host.numpy()) * \
        case.scales.astype(np.float64)[:, :, None, None, :, None]
    for r, n in enumerate(case.lengths):
        keys, _ = case.rows_of(r, 0, np.arange(n))
        x = keys @ q[r, 0, 0].double().numpy() * scale * np.log2(np.e)
        tops = [x[t:t + 32].max() for t in range(0, n // 2 - 32, 32)]
        assert len(tops) > 1 and (np.diff(tops) > 5).all()
    for s in (scale, -scale, 0.1 * scale):
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=s)
        case.cache.check()
        case.check(out, lse, s, 0)


@pytest.mark.parametrize("lengths, kw, window", [
    ([300, 17, 0, 64, 40], dict(heads=2, queries=4, dim=64, new=40), 0),
    ([300, 17, 0, 64, 40], dict(heads=1, queries=2, dim=128, new=40, block=5), 33),
    ([200], dict(heads=1, queries=8, dim=128, new=200, pool="f16"), 0),
    ([150, 90], dict(heads=1, queries=3, dim=256, new=70, pool="e4m3"), 20),
    ([130, 33], dict(heads=1, queries=1, dim=64, new=130), 1),
    ([300, 17, 0, 64, 40], dict(dim=576, queries=4, new=40), 0),
    ([300, 17, 0], dict(dim=576, queries=16, new=21, block=8), 33),
    ([140], dict(dim=576, queries=1, new=140, block=5, pool="f16"), 0)])
def test_chunks_of_many_newest_tokens(lengths, kw, window):
    """More rows than one pass takes, and more newest tokens than some requests have."""
    base.Case(122, lengths, **kw).attend(scale=0.1, window=window)


@pytest.mark.parametrize("block", [16, 6])
def test_latents_past_four_gigabytes(block):
    """Blocks 1.5 GB apart, read in boxes (16) and row by row (6), and written."""
    from prefill_decode_paged_gb300 import KVCache
    stride, N, D = 3 << 29, 5, 576
    big = torch.empty((N - 1) * stride + block * 2 * D, dtype=torch.uint8, device="cuda")
    small = base.Case(123, [5 * block], dim=D, queries=16, block=block)
    order = [4, 2, 0, 3, 1]
    view = big.view(torch.bfloat16).as_strided((N, block, 1, D), (stride // 2, D, D, 1))
    for k in range(5):
        view[order[k]] = small.dev[0, 0, int(small.table[0, k])]
    cache = KVCache(None, num_layers=1, num_components=1, kv_heads=1, head_dim=D, block=block, num_blocks=N,
                    dtype=1, query_heads=16,
                    layout=dict(bases=[view], block_stride=stride, token_stride=2 * D, head_stride=2 * D,
                                shape=(N, block, 1, D), elem_bytes=2))
    table = torch.tensor([order], dtype=torch.int32, device="cuda")
    out, lse = cache.attend(0, small.q, small.dlen, table, scale=0.07)
    cache.check()
    small.check(out, lse, 0.07, 0)
    row = torch.randn((1, 1, D), device="cuda").bfloat16()
    at = torch.tensor([5], dtype=torch.int32, device="cuda")
    cache.append(0, row, None, torch.zeros(1, dtype=torch.int32, device="cuda"), at, table)
    cache.check()
    assert torch.equal(view[4, 5], row[0])
    cache.close()
    del big, view
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_append_of_eight_bit_latents(tokens):
    """A 576-element row with its last 64 rotated, into codes, and its queries' rotated part."""
    base.test_append(1, 16, 576, 64, 64, True, True, "e4m3", "bf16", 16, tokens)


def test_append_of_many_eight_bit_latents_is_that_of_few():
    base.test_append_of_many_tokens_is_that_of_few(1, 16, 576, 64, 64, True, True, "e4m3", "bf16", 16, 1100)
