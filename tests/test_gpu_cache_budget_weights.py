"""The weights of a decode under a budget, each step's against 64 bits over what the pool's bytes stand for.

Bound of a step: ``test_gpu_cache_weigh``'s of what it adds, and one fp32 rounding of the sum. Whatever is added
sums up to the query heads of a key head, as each head's softmax does to one."""
import numpy as np
import pytest
import torch

import cache_more_ref as ref
import cache_ref
from prefill_decode_paged_gb300 import KVCache, rotary_table

pytestmark = pytest.mark.gpu

R, H, Q, D, B, N = 3, 2, 4, 64, 8, 24


def rows_in(raw, pool):
    """What a pool's bytes stand for: [2][N][B][H][D] float64."""
    shape = (2, N, B, H)
    if pool == "bf16":
        return raw.view(torch.bfloat16).view(shape + (D,)).double().cpu().numpy()
    host = raw.cpu().numpy()
    if pool == "e4m3":
        return cache_ref.decode_e4m3(host.reshape(shape + (D,))) * float(np.float32(0.05))
    n = 2 * N * B * H * D // 2
    return ref.values(host[:n].reshape(shape + (D // 2,)), host[n:].reshape(shape + (D // 16,)))


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("pool", ["bf16", "e4m3", "e2m1"])
def test_each_step_adds_its_own_weights(pool, cap):
    keep, recent, steps, prompts = 40, 12, 20, [33, 40, 5]
    room, scale = keep + 8, D ** -0.5
    gen = torch.Generator("cuda").manual_seed(17)
    size = {"bf16": 2 * D, "e4m3": D, "e2m1": D * 9 // 16}[pool]
    raw = torch.zeros(2 * N * B * H * size, dtype=torch.uint8, device="cuda")
    table = torch.randperm(N, generator=gen, device="cuda")[:R * (room // B)].to(torch.int32).view(R, room // B)
    host_table = table.cpu().numpy()
    angles = torch.from_numpy(rotary_table(200, D)).cuda()
    cache = KVCache(raw, num_layers=1, num_components=2, kv_heads=H, head_dim=D, block=B, num_blocks=N,
                    dtype={"bf16": 1, "e4m3": 2, "e2m1": 5}[pool],
                    scales=np.full((1, 2), 0.05) if pool == "e4m3" else None, query_heads=Q, max_requests=R)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    req = torch.repeat_interleave(torch.arange(R), torch.tensor(prompts)).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in prompts]).to(torch.int32).cuda()
    cache.append(0, randn(sum(prompts), H, D), randn(sum(prompts), H, D), req, pos, table, rotary=angles)
    each = torch.arange(R, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    true = lengths.clone()
    weights = torch.zeros((R, H, room), device="cuda")
    for s in range(steps):
        before = weights.double().cpu().numpy()
        q = cache.append(0, randn(R, H, D), randn(R, H, D), each, lengths, table, rotary=angles, q=randn(R, Q, D),
                         angles=true)
        lengths, true = lengths + 1, true + 1
        _, lse = cache.attend(0, q, lengths, table, cap=cap)
        cache.weigh(0, q, lse, lengths, table, weights, cap=cap)
        n, wide = lengths.tolist(), rows_in(raw, pool)

        def rows_of(r, g, j):
            at = host_table[r, j // B], j % B, g // (Q // H)
            return wide[0][at], wide[1][at]

        q64 = q.double().cpu().numpy()
        want = ref.attend(q64[:, None], rows_of, n, scale, cap=cap, width=room, group=Q // H,
                          lse_in=lse.double().cpu().numpy()[:, None])
        w, off = want["weights"], want["weights_off"]
        if pool != "bf16":
            # elements of q below 2^-14 of its largest become multiples of 2^-24 of it
            off = off + w * 2.0 ** -24 * np.abs(q64).max() * scale * np.abs(wide).max() * D
        target = before + w
        bound = off + (Q // H + 4) * 2.0 ** -24 * w + 2.0 ** -24 * np.abs(target) + 2.0 ** -126
        got = weights.double().cpu().numpy()
        held = np.arange(room)[None, None] < np.array(n)[:, None, None]
        assert (np.abs(got - target) <= np.where(held, bound, 0)).all(), np.abs(got - target).max()
        added = (got - before).sum(-1)
        assert np.abs(added - Q // H).max() <= 2.0 ** -8         # (and lse is that of these scores)
        if s % 8 == 7:
            cache.evict(0, weights, lengths, table, keep, recent)
            lengths = lengths.clamp(max=keep)
    cache.check()
    assert n == [44, 44, 25]
    cache.close()
