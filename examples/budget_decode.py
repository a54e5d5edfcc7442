"""A decode under a memory budget: prompts handed over in 16 bits move to a 4-bit pool, and each request keeps its
newest tokens and those that got the most attention.

The hand-off writes a bf16 pool, as in ``decode_steps.py``; its rows are read back and appended to the 4-bit pool
(already rotated, so without a table). The prompts' weights come from their last tokens' queries; an eviction brings
every request to ``keep`` tokens; then steps of append, attention and weights, one CUDA graph, with an eviction, another
graph, whenever ``slack`` tokens have come. Weights of a model are random numbers here: the point is the calls.

    python examples/budget_decode.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import workloads as wl                                                          # noqa: E402
from prefill_decode_paged_gb300 import (DTYPE_BF16, DTYPE_FP4_E2M1, KVCache, RelayoutPlan,   # noqa: E402
                                        rotary_table)


def main(kv_heads=4, query_heads=16, dim=128, prompts=(700, 90, 256), keep=128, recent=32, slack=16, steps=40,
         watch=8, cap=30.0, seed=1):
    """Runs the steps; returns the last outputs, the weights and what is cached."""
    w = wl.custom("budget_decode", seed, num_layers=1, num_components=2, kv_heads=kv_heads, head_dim=dim, elem_bytes=2,
                  src_tp=2, dst_tp=1, src_block=16, dst_block=32, seq_lens=list(prompts), values="randn")
    R, B = w.num_requests, 32
    src = [t.view(torch.bfloat16) for t in w.src_pools_torch("cuda")]
    wide = torch.zeros(w.dst_shape(), dtype=torch.bfloat16, device="cuda")
    with RelayoutPlan(src, [wide], **w.geometry()) as plan:                     # the hand-off
        plan.run_all()
        torch.cuda.synchronize()
    table = np.zeros((R, int(max(np.diff(w.dst_off)))), dtype=np.int32)
    for r in range(R):
        ids = w.dst_bt[w.dst_off[r]:w.dst_off[r + 1]]
        table[r, :len(ids)] = ids
    table = torch.from_numpy(table).cuda()

    # a 4-bit pool for the prompts as they come, and blocks for what stays of them
    need = [-(-n // B) for n in prompts]
    stay = -(-(keep + slack) // B)
    blocks = sum(need) + R * stay
    four = torch.zeros(2 * blocks * B * kv_heads * (dim // 2 + dim // 16), dtype=torch.uint8, device="cuda")
    first, at = torch.zeros((R, max(need)), dtype=torch.int32), 0
    for r, k in enumerate(need):
        first[r, :k] = torch.arange(at, at + k)
        at += k
    first = first.cuda()
    small = torch.arange(at, at + R * stay, dtype=torch.int32, device="cuda").view(R, stay)

    requests = torch.repeat_interleave(torch.arange(R), torch.tensor(prompts)).to(torch.int32).cuda()
    positions = torch.cat([torch.arange(n) for n in prompts]).to(torch.int32).cuda()
    geometry = dict(num_layers=1, num_components=2, kv_heads=kv_heads, head_dim=dim, block=B)
    cache = KVCache(four, num_blocks=blocks, dtype=DTYPE_FP4_E2M1, query_heads=query_heads, max_requests=R,
                    max_new=watch, **geometry)
    with KVCache(wide, num_blocks=w.dst_num_blocks, dtype=DTYPE_BF16, **geometry) as handed:
        k, v = handed.read(0, requests, positions, table)
        cache.append(0, k, v, requests, positions, first)

    # what the prompts' last tokens looked at decides which of their tokens stay
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    q = torch.randn((R, watch, query_heads, dim), generator=gen, device="cuda").bfloat16()
    _, lse = cache.attend(0, q, lengths, first, cap=cap)
    weights = cache.weigh(0, q, lse, lengths, first, torch.zeros((R, kv_heads, max(prompts)), device="cuda"), cap=cap)
    weights, _ = cache.evict(0, weights, lengths, first, keep, recent, into=small, out=torch.zeros_like(weights))
    weights = weights[:, :, :keep + slack].contiguous()

    places = lengths.clamp(max=keep)                    # where each request's next token goes
    true = lengths.clone()                              # and where it stands in its text
    lengths = places.clone()
    angles = torch.from_numpy(rotary_table(max(prompts) + steps, dim)).cuda()
    each = torch.arange(R, dtype=torch.int32, device="cuda")
    qkv = torch.empty((R, query_heads + 2 * kv_heads, dim), dtype=torch.bfloat16, device="cuda")
    turned = torch.empty((R, query_heads, dim), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(turned), torch.empty((R, query_heads), device="cuda")
    slots = torch.empty((R, kv_heads, keep), dtype=torch.int32, device="cuda")

    def step():
        lengths.add_(1)
        q, k, v = qkv.split([query_heads, kv_heads, kv_heads], 1)
        cache.append(0, k, v, each, places, small, rotary=angles, q=q, q_out=turned, angles=true)
        cache.attend(0, turned, lengths, small, out=out, lse=lse, cap=cap)
        cache.weigh(0, turned, lse, lengths, small, weights, cap=cap)
        places.add_(1)
        true.add_(1)

    def evict():
        cache.evict(0, weights, lengths, small, keep, recent, slots=slots)
        lengths.clamp_(max=keep)
        places.copy_(lengths)

    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, body in zip(graphs, (step, evict)):
        with torch.cuda.graph(graph):
            body()
    for s in range(steps):
        qkv.normal_(generator=gen)
        graphs[0].replay()
        if s % slack == slack - 1:
            graphs[1].replay()
    cache.check()                                       # nothing was out of range
    print(f"{steps} steps of {R} requests; {list(map(int, true))} tokens each, of which {lengths.tolist()} are cached, "
          f"in {four.numel() / wide.numel() / 2:.2f} of the 16-bit pool's memory")
    result = dict(out=out, lse=lse, weights=weights, lengths=lengths, true=true, cache=cache, small=small)
    return result


if __name__ == "__main__":
    main()["cache"].close()
