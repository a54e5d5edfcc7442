"""A prompt batch handed from prefill to decode, then decoded: relayout, append, attend.

The prefill side holds two tensor-parallel shards, the decode side four. The hand-off writes the
decode pools; each decode shard then appends every step's keys and values (rotated on the way) and
attends to its heads. Weights and activations are random numbers: the point is the calls, in the
order in which an engine makes them. One step of all layers and shards is captured in a CUDA graph;
lengths, positions and the block table stay on the device and are advanced there.

    python examples/decode_steps.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import workloads as wl                                                          # noqa: E402
from prefill_decode_paged_gb300 import DTYPE_BF16, KVCache, RelayoutPlan, rotary_table   # noqa: E402


def main(layers=4, kv_heads=8, query_heads=32, dim=128, prompts=(700, 33, 256), steps=24, seed=1):
    """Runs the steps; returns every shard's last outputs [R][Hq / tp][D] and what made them."""
    w = wl.custom("decode_steps", seed, num_layers=layers, num_components=2, kv_heads=kv_heads,
                  head_dim=dim, elem_bytes=2, src_tp=2, dst_tp=4, src_block=16, dst_block=32,
                  seq_lens=list(prompts), values="randn", dst_reserve=steps + 1)
    tp, R = w.dst_tp, w.num_requests
    src = [t.view(torch.bfloat16) for t in w.src_pools_torch("cuda")]
    dst = [torch.zeros(w.dst_shape(), dtype=torch.bfloat16, device="cuda") for _ in range(tp)]

    # the decode side's block table: prompt blocks and those reserved for the steps
    width = int(max(np.diff(w.dst_off)))
    table = np.zeros((R, width), dtype=np.int32)
    for r in range(R):
        ids = w.dst_bt[w.dst_off[r]:w.dst_off[r + 1]]
        table[r, :len(ids)] = ids
    table = torch.from_numpy(table).cuda()

    with RelayoutPlan(src, dst, **w.geometry()) as plan:                       # the hand-off
        plan.run_all()
        torch.cuda.synchronize()

    H, Hq = kv_heads // tp, query_heads // tp
    caches = [KVCache(dst[s], num_layers=layers, num_components=2, kv_heads=H, head_dim=dim,
                      block=w.dst_block, num_blocks=w.dst_num_blocks, dtype=DTYPE_BF16,
                      query_heads=Hq, max_requests=R) for s in range(tp)]
    angles = torch.from_numpy(rotary_table(max(prompts) + steps + 1, dim)).cuda()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    # this step's projections, packed [q | k | v] per shard as one matrix product gives them
    qkv = [torch.empty((layers, R, Hq + 2 * H, dim), dtype=torch.bfloat16, device="cuda") for _ in range(tp)]
    out = [torch.empty((layers, R, Hq, dim), dtype=torch.bfloat16, device="cuda") for _ in range(tp)]
    turned = torch.empty((R, Hq, dim), dtype=torch.bfloat16, device="cuda")
    requests = torch.arange(R, dtype=torch.int32, device="cuda")
    positions = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    lengths = positions + 1

    def step():
        for layer in range(layers):
            for s, cache in enumerate(caches):
                q, k, v = qkv[s][layer].split([Hq, H, H], 1)
                cache.append(layer, k, v, requests, positions, table, rotary=angles, q=q, q_out=turned)
                cache.attend(layer, turned, lengths, table, out=out[s][layer], lse=False)
        positions.add_(1)
        lengths.add_(1)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    history = []
    ms = 0.0
    for _ in range(steps):
        for t in qkv:
            t.normal_(generator=gen)
        history.append([t.clone() for t in qkv])
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        ms += start.elapsed_time(end)
    for cache in caches:
        cache.check()                                  # nothing was out of range
        cache.close()
    print(f"{steps} steps of {R} requests, {layers} layers, {tp} shards: {1e3 * ms / steps:.1f} us a step "
          f"({1e3 * ms / steps / layers / tp:.1f} us an append and attention)")
    return dict(out=out, history=history, src=src, workload=w, angles=angles, positions=positions)


if __name__ == "__main__":
    main()
