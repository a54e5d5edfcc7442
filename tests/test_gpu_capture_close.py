"""Handles that are closed, as by the garbage collector, while a stream is captured."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _cache():
    from prefill_decode_paged_gb300 import KVCache
    pool = torch.zeros((1, 1, 8, 16, 1, 576), dtype=torch.bfloat16, device="cuda")
    return KVCache(pool, num_layers=1, num_components=1, kv_heads=1, head_dim=576, block=16, num_blocks=8,
                   dtype=1, query_heads=16, max_requests=2)


def _plan():
    from prefill_decode_paged_gb300 import RelayoutPlan
    pools = [torch.zeros((1, 2, 4, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids, off = np.arange(3, dtype=np.int32), np.array([0, 3])
    return RelayoutPlan(pools[:1], pools[1:], num_layers=1, num_components=2, kv_heads=2, head_dim=64, elem_bytes=2,
                        src_tp=1, dst_tp=1, src_block=16, dst_block=16, src_num_blocks=4, dst_num_blocks=4,
                        seq_lens=[40], src_off=off, src_bt=ids, dst_off=off, dst_bt=ids)


@pytest.mark.parametrize("make", [_cache, _plan])
def test_a_capture_outlives_handles_closed_in_it(make):
    victim = make()
    x = torch.zeros(1000, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.add_(1)
        victim.close()
        x.add_(1)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert (x == 6).all()
    # and the memory has been given back: as much again is there, many times over
    free = torch.cuda.mem_get_info()[0]
    for _ in range(8):
        make().close()
    assert torch.cuda.mem_get_info()[0] >= free - (64 << 20)
