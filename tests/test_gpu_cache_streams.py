"""Results that calls on another stream than the current one make."""
import pytest
import torch

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu

KINDS = [dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16)]


def _streams(kind):
    """(what `stream=` is given, the torch stream to wait for it on)"""
    if kind == "torch":
        s = torch.cuda.Stream()
        return s, s
    if kind == "handle":
        s = torch.cuda.Stream()
        return s.cuda_stream, s
    return 0, torch.cuda.default_stream()


@pytest.mark.parametrize("kind", ["torch", "handle", "legacy"])
@pytest.mark.parametrize("kw", KINDS)
def test_results_are_not_memory_that_the_current_stream_still_uses(kw, kind):
    """Tensors of the results' sizes are filled on a busy current stream and dropped before they are; the calls on
    the other stream must not be given their memory. Nothing waits for the device in between."""
    case = Case(95, [2500, 100], **kw)
    given, other = _streams(kind)
    angles = torch.from_numpy(_angles(64)).cuda()
    T, H, D = 9, case.H, case.D
    k = torch.randn((T, H, D), device="cuda").to(case.q.dtype)
    q = torch.randn((T, case.Q, D), device="cuda").to(case.q.dtype)
    requests = torch.zeros(T, dtype=torch.int32, device="cuda")
    padding = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    shapes = [((2, 1, case.Q, case.V), case.q.dtype), ((2, 1, case.Q), torch.float32), (q.shape, q.dtype)]
    current = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        torch.cuda._sleep(40_000_000)
        used = [torch.empty(s, dtype=t, device="cuda").fill_(float("nan")) for s, t in shapes]
        held = {t.data_ptr() for t in used}
        del used
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1, stream=given)
        turned = case.cache.append(0, k, None if case.latent else k, requests, padding, case.dtable,
                                   rotary=angles, q=q, stream=given)
    assert not held & {t.data_ptr() for t in (out, lse, turned)}
    other.synchronize()
    current.synchronize()
    case.cache.check()
    case.check(out, lse, 0.1, 0)


@pytest.mark.parametrize("kind", ["torch", "handle"])
@pytest.mark.parametrize("kw", KINDS)
def test_dropped_results_stay_with_their_stream(kw, kind):
    """What takes their memory next is work of the same stream, which comes after."""
    case = Case(96, [2500, 100], **kw)
    given, other = _streams(kind)
    torch.cuda.synchronize()
    out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1, stream=given)
    shape, held = out.shape, {out.data_ptr(), lse.data_ptr()}
    del out, lse
    others = [torch.empty(shape, dtype=case.q.dtype, device="cuda") for _ in range(8)]
    assert not held & {t.data_ptr() for t in others}
    other.synchronize()
    case.cache.check()


@pytest.mark.parametrize("kw", KINDS)
def test_results_inside_a_capture_of_the_given_stream(kw):
    case = Case(97, [700, 33], **kw)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out, lse = case.cache.attend(0, case.q, case.dlen, case.dtable, scale=0.1, stream=side)
    graph.replay()
    case.cache.check()
    case.check(out, lse, 0.1, 0)


def _angles(dim):
    from prefill_decode_paged_gb300 import rotary_table
    return rotary_table(16, dim)
