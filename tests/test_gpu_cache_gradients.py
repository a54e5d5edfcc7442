"""The calls have no backward pass, and say so."""
import pytest
import torch

from test_gpu_cache import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(heads=2, queries=8, dim=64), dict(dim=576, queries=16)])
def test_tensors_that_require_a_gradient_are_refused_where_one_is_recorded(kw):
    case = Case(105, [70, 9], **kw)
    before, lse = case.attend(scale=0.1)
    q = case.q.clone().requires_grad_()
    k = torch.randn((1, case.H, case.D), device="cuda").to(q.dtype)
    v = None if case.latent else k.clone()
    turned = torch.randn((1, case.Q, case.D), device="cuda").to(q.dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    at = torch.zeros(1, **i32), torch.full((1,), -1, **i32), case.dtable

    def append(k, v, q):
        from prefill_decode_paged_gb300 import rotary_table
        return case.cache.append(0, k, v, *at, rotary=torch.from_numpy(rotary_table(4, 64)).cuda(), q=q)
    with pytest.raises(ValueError, match="gradient"):
        case.cache.attend(0, q, case.dlen, case.dtable, scale=0.1)
    for which in range(3):
        tensors = [k, v, turned]
        if tensors[which] is not None:
            tensors[which] = tensors[which].clone().requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                append(*tensors)
            with torch.no_grad():
                append(*tensors)
    append(k, v, turned)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            out, l2 = case.cache.attend(0, q, case.dlen, case.dtable, scale=0.1)
        assert torch.equal(out, before) and torch.equal(l2, lse)
    out, l2 = case.cache.attend(0, q.detach(), case.dlen, case.dtable, scale=0.1)
    assert torch.equal(out, before) and torch.equal(l2, lse)
    case.cache.check()
