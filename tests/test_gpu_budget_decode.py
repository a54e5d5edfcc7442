"""The example of a decode under a memory budget: it runs, and caches what it says."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "budget_decode.py")
    spec = importlib.util.spec_from_file_location("budget_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kw", [{}, dict(kv_heads=2, query_heads=2, dim=64, prompts=(40, 300), keep=64, recent=64,
                                         slack=8, steps=9, watch=1)])
def test_budget_decode(kw):
    r = _example().main(**kw)
    prompts, steps = kw.get("prompts", (700, 90, 256)), kw.get("steps", 40)
    keep, slack = kw.get("keep", 128), kw.get("slack", 16)
    assert r["true"].tolist() == [n + steps for n in prompts]
    assert all(min(n, keep) <= x <= keep + slack for n, x in zip(prompts, r["lengths"].tolist()))
    assert torch.isfinite(r["out"].float()).all() and torch.isfinite(r["lse"]).all()
    for i, n in enumerate(r["lengths"].tolist()):
        assert not r["weights"][i, :, n:].any() and (r["weights"][i, :, :n] >= 0).all()
    r["cache"].close()
