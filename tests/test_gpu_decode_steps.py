"""The example that hands prompts over and decodes them, against 64 bits."""
import os
import sys

import numpy as np
import pytest

import cache_ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_hand_off_then_decode():
    import decode_steps
    heads, queries, dim, prompts, steps = 4, 8, 64, (70, 3, 33), 5
    r = decode_steps.main(layers=2, kv_heads=heads, query_heads=queries, dim=dim, prompts=prompts, steps=steps)
    w, angles = r["workload"], r["angles"].cpu().numpy()
    assert r["positions"].tolist() == [n + steps for n in prompts]
    H, Hq, tp = heads // 4, queries // 4, 4
    src = [t.double().cpu().numpy() for t in r["src"]]
    for layer in range(2):
        for s in range(tp):
            for i, n in enumerate(prompts):
                ids = w.src_bt[w.src_off[i]:w.src_off[i + 1]]
                at = np.arange(n)
                past = [src[s // 2][layer, c, ids[at // w.src_block], at % w.src_block, s % 2 * H:s % 2 * H + H]
                        for c in range(2)]
                rows = [h[s][layer, i].double().cpu().numpy() for h in r["history"]]
                new = [cache_ref.rotate(x[None, Hq:Hq + H], [n + t], angles, dim, False, False)[0]
                       for t, x in enumerate(rows)]
                q = cache_ref.rotate(rows[-1][None, :Hq], [n + steps - 1], angles, dim, False, False)[0]
                keys = np.concatenate([past[0], np.stack(new)])
                values = np.concatenate([past[1], np.stack([x[Hq + H:] for x in rows])])
                for g in range(Hq):
                    k, v = keys[:, g // (Hq // H)], values[:, g // (Hq // H)]
                    x = k @ q[g] * dim ** -0.5
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    got = r["out"][s][layer, i, g].double().cpu().numpy()
                    # queries and new keys are rounded to bf16 once more: 2^-8 of each logit's terms
                    size = (np.abs(k) @ np.abs(q[g])).max() * dim ** -0.5
                    tol = 2.0 ** -8 * np.abs(p @ v) + 2 * (2 * 2.0 ** -8 * size) * (p @ np.abs(v)) + 2.0 ** -12
                    assert (np.abs(got - p @ v) <= tol).all()
