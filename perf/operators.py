"""The decode side's operators as a user of the package calls them, with plain forms to compare them with.

Three operators work on a decode pool in the package's layout [L][C][N][B][H][D]:

``append``  writes new tokens' keys and values (or latents) through the block table, with the
            position rotation applied to the keys and to the queries on the way, and quantized
            to 8 bits with per-head scales where the pool holds E4M3;
``attend``  attention of each request's newest tokens over its paged keys and values;
``latent``  the same over a paged latent (one 576-wide row a token; the first 512 are the values).

``own`` false: elementary torch operations in 32 bits. ``own`` true: the package's kernels.
"""
import math
import random

import torch

own = False

BF16, E4M3, F16 = 1, 2, 3                      # the package's element type numbers
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.uint8}
NUMBER = {"bf16": BF16, "f16": F16, "e4m3": E4M3}
LATENT, VALUES = 576, 512                      # a latent row and the part of it that is the value


# -- cases ----------------------------------------------------------------------

def listed():
    return [
        # one request generates one token; 8 key heads, 32 query heads
        {"name": "append-one", "op": "append", "requests": 1, "shortest": 100, "longest": 100,
         "pick": 0, "new": 1, "heads": 8, "queries": 32, "dim": 128, "qdim": 128, "rotated": 128,
         "interleaved": False, "last": False, "pool": "bf16", "type": "bf16", "block": 32},
        # a decode batch of 64 requests into an 8-bit cache, half of each head rotated
        {"name": "append-batch-e4m3", "op": "append", "requests": 64, "shortest": 700,
         "longest": 4096, "pick": 1, "new": 1, "heads": 8, "queries": 64, "dim": 128,
         "qdim": 128, "rotated": 64, "interleaved": False, "last": False, "pool": "e4m3",
         "type": "bf16", "block": 64},
        # whole prompts of 512 to 4096 tokens
        {"name": "append-prompts", "op": "append", "requests": 16, "shortest": 512,
         "longest": 4096, "pick": 2, "new": 0, "heads": 8, "queries": 32, "dim": 128,
         "qdim": 128, "rotated": 128, "interleaved": False, "last": False, "pool": "bf16",
         "type": "bf16", "block": 32},
        # latent rows of short prompts: the last 64 of 576 are rotated, pairs side by side;
        # the queries' rotated part alone, 16 heads a shard
        {"name": "append-latent", "op": "append", "requests": 12, "shortest": 1, "longest": 777,
         "pick": 3, "new": 0, "heads": 1, "queries": 16, "dim": LATENT, "qdim": 64, "rotated": 64,
         "interleaved": True, "last": True, "pool": "bf16", "type": "bf16", "block": 16},
        # one short request, two heads of 64 in float16: the latency of a call
        {"name": "attend-one-short", "op": "attend", "requests": 1, "shortest": 100,
         "longest": 100, "pick": 0, "new": 1, "heads": 2, "queries": 2, "dim": 64,
         "pool": "f16", "type": "f16", "block": 32, "window": 0},
        # 16 requests of 512 to 4096 tokens; 4 query heads to a key head
        {"name": "attend-batch", "op": "attend", "requests": 16, "shortest": 512,
         "longest": 4096, "pick": 1, "new": 1, "heads": 8, "queries": 32, "dim": 128,
         "pool": "bf16", "type": "bf16", "block": 32, "window": 0},
        # four prompts of 32768 less a few; a shard with half of 8 key heads
        {"name": "attend-long", "op": "attend", "requests": 4, "shortest": 32705,
         "longest": 32767, "pick": 2, "new": 1, "heads": 4, "queries": 32, "dim": 128,
         "pool": "bf16", "type": "bf16", "block": 64, "window": 0},
        # one very long request on an 8-bit cache
        {"name": "attend-long-e4m3", "op": "attend", "requests": 1, "shortest": 131071,
         "longest": 131071, "pick": 3, "new": 1, "heads": 8, "queries": 64, "dim": 128,
         "pool": "e4m3", "type": "bf16", "block": 32, "window": 0},
        # four drafted tokens a request, a sliding window, lengths from zero on; one key head
        {"name": "attend-draft-window", "op": "attend", "requests": 48, "shortest": 0,
         "longest": 8192, "pick": 4, "new": 4, "heads": 1, "queries": 8, "dim": 128,
         "pool": "bf16", "type": "bf16", "block": 32, "window": 1024},
        # one request of 4096 latents, 16 heads a shard
        {"name": "latent-one", "op": "latent", "requests": 1, "shortest": 4096, "longest": 4096,
         "pick": 0, "new": 1, "heads": 1, "queries": 16, "dim": LATENT, "pool": "bf16",
         "type": "bf16", "block": 16, "window": 0},
        # 64 requests of 1024 to 16384 latents, all 128 heads
        {"name": "latent-batch", "op": "latent", "requests": 64, "shortest": 1024,
         "longest": 16384, "pick": 1, "new": 1, "heads": 1, "queries": 128, "dim": LATENT,
         "pool": "bf16", "type": "bf16", "block": 16, "window": 0},
        # two drafted tokens a request, 16 heads a shard, lengths from a few on
        {"name": "latent-draft", "op": "latent", "requests": 9, "shortest": 5, "longest": 6001,
         "pick": 2, "new": 2, "heads": 1, "queries": 16, "dim": LATENT, "pool": "bf16",
         "type": "bf16", "block": 64, "window": 0},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "latent", "latent"])
    requests = _log(rng, 1, 64)
    c = {"op": op, "requests": requests, "pick": rng.randrange(1 << 20)}
    if op == "append":
        latent = rng.random() < 0.3
        prompt = rng.random() < 0.5
        most = max(2, min(4096, 36000 // requests)) if prompt else 4096
        c["longest"] = _log(rng, 2, most)
        c["shortest"] = rng.randint(1, c["longest"])
        c["new"] = 0 if prompt else rng.randint(1, min(4, c["shortest"]))
        if latent:
            c.update(heads=1, queries=rng.choice([1, 16, 31, 32]), dim=LATENT, qdim=64,
                     rotated=64, interleaved=rng.random() < 0.8, last=True, pool="bf16",
                     type="bf16")
        else:
            dim = rng.choice([64, 96, 128, 128, 128, 256])
            heads = rng.choice([1, 2, 3, 4, 8])
            pool = rng.choice(["bf16", "bf16", "f16", "e4m3"])
            c.update(heads=heads, queries=heads * rng.choice([1, 2, 4]), dim=dim, qdim=dim,
                     rotated=rng.choice([dim, dim, dim // 2]),
                     interleaved=rng.random() < 0.4, last=rng.random() < 0.2, pool=pool,
                     type="f16" if pool == "f16" else "bf16")
    elif op == "attend":
        heads = rng.choice([1, 1, 2, 3, 4, 8])
        dim = rng.choice([64, 96, 128, 128, 128, 256])
        pool = rng.choice(["bf16", "bf16", "f16", "e4m3"])
        c.update(heads=heads, queries=heads * rng.choice([1, 2, 4, 5, 8, 16]), dim=dim, pool=pool,
                 type="f16" if pool == "f16" else "bf16", new=rng.choice([1, 1, 1, 2, 3, 4]),
                 window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]))
        most = min(131072, 100000000 // (requests * heads * dim),
                   25000000000 // (requests * c["queries"] * c["new"] * dim))
        c["longest"] = _log(rng, 16, max(17, most))
        c["shortest"] = rng.randint(0, c["longest"])
    else:
        c.update(heads=1, queries=rng.choice([8, 16, 16, 32, 64, 128]), dim=LATENT, pool="bf16",
                 type="bf16", new=rng.choice([1, 1, 2, 3]), window=0)
        rows = max(1, c["queries"] * c["new"] / 128)
        c["longest"] = _log(rng, 16, min(65536, int(500000 / requests / rows)))
        c["shortest"] = rng.randint(0, c["longest"])
    c["block"] = rng.choice([1, 16, 16, 24, 32, 64, 64, 128])
    return c


def lengths(case):
    """Tokens that each request holds, its new ones included; the longest and the shortest occur."""
    r = random.Random(case["pick"])
    got = [r.randint(case["shortest"], case["longest"]) for _ in range(case["requests"])]
    got[r.randrange(len(got))] = case["longest"]
    if len(got) > 1:
        got[(got.index(case["longest"]) + 1) % len(got)] = case["shortest"]
    return got


def fresh(case):
    """How many of each request's tokens are new (0 in a case: all of them, a prompt)."""
    return [n if case["new"] == 0 else min(case["new"], n) for n in lengths(case)]


def per_row(case):
    return 1 if case["pool"] == "e4m3" else 2


def work(case):
    lens, D, H, Q = lengths(case), case["dim"], case["heads"], case["queries"]
    if case["op"] == "append":
        tokens = sum(fresh(case))
        comps = 1 if D == LATENT else 2
        row = comps * H * D * (2 + per_row(case)) + 2 * 2 * Q * case["qdim"] + 12
        return {"bytes": tokens * row + 4 * case["rotated"] * min(tokens, max(lens)),
                "flops": tokens * 3 * case["rotated"] * (H + Q)}
    m, w = case["new"], case["window"]
    seen = cached = 0
    for n in lens:
        ends = [n - m + i + 1 for i in range(m)]                  # keys that query i may see
        seen += sum(min(e, w) if w else e for e in ends if e > 0)
        first = max(0, ends[0] - w) if w else 0
        cached += max(0, n - first)
    values = VALUES if case["op"] == "latent" else D
    comps = 1 if case["op"] == "latent" else 2
    io = len(lens) * m * Q * (2 * D + 2 * values + 4)
    return {"bytes": cached * comps * H * D * per_row(case) + io + 4 * cached // case["block"],
            "flops": 2 * seen * Q * (D + values)}


# -- inputs ---------------------------------------------------------------------

def _normal(gen, shape, dtype, spread=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * spread).to(dtype)


def _table(case, gen):
    """A decode pool's size and block table: the blocks of a permutation, request by request."""
    B, lens = case["block"], lengths(case)
    need = [-(-(n + 1) // B) for n in lens]                       # one slot more, as an engine keeps
    blocks = max(1, math.ceil(1.25 * sum(need)))
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    width = max(need)
    at = torch.zeros((len(lens), width), dtype=torch.int64)
    start = 0
    for r, k in enumerate(need):
        at[r, :k] = torch.arange(start, start + k)
        start += k
    return blocks, order[at.to("cuda")].contiguous()


def _codes(gen, shape):
    """Every E4M3 byte but the two NaN patterns, those of small numbers more often: codes of
    normal values at the scale that fits them."""
    x = torch.randn(shape, generator=gen, device="cuda") * 16.0
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _inputs(case, seed):
    """The values of a case, from the seed alone: a dict of tensors on the GPU."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TORCH[case["type"]]
    H, D, Q, B = case["heads"], case["dim"], case["queries"], case["block"]
    comps = 1 if D == LATENT else 2
    lens = lengths(case)
    blocks, table = _table(case, gen)
    s = {"case": case, "blocks": blocks, "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    shape = (1, comps, blocks, B, H, D)
    s["scales"] = None
    if case["pool"] == "e4m3":                                    # per head, near 1/16
        s["scales"] = (torch.rand((1, comps, H), generator=gen, device="cuda") + 0.5) / 16
    if case["op"] == "append":
        new = fresh(case)
        T = sum(new)
        s["requests"] = torch.cat([torch.full((k,), r, dtype=torch.int32)
                                   for r, k in enumerate(new)]).to("cuda")
        s["positions"] = torch.cat([torch.arange(n - k, n, dtype=torch.int32)
                                    for n, k in zip(lens, new)]).to("cuda")
        s["k"] = _normal(gen, (T, H, D), dt)
        s["v"] = _normal(gen, (T, H, D), dt) if comps == 2 else None
        s["q"] = _normal(gen, (T, Q, case["qdim"]), dt)
        half = case["rotated"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
        s["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["pool"] = torch.zeros(shape, dtype=TORCH[case["pool"]], device="cuda")
        s["q_out"] = torch.zeros_like(s["q"])
    else:
        m = case["new"]
        s["pool"] = _codes(gen, shape) if case["pool"] == "e4m3" else \
            _normal(gen, shape, TORCH[case["pool"]])
        s["q"] = _normal(gen, (len(lens), m, Q, D), dt, 2.0)
        values = VALUES if case["op"] == "latent" else D
        s["out"] = torch.empty((len(lens), m, Q, values), dtype=dt, device="cuda")
        s["lse"] = torch.empty((len(lens), m, Q), dtype=torch.float32, device="cuda")
        # a latent stands for keys of 128 + 64, whose scale it keeps
        s["scale"] = 192.0 ** -0.5 if case["op"] == "latent" else D ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from prefill_decode_paged_gb300 import KVCache
        m = case["new"] if case["op"] != "append" else 1
        s["cache"] = KVCache(s["pool"], num_layers=1, num_components=s["pool"].shape[1],
                             kv_heads=case["heads"], head_dim=case["dim"], block=case["block"],
                             num_blocks=s["blocks"], dtype=NUMBER[case["pool"]],
                             scales=None if s["scales"] is None else s["scales"].cpu().numpy(),
                             per_head=True, query_heads=case["queries"],
                             max_requests=case["requests"], max_new=m)
    return s


# -- the plain forms ------------------------------------------------------------

def _rotate(x, cos, sin, case):
    """x [T, heads, dim] in 32 bits with its rotated part turned by each token's angles."""
    R = case["rotated"]
    first = x.shape[-1] - R if case["last"] else 0
    part = x[..., first:first + R]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :R // 2], part[..., R // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([x[..., :first], turned, x[..., first + R:]], -1)


def _store(x, s, comp):
    """32-bit rows in the pool's type."""
    if s["scales"] is None:
        return x.to(s["pool"].dtype)
    y = x * (1.0 / s["scales"][0, comp])[None, :, None]
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    case, B = s["case"], s["case"]["block"]
    pos, req = s["positions"].long(), s["requests"].long()
    block = s["table"][req, pos // B].long()
    angles = s["rotary"][pos][:, None, :]
    cos, sin = angles[..., :case["rotated"] // 2], angles[..., case["rotated"] // 2:]
    s["pool"][0, 0].index_put_((block, pos % B), _store(_rotate(s["k"].float(), cos, sin, case), s, 0))
    if s["v"] is not None:
        s["pool"][0, 1].index_put_((block, pos % B), _store(s["v"].float(), s, 1))
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case))
    return s


def _gathered(s, comp):
    """One component's rows in request order, in 32 bits: [R, S, H, D]."""
    rows = s["pool"][0, comp][s["table"].long()].flatten(1, 2)
    if s["scales"] is None:
        return rows.float()
    return rows.view(torch.float8_e4m3fn).float() * s["scales"][0, comp][:, None]


def _plain_attend(s):
    case = s["case"]
    R, m, Q, D = s["q"].shape
    H, w = case["heads"], case["window"]
    keys = _gathered(s, 0)                                        # [R, S, H, D]
    values = keys[..., :VALUES] if case["op"] == "latent" else _gathered(s, 1)
    q = s["q"].float().view(R, m, H, Q // H, D).permute(0, 2, 1, 3, 4).reshape(R, H, -1, D)
    logits = torch.matmul(q, keys.permute(0, 2, 3, 1)) * s["scale"]   # [R, H, m * G, S]
    at = torch.arange(keys.shape[1], device="cuda")[None, None, :]
    end = s["lens"].long()[:, None] - m + torch.arange(m, device="cuda")[None, :]
    seen = at <= end[:, :, None]                                  # [R, m, S]
    if w:
        seen = seen & (at > end[:, :, None] - w)
    seen = seen[:, None, :, None, :].expand(R, H, m, Q // H, -1).reshape(R, H, -1, keys.shape[1])
    logits = torch.where(seen, logits, torch.full_like(logits, -math.inf))
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    out = torch.matmul(p, values.permute(0, 2, 1, 3))             # [R, H, m * G, V]
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))

    def back(x):
        return x.view(R, H, m, Q // H, -1).permute(0, 2, 1, 3, 4).reshape(R, m, Q, -1)
    s["out"].copy_(back(out))
    s["lse"].copy_(back(lse)[..., 0])
    return s


def _outputs(s):
    if s["case"]["op"] == "append":
        pool = s["pool"] if s["scales"] is None else s["pool"].view(torch.float8_e4m3fn)
        return {"pool": pool, "q": s["q_out"]}
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    case = s["case"]
    if not own:
        return _outputs(_plain_append(s) if case["op"] == "append" else _plain_attend(s))
    if case["op"] == "append":
        s["cache"].append(0, s["k"], s["v"], s["requests"], s["positions"], s["table"],
                          rotary=s["rotary"], interleaved=case["interleaved"],
                          rotate_last=case["last"], q=s["q"], q_out=s["q_out"])
    else:
        s["cache"].attend(0, s["q"], s["lens"], s["table"], out=s["out"], lse=s["lse"],
                          scale=s["scale"], window=case["window"])
    return _outputs(s)


# -- the definitions in 64 bits -------------------------------------------------

def _exact_append(s):
    case, B = s["case"], s["case"]["block"]
    half = case["rotated"] // 2
    pos = s["positions"].double()

    def turn(x):
        """Each pair (a, b) of the rotated part as the complex number a + ib, times e^(i angle)."""
        x = x.double()
        table = s["rotary"].double()[s["positions"].long()][:, None, :]
        unit = torch.complex(table[..., :half].contiguous(), table[..., half:].contiguous())
        first = x.shape[-1] - 2 * half if case["last"] else 0
        lo, hi = (first, first + 2 * half)
        if case["interleaved"]:
            ia, ib = torch.arange(lo, hi, 2), torch.arange(lo + 1, hi, 2)
        else:
            ia, ib = torch.arange(lo, lo + half), torch.arange(lo + half, hi)
        z = torch.complex(x[..., ia.to("cuda")], x[..., ib.to("cuda")]) * unit
        y = x.clone()
        y[..., ia.to("cuda")], y[..., ib.to("cuda")] = z.real, z.imag
        return y

    pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
    slots = s["table"].long()[s["requests"].long(), torch.div(pos, B, rounding_mode="floor").long()] \
        * B + s["positions"].long() % B
    for comp, rows in enumerate([turn(s["k"])] + ([s["v"].double()] if s["v"] is not None else [])):
        if s["scales"] is not None:
            rows = rows / s["scales"].double()[0, comp][None, :, None]
            rows = rows.clamp(-448.0, 448.0)
        pool[0, comp].view(-1, *pool.shape[-2:])[slots] = rows
    return {"pool": pool, "q": turn(s["q"])}


def _exact_attend(s):
    case = s["case"]
    R, m, Q, D = s["q"].shape
    H, w, B, lens = case["heads"], case["window"], case["block"], lengths(case)
    V = VALUES if case["op"] == "latent" else D
    out = torch.zeros((R, m, Q, V), dtype=torch.float64, device="cuda")
    lse = torch.full((R, m, Q), -math.inf, dtype=torch.float64, device="cuda")

    def rows_of(comp, slots):
        plane = s["pool"][0, comp].reshape(-1, H, D)[slots]
        if s["scales"] is None:
            return plane.double()
        return plane.view(torch.float8_e4m3fn).double() * s["scales"].double()[0, comp][:, None]

    for r, n in enumerate(lens):
        for i in range(m):
            last = n - m + i
            if last < 0:
                continue
            first = max(0, last - w + 1) if w else 0
            j = torch.arange(first, last + 1, device="cuda")
            slots = s["table"][r].long()[j // B] * B + j % B
            keys = rows_of(0, slots)
            values = keys[..., :V] if case["op"] == "latent" else rows_of(1, slots)
            for h in range(H):
                qs = s["q"][r, i, h * (Q // H):(h + 1) * (Q // H)].double()
                x = qs @ keys[:, h].T * s["scale"]
                z = torch.logsumexp(x, -1)
                lse[r, i, h * (Q // H):(h + 1) * (Q // H)] = z
                out[r, i, h * (Q // H):(h + 1) * (Q // H)] = torch.exp(x - z[:, None]) @ values[:, h]
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
