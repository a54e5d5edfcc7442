"""A decode cache under memory pressure: the operators that keep it small, as a user of the package calls them, with plain forms.

``append``  new tokens' keys and values into a 4-bit pool (position rotation on the way), and the same
            tokens read back as 16-bit rows, as a prefill over a cached prefix takes them;
``attend``  attention of each request's newest tokens over paged keys and values: over 4-bit pools, and with
            scores that are capped by a tanh or biased by the distance, over any pool;
``weigh``   how much attention each cached key got from the newest tokens, for each key head;
``evict``   of each head's cached tokens the newest and those of the largest weights are kept, moved
            together through a second block table.

``own`` false: elementary torch operations in 32 bits. ``own`` true: the package's kernels.

A 4-bit pool holds, for each row of D elements, D/2 bytes of E2M1 codes (even elements in the low halves) and
D/16 E4M3 block scales: the codes of all planes first, then the block scales of all planes.
"""
import math
import random

import torch

own = False

NUMBER = {"bf16": 1, "e4m3": 2, "f16": 3, "e2m1": 5}              # the package's element type numbers
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
GROUP = 16                                                        # elements of a block scale


# -- cases ----------------------------------------------------------------------

def _append(name, **kw):
    return dict({"name": name, "op": "append", "pick": 0, "new": 1, "heads": 8, "queries": 32, "dim": 128,
                 "rotated": 128, "interleaved": False, "last": False, "pool": "e2m1", "type": "bf16",
                 "block": 32}, **kw)


def _attend(name, **kw):
    return dict({"name": name, "op": "attend", "pick": 1, "new": 1, "heads": 8, "queries": 32, "dim": 128,
                 "pool": "e2m1", "type": "bf16", "block": 32, "window": 0, "cap": 0.0, "bias": False}, **kw)


def _weigh(name, **kw):
    return dict(_attend(name, pool="bf16", add=True), op="weigh", **kw)


def _evict(name, **kw):
    return dict({"name": name, "op": "evict", "pick": 2, "heads": 8, "dim": 128, "pool": "bf16", "type": "bf16",
                 "block": 32}, **kw)


def listed():
    return [
        # one request generates one token into a 4-bit cache; 8 key heads, 32 query heads
        _append("append-one", requests=1, shortest=100, longest=100),
        # whole prompts of 512 to 4096 tokens into a 4-bit cache
        _append("append-prompts", requests=16, shortest=512, longest=4096, new=0),
        # one request of 4096 tokens on a 4-bit cache: the latency of a step
        _attend("attend-one", requests=1, shortest=4096, longest=4096),
        # a full decode batch on a 4-bit cache
        _attend("attend-batch", requests=64, shortest=4096, longest=8192, queries=64),
        # four drafted tokens a request, lengths from zero on, one key head of a shard with 8 query heads
        _attend("attend-draft", requests=48, shortest=0, longest=8192, new=4, heads=1, queries=8),
        # capped scores, a window, heads of 256
        _attend("attend-capped", requests=16, shortest=512, longest=8191, heads=4, queries=8, dim=256,
                pool="bf16", window=4096, cap=50.0, block=16),
        # scores biased by the distance, as many key heads as query heads, half precision
        _attend("attend-biased", requests=4, shortest=16000, longest=16384, heads=16, queries=16, pool="f16",
                type="f16", bias=True, block=64),
        # the weights of a decode batch, added to those of earlier steps
        _weigh("weigh-batch", requests=16, shortest=512, longest=4096),
        # the last 16 tokens of long prompts say which keys matter; an 8-bit cache
        _weigh("weigh-prompts", requests=4, shortest=16001, longest=32768, new=16, pool="e4m3", add=False),
        # one short request after 64 steps over its budget, two heads of a shard in 8 bits
        _evict("evict-one", requests=1, shortest=1088, longest=1088, keep=1024, recent=256, heads=2, pool="e4m3"),
        # a batch cut to half its length
        _evict("evict-batch", requests=16, shortest=2000, longest=8192, keep=2048, recent=512),
        # long prompts cut to what their decode may hold
        _evict("evict-prompts", requests=4, shortest=32000, longest=32768, keep=8192, recent=1000, heads=4,
               block=64),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "weigh", "evict", "evict"])
    requests = _log(rng, 1, 64)
    block = rng.choice([1, 16, 16, 24, 32, 64, 64, 128])
    pick = rng.randrange(1 << 20)
    heads = rng.choice([1, 1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 128, 128, 192, 256])
    if op == "append":
        prompt = rng.random() < 0.5
        longest = _log(rng, 2, max(2, min(4096, 36000 * 1024 // (requests * heads * dim))) if prompt else 4096)
        shortest = rng.randint(1, longest)
        return _append("", requests=requests, longest=longest, shortest=shortest, pick=pick, block=block,
                       new=0 if prompt else rng.randint(1, min(4, shortest)), heads=heads,
                       queries=heads * rng.choice([1, 2, 4]), dim=dim,
                       rotated=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.4,
                       last=rng.random() < 0.2, type=rng.choice(["bf16", "bf16", "f16"]))
    pool = rng.choice(["bf16", "f16", "e4m3", "e2m1"])
    kind = "f16" if pool == "f16" else "bf16"
    if op == "evict":
        pool, kind = ("bf16", "bf16") if pool == "e2m1" else (pool, kind)
        longest = _log(rng, 16, min(65536, 100000000 // (requests * heads * dim)))
        keep = rng.randint(1, longest)
        return _evict("", requests=requests, longest=longest, shortest=rng.randint(0, longest), pick=pick,
                      block=block, heads=heads, dim=dim, keep=keep, recent=rng.randint(0, keep), pool=pool,
                      type=kind)
    queries = heads * rng.choice([1, 2, 4, 5, 8, 16])
    new = rng.choice([1, 1, 1, 2, 3, 4]) if op == "attend" else rng.choice([1, 1, 4, 16])
    longest = _log(rng, 16, max(17, min(131072, 200000000 // (requests * heads * dim),
                                        (3 if op == "attend" else 6) * 10 ** 9 // (requests * queries * new * dim))))
    plain = op == "attend" and pool != "e2m1"                     # (4-bit pools, or scores of another form)
    form = rng.choice([1, 2, 3] if plain else [0, 0, 1, 2, 3])
    kw = dict(requests=requests, longest=longest, shortest=rng.randint(0, longest), pick=pick, block=block,
              heads=heads, queries=queries, dim=dim, pool=pool, type=kind, new=new,
              window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
              cap=rng.choice([20.0, 30.0, 50.0]) if form & 1 else 0.0, bias=bool(form & 2))
    if op == "attend":
        return _attend("", **kw)
    return dict(_weigh(""), add=rng.random() < 0.5, **kw)


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


def row_bytes(case):
    D = case["dim"]
    return {"bf16": 2 * D, "f16": 2 * D, "e4m3": D, "e2m1": D // 2 + D // GROUP}[case["pool"]]


def work(case):
    lens, D, H, row = lengths(case), case["dim"], case["heads"], row_bytes(case)
    if case["op"] == "append":
        tokens, Q = sum(fresh(case)), case["queries"]
        # rows in, codes and scales out and in again, rows out; queries in and out
        each = 2 * H * (2 * D + 2 * row + 2 * D) + 2 * 2 * Q * D + 12
        return {"bytes": tokens * each + 4 * case["rotated"] * min(tokens, max(lens)),
                "flops": tokens * (3 * case["rotated"] * (H + Q) + 4 * H * D)}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": H * (kept * (2 * 2 * row + 4) + 2 * 4 * sum(lens)), "flops": H * sum(lens)}
    m, w, Q = case["new"], case["window"], case["queries"]
    seen = cached = 0
    for n in lens:
        ends = [n - m + i + 1 for i in range(m)]                  # keys that query i may see
        seen += sum(min(e, w) if w else e for e in ends if e > 0)
        first = max(0, ends[0] - w) if w else 0
        cached += max(0, n - first)
    if case["op"] == "weigh":
        io = len(lens) * m * Q * (2 * D + 4) + (8 if case["add"] else 4) * H * sum(lens)
        return {"bytes": cached * H * row + io + 4 * cached // case["block"], "flops": 2 * seen * Q * D}
    io = len(lens) * m * Q * (4 * D + 4)
    return {"bytes": cached * 2 * H * row + io + 4 * cached // case["block"], "flops": 4 * seen * Q * D}


# -- inputs ---------------------------------------------------------------------

def _normal(gen, shape, dtype, spread=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * spread).to(dtype)


def _tables(case, gen, longest):
    """A decode pool's size and block tables for requests of `longest` tokens each list: a permutation's blocks."""
    B = case["block"]
    need = [[-(-(n + 1) // B) for n in lens] for lens in longest]  # one slot more, as an engine keeps
    blocks = max(1, math.ceil(1.1 * sum(map(sum, need))))
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    tables, start = [], 0
    for counts in need:
        at = torch.zeros((len(counts), max(counts)), dtype=torch.int64)
        for r, k in enumerate(counts):
            at[r, :k] = torch.arange(start, start + k)
            start += k
        tables.append(order[at.to("cuda")].contiguous())
    return blocks, tables


def _four_bits(x):
    """Rows [..., D] in 32 bits as (codes [..., D / 2], block scales [..., D / 16]), both uint8."""
    y = x.unflatten(-1, (-1, GROUP))
    b = (y.abs().amax(-1) * torch.tensor(1.0 / 6.0, dtype=torch.float32, device=x.device)).clamp(max=448.0)
    b = b.to(torch.float8_e4m3fn)
    b = torch.where(b.float() < 2.0 ** -9, torch.full_like(b.float(), 2.0 ** -9), b.float())
    y = y * (1.0 / b)[..., None]
    a = y.abs()
    code = torch.zeros_like(y, dtype=torch.uint8)
    # the border of two neighbours goes to the one whose code is even
    for low, border in enumerate([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]):
        code += ((a > border) if low % 2 == 0 else (a >= border)).to(torch.uint8)
    code += 8 * torch.signbit(y).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), b.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, scales):
    """What codes and block scales stand for, in 32 bits."""
    one = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    one = torch.cat([one, -one])
    both = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)   # of each byte
    x = both[codes.int()].flatten(-2).unflatten(-1, (-1, GROUP))
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _views(pool, case, blocks):
    """A 4-bit pool's codes [2][N][B][H][D / 2] and block scales [2][N][B][H][D / 16]."""
    D = case["dim"]
    rows = 2 * blocks * case["block"] * case["heads"]
    shape = (2, blocks, case["block"], case["heads"])
    return pool[:rows * (D // 2)].view(shape + (D // 2,)), pool[rows * (D // 2):].view(shape + (D // GROUP,))


def _filled(case, gen, blocks):
    """A pool of normal values in the case's type."""
    B, H, D = case["block"], case["heads"], case["dim"]
    if case["pool"] == "e2m1":
        pool = torch.empty(2 * blocks * B * H * (D // 2 + D // GROUP), dtype=torch.uint8, device="cuda")
        codes, scales = _views(pool, case, blocks)
        some = max(1, (1 << 26) // (B * H * D))                   # blocks at a time
        for comp in range(2):
            for at in range(0, blocks, some):
                x = torch.randn((min(some, blocks - at), B, H, D), generator=gen, device="cuda")
                codes[comp, at:at + some], scales[comp, at:at + some] = _four_bits(x)
        return pool
    if case["pool"] == "e4m3":
        x = torch.randn((1, 2, blocks, B, H, D), generator=gen, device="cuda") * 16.0
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _normal(gen, (1, 2, blocks, B, H, D), TORCH[case["pool"]])


def _inputs(case, seed):
    """The values of a case, from the seed alone: a dict of tensors on the GPU."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, H, D = TORCH[case["type"]], case["heads"], case["dim"]
    lens = lengths(case)
    R = len(lens)
    s = {"case": case, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "plane": None}
    if case["op"] == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        s["blocks"], (s["table"], s["into"]) = _tables(case, gen, [lens, kept])
    else:
        s["blocks"], (s["table"],) = _tables(case, gen, [lens])
    if case["pool"] == "e4m3":                                    # per head, near 1/16
        s["plane"] = (torch.rand((1, 2, H), generator=gen, device="cuda") + 0.5) / 16
    elif case["pool"] == "e2m1" and case["op"] != "append":
        s["plane"] = torch.rand((1, 2, H), generator=gen, device="cuda") + 0.5
    if case["op"] == "append":
        Q, new = case["queries"], fresh(case)
        T = sum(new)
        s["requests"] = torch.cat([torch.full((k,), r, dtype=torch.int32)
                                   for r, k in enumerate(new)]).to("cuda")
        s["positions"] = torch.cat([torch.arange(n - k, n, dtype=torch.int32)
                                    for n, k in zip(lens, new)]).to("cuda")
        s["k"], s["v"] = _normal(gen, (T, H, D), dt), _normal(gen, (T, H, D), dt)
        s["q"] = _normal(gen, (T, Q, D), dt)
        half = case["rotated"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
        s["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["pool"] = torch.zeros(2 * s["blocks"] * case["block"] * H * row_bytes(case), dtype=torch.uint8,
                                device="cuda")
        s["q_out"], s["k_out"], s["v_out"] = (torch.zeros_like(s[n]) for n in ("q", "k", "v"))
        return s
    s["pool"] = _filled(case, gen, s["blocks"])
    if case["op"] == "evict":
        # a few keys get much of the attention, many almost none, some exactly none
        S = max(lens + [1])
        w = torch.exp(2.0 * torch.randn((R, H, S), generator=gen, device="cuda") - 6.0)
        s["weights"] = torch.where(torch.rand((R, H, S), generator=gen, device="cuda") < 0.05,
                                   torch.zeros_like(w), w)
        s["weights_out"] = torch.zeros_like(w)
        s["slots"] = torch.full((R, H, case["keep"]), -1, dtype=torch.int32, device="cuda")
        return s
    m, Q = case["new"], case["queries"]
    s["q"] = _normal(gen, (R, m, Q, D), dt, 2.0)
    s["scale"] = D ** -0.5
    s["slopes"] = None
    if case["bias"]:                                              # 2^(-8 / Q), its square, ...
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Q + 1, dtype=torch.float64, device="cuda") / Q).float()
    s["lse"] = torch.empty((R, m, Q), dtype=torch.float32, device="cuda")
    if case["op"] == "weigh":
        s["lse"].copy_(_lse(_logits(s), case))                    # as the attention before it gave it
        s["before"] = torch.rand((R, H, max(lens + [1])), generator=gen, device="cuda")
        s["weights"] = s["before"].clone()
    else:
        s["out"] = torch.empty_like(s["q"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from prefill_decode_paged_gb300 import KVCache
        s["cache"] = KVCache(s["pool"], num_layers=1, num_components=2, kv_heads=case["heads"],
                             head_dim=case["dim"], block=case["block"], num_blocks=s["blocks"],
                             dtype=NUMBER[case["pool"]],
                             scales=None if s["plane"] is None else s["plane"].cpu().numpy(), per_head=True,
                             query_heads=case.get("queries", case["heads"]), max_requests=case["requests"],
                             max_new=max(1, case.get("new", 1)) if case["op"] != "append" else 1)
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


def _plain_append(s):
    case, B = s["case"], s["case"]["block"]
    pos, req = s["positions"].long(), s["requests"].long()
    block = s["table"][req, pos // B].long()
    angles = s["rotary"][pos][:, None, :]
    cos, sin = angles[..., :case["rotated"] // 2], angles[..., case["rotated"] // 2:]
    codes, scales = _views(s["pool"], case, s["blocks"])
    for comp, x in enumerate([_rotate(s["k"].float(), cos, sin, case), s["v"].float()]):
        c, b = _four_bits(x)
        codes[comp].index_put_((block, pos % B), c)
        scales[comp].index_put_((block, pos % B), b)
        s["kv"[comp] + "_out"].copy_(_values(codes[comp][block, pos % B], scales[comp][block, pos % B]))
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case))


def _gathered(s, comp):
    """One component's rows in request order, in 32 bits: [R, S, H, D]."""
    at = s["table"].long()
    if s["case"]["pool"] == "e2m1":
        codes, scales = _views(s["pool"], s["case"], s["blocks"])
        rows = _values(codes[comp][at], scales[comp][at]).flatten(1, 2)
    else:
        rows = s["pool"][0, comp][at].flatten(1, 2)
        rows = rows.view(torch.float8_e4m3fn).float() if s["case"]["pool"] == "e4m3" else rows.float()
    return rows if s["plane"] is None else rows * s["plane"][0, comp][:, None]


def _logits(s):
    """[R, H, m * G, S], minus infinity where a query does not see a key."""
    case = s["case"]
    R, m, Q, D = s["q"].shape
    H, w = case["heads"], case["window"]
    keys = _gathered(s, 0)                                        # [R, S, H, D]
    q = s["q"].float().view(R, m, H, Q // H, D).permute(0, 2, 1, 3, 4).reshape(R, H, -1, D)
    x = torch.matmul(q, keys.permute(0, 2, 3, 1)) * s["scale"]    # [R, H, m * G, S]
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    at = torch.arange(keys.shape[1], device="cuda")[None, None, :]
    end = s["lens"].long()[:, None] - m + torch.arange(m, device="cuda")[None, :]
    away = at - end[:, :, None]                                   # [R, m, S]
    if s["slopes"] is not None:
        # [R, H, m, G, S]
        bias = s["slopes"].view(1, H, 1, Q // H, 1) * away[:, None, :, None, :].float()
        x = x + bias.reshape(R, H, -1, keys.shape[1])
    seen = away <= 0
    if w:
        seen = seen & (away > -w)
    seen = seen[:, None, :, None, :].expand(R, H, m, Q // H, -1).reshape(R, H, -1, keys.shape[1])
    return torch.where(seen, x, torch.full_like(x, -math.inf))


def _back(x, case):
    """[R, H, m * G, V] as [R, m, Q, V]."""
    R, H, m = x.shape[0], case["heads"], case["new"]
    return x.view(R, H, m, -1, x.shape[-1]).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _lse(x, case):
    top = x.amax(-1, keepdim=True)
    base = torch.where(top > -math.inf, top, torch.zeros_like(top))
    return _back(base + torch.log(torch.exp(x - base).sum(-1, keepdim=True)), case)[..., 0]


def _plain_attend(s):
    x = _logits(s)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    s["out"].copy_(_back(torch.matmul(p, _gathered(s, 1).permute(0, 2, 1, 3)), s["case"]))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    s["lse"].copy_(_back(lse, s["case"])[..., 0])


def _plain_weigh(s):
    case = s["case"]
    x = _logits(s)
    R, m, Q = s["lse"].shape
    H, S = case["heads"], s["weights"].shape[2]
    lse = s["lse"].view(R, m, H, Q // H).permute(0, 2, 1, 3).reshape(R, H, -1, 1)
    p = torch.where(x > -math.inf, torch.exp(x - lse), torch.zeros_like(x)).sum(2)[..., :S]
    if p.shape[2] < S:
        p = torch.nn.functional.pad(p, (0, S - p.shape[2]))
    held = torch.arange(S, device="cuda")[None, None, :] < s["lens"].long()[:, None, None]
    old = s["before"]
    s["weights"].copy_(torch.where(held, p + old if case["add"] else p, old))


def _plain_evict(s):
    case, B = s["case"], s["case"]["block"]
    keep, recent, w = case["keep"], case["recent"], s["weights"]
    R, H, S = w.shape
    n = s["lens"].long()[:, None, None]
    at = torch.arange(S, device="cuda")[None, None, :]
    short, old = n <= keep, at < n - recent
    # the largest weights first, the lower slot first where they are equal
    order = torch.sort(torch.where(old, w, torch.full_like(w, -1.0)), dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(2, order, at.expand(R, H, S).contiguous())
    kept = (at < n) & (short | ~old | (rank < keep - recent))
    count = torch.minimum(n, torch.full_like(n, keep))
    # kept slots, ascending, ahead of the others
    src = torch.sort(torch.where(kept, at, at + S), dim=-1)[0][..., :keep] % S
    src = torch.nn.functional.pad(src, (0, keep - src.shape[2]))
    to = torch.arange(keep, device="cuda")[None, None, :]
    there = to < count
    s["slots"].copy_(torch.where(there, src.to(torch.int32), s["slots"]))
    moved = torch.where(there, w.gather(2, src), torch.zeros_like(w[:, :, :1]))
    moved = moved[..., :S] if keep >= S else torch.nn.functional.pad(moved, (0, S - keep))
    s["weights_out"].copy_(torch.where(at < n, moved, s["weights_out"]))
    r, h, i = torch.nonzero(there.expand(R, H, keep), as_tuple=True)
    j = src[r, h, i]
    a, b = s["table"][r, j // B].long(), s["into"][r, i // B].long()
    for comp in range(2):
        plane = s["pool"][0, comp]
        plane.index_put_((b, i % B, h), plane[a, j % B, h])


PLAIN = {"append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}


def _outputs(s):
    op = s["case"]["op"]
    if op == "append":
        return {"k": s["k_out"], "v": s["v_out"], "q": s["q_out"]}
    if op == "attend":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weigh":
        return {"weights": s["weights"]}
    pool = s["pool"].view(torch.float8_e4m3fn) if s["case"]["pool"] == "e4m3" else s["pool"]
    return {"pool": pool, "weights": s["weights_out"], "slots": s["slots"]}


def run(s):
    case = s["case"]
    if not own:
        PLAIN[case["op"]](s)
        return _outputs(s)
    cache = s["cache"]
    if case["op"] == "append":
        cache.append(0, s["k"], s["v"], s["requests"], s["positions"], s["table"], rotary=s["rotary"],
                     interleaved=case["interleaved"], rotate_last=case["last"], q=s["q"], q_out=s["q_out"])
        cache.read(0, s["requests"], s["positions"], s["table"], k=s["k_out"], v=s["v_out"])
    elif case["op"] == "attend":
        cache.attend(0, s["q"], s["lens"], s["table"], out=s["out"], lse=s["lse"], scale=s["scale"],
                     window=case["window"], cap=case["cap"], slopes=s["slopes"])
    elif case["op"] == "weigh":
        if case["add"]:
            s["weights"].copy_(s["before"])                       # (each pass adds to the same)
        cache.weigh(0, s["q"], s["lse"], s["lens"], s["table"], s["weights"], add=case["add"],
                    scale=s["scale"], window=case["window"], cap=case["cap"], slopes=s["slopes"])
    else:
        cache.evict(0, s["weights"], s["lens"], s["table"], case["keep"], case["recent"], into=s["into"],
                    out=s["weights_out"], slots=s["slots"])
    return _outputs(s)


# -- the definitions in 64 bits -------------------------------------------------

def _nearest(x, lowest, bits, most):
    """x in 64 bits to the nearest number of `bits` bits and a power of two not below `lowest`; ties to even."""
    step = torch.exp2(torch.frexp(x)[1].double() - 1).clamp(min=lowest) * 2.0 ** (1 - bits)
    return (torch.round(x / step) * step).clamp(-most, most)


def _through_four_bits(x):
    """Rows [..., D] in 64 bits as a 4-bit pool holds them. (Three products are fp32 numbers by definition.)"""
    y = x.float().double().unflatten(-1, (-1, GROUP))
    sixth = float(torch.tensor(1.0 / 6.0, dtype=torch.float32))
    b = _nearest((y.abs().amax(-1, keepdim=True) * sixth).float().double(), 2.0 ** -6, 4, 448.0)
    b = b.clamp(min=2.0 ** -9)
    code = _nearest((y * (1.0 / b).float().double()).float().double(), 1.0, 2, 6.0)
    return (code * b).flatten(-2)


def _exact_append(s):
    case = s["case"]
    half = case["rotated"] // 2

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

    return {"k": _through_four_bits(turn(s["k"])), "v": _through_four_bits(s["v"].double()),
            "q": turn(s["q"])}


def _rows_of(s, comp, slots, h):
    """Head h's rows at these slots of a plane, in 64 bits."""
    case, D = s["case"], s["case"]["dim"]
    H = case["heads"]
    if case["pool"] == "e2m1":
        codes, scales = _views(s["pool"], case, s["blocks"])
        codes, scales = codes[comp].flatten(0, 1)[slots, h], scales[comp].flatten(0, 1)[slots, h]
        nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        e, f = (nib >> 1) & 3, nib & 1
        mag = torch.where(e == 0, 0.5 * f, (2.0 + f) * torch.exp2(e.double() - 2.0))
        rows = torch.where(nib >= 8, -mag, mag).double() * \
            scales.view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, -1)
    else:
        rows = s["pool"][0, comp].view(-1, H, D)[slots, h]
        rows = rows.view(torch.float8_e4m3fn).double() if case["pool"] == "e4m3" else rows.double()
    return rows if s["plane"] is None else rows * float(s["plane"][0, comp, h])


def _exact_scores(s):
    """For each request, new token and key head: (r, i, h, keys' positions, their slots, logits [G, keys])."""
    case = s["case"]
    R, m, Q, D = s["q"].shape
    H, w, B = case["heads"], case["window"], case["block"]
    G = Q // H
    for r, n in enumerate(lengths(case)):
        low = max(0, n - m + 1 - w) if w else 0
        j = torch.arange(low, n, device="cuda")
        if n == 0:
            continue
        slots = s["table"][r].long()[j // B] * B + j % B
        for h in range(H):
            keys = _rows_of(s, 0, slots, h)
            for i in range(m):
                last = n - m + i
                if last < 0:
                    continue
                first = max(0, last - w + 1) if w else 0
                x = s["q"][r, i, h * G:(h + 1) * G].double() @ keys[first - low:last + 1 - low].T * s["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if s["slopes"] is not None:
                    x = x + s["slopes"][h * G:(h + 1) * G].double()[:, None] * (j[first - low:last + 1 - low] - last)
                yield r, i, h, slice(first, last + 1), slots[first - low:last + 1 - low], x


def _exact_attend(s):
    G = s["case"]["queries"] // s["case"]["heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for r, i, h, _, slots, x in _exact_scores(s):
        z = torch.logsumexp(x, -1)
        lse[r, i, h * G:(h + 1) * G] = z
        out[r, i, h * G:(h + 1) * G] = torch.exp(x - z[:, None]) @ _rows_of(s, 1, slots, h)
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    case = s["case"]
    G = case["queries"] // case["heads"]
    w = s["before"].double()
    if not case["add"]:
        for r, n in enumerate(lengths(case)):
            w[r, :, :n] = 0.0
    for r, i, h, at, _, x in _exact_scores(s):
        w[r, h, at] += torch.exp(x - s["lse"][r, i, h * G:(h + 1) * G].double()[:, None]).sum(0)
    return {"weights": w}


def _exact_evict(s):
    case, B, keep = s["case"], s["case"]["block"], s["case"]["keep"]
    pool = s["pool"].view(torch.float8_e4m3fn) if case["pool"] == "e4m3" else s["pool"]
    pool = pool.double()
    first, out = pool.clone(), s["weights_out"].double()
    slots = s["slots"].clone()
    for r, n in enumerate(lengths(case)):
        for h in range(case["heads"]):
            w = s["weights"][r, h, :n].tolist()
            old = n - case["recent"]
            best = sorted(range(max(0, old)), key=lambda j: (-w[j], j))[:keep - case["recent"]] \
                if n > keep else range(n)
            kept = sorted(best) + (list(range(old, n)) if n > keep else [])
            j = torch.tensor(kept, dtype=torch.int64, device="cuda")
            i = torch.arange(len(kept), device="cuda")
            a, b = s["table"][r, j // B].long(), s["into"][r, i // B].long()
            pool[0, :, b, i % B, h] = first[0, :, a, j % B, h]
            out[r, h, :n] = 0.0
            out[r, h, :len(kept)] = s["weights"][r, h, j].double()
            slots[r, h, :len(kept)] = j.to(torch.int32)
    return {"pool": pool, "weights": out, "slots": slots}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](s)
