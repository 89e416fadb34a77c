"""Cases, plain forms and exact forms of the serving operators: rotary positions, page plans, the 4-bit cache and attention
over it.

The shapes are the LLaMA2-7B (32 heads) and LLaMA2-70B (64 query heads on 8 kv heads) layers of ``workloads.py``, at the
context lengths of its runs (up to 102400 tokens), as a server sees them: a request at a time or a batch, one token a step, a
few drafted tokens, or a chunk of a prompt.

The 4-bit cache. A page of a kv head is a row of sub-blocks of 16 tokens, each of 20 d bytes (nG = d / 32 groups of 32
channels): k codes (8 d bytes), k scales and k minima (fp16 [16][nG] each), v codes (8 d bytes), v (scale, minimum) pairs
(fp16 [16][nG][2]). A value is minimum + scale * code. ``_places`` has the byte and shift of each code.
"""
import math
import random

import torch

own = False

DEV = "cuda"
FP16_MAX = 65504.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one request: the latency of a decode step's rotation (7B layer, 32k extension by interpolation)
        {"name": "rope token", "op": "rope", "B": 1, "N": 1, "Hq": 32, "Hkv": 32, "d": 128, "rot": 128, "layout": "interleaved",
         "base": 10000.0, "pi": 8.0, "orig": 0, "mscale": 1.0, "far": 32767, "dtype": "bf16", "grad": False},
        # the 7B 32k training step's rotation and its gradient
        {"name": "rope train 32k", "op": "rope", "B": 1, "N": 32768, "Hq": 32, "Hkv": 32, "d": 128, "rot": 128,
         "layout": "interleaved", "base": 10000.0, "pi": 8.0, "orig": 0, "mscale": 1.0, "far": 32768, "dtype": "bf16", "grad": True},
        # a padded batch in fp32, halves layout, 64 of 96 channels rotated, frequencies interpolated by parts
        {"name": "rope half part f32", "op": "rope", "B": 3, "N": 1111, "Hq": 24, "Hkv": 8, "d": 96, "rot": 64, "layout": "half",
         "base": 10000.0, "pi": 25.0, "orig": 4096, "mscale": 1.25, "far": 102399, "dtype": "f32", "grad": False},
        # pages and slots of one decode step of 64 requests
        {"name": "plan tokens", "op": "plan", "R": 64, "ctx": 8192, "new": 1, "P": 64, "width": 512},
        # pages and slots of a batch of prompts that arrive at once, some continuing, many pages each
        {"name": "plan prompts", "op": "plan", "R": 509, "ctx": 2000, "new": 4001, "P": 16, "width": 512},
        # one token of each of 64 requests into the 70B layer's cache
        {"name": "append tokens", "op": "append", "T": 64, "Hkv": 8, "d": 128, "P": 64, "dtype": "bf16"},
        # a 32k prompt into the 7B layer's cache
        {"name": "append prompt 32k", "op": "append", "T": 32768, "Hkv": 32, "d": 128, "P": 64, "dtype": "bf16"},
        # one short request, 7B layer: latency
        {"name": "attn token short", "op": "attn", "R": 1, "ctx": 1000, "new": 1, "Hq": 32, "Hkv": 32, "d": 128, "P": 64, "dtype": "bf16"},
        # one token over a ~100k context, 7B layer: the longest cache of the workloads
        {"name": "attn token 100k", "op": "attn", "R": 1, "ctx": 102400, "new": 1, "Hq": 32, "Hkv": 32, "d": 128, "P": 64, "dtype": "bf16"},
        # a batch of ragged requests up to 32k, 70B layer
        {"name": "attn batch 32k", "op": "attn", "R": 24, "ctx": 32768, "new": 1, "Hq": 64, "Hkv": 8, "d": 128, "P": 64, "dtype": "bf16"},
        # a few drafted tokens of each request are checked at once; small heads and small pages
        {"name": "attn drafted", "op": "attn", "R": 13, "ctx": 6001, "new": 5, "Hq": 32, "Hkv": 8, "d": 64, "P": 16, "dtype": "bf16"},
        # a chunk of a long prompt over what is cached of it, 70B layer
        {"name": "attn chunk", "op": "attn", "R": 2, "ctx": 16384, "new": 512, "Hq": 64, "Hkv": 8, "d": 128, "P": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "plan", "append", "attn", "attn"])
    if op == "rope":
        Hkv, d = rng.choice([1, 2, 8, 32]), rng.choice([64, 80, 96, 128, 256])
        Hq = Hkv * rng.choice([1, 3, 8] if Hkv < 32 else [1])
        B = rng.choice([1, 1, 2, 5])
        N = _log(rng, 1, max(1, min(32768, 32768 * 64 * 128 // (B * (Hq + Hkv) * d))))
        rot = rng.choice([d, d, d // 2, 32])
        return {"op": op, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "layout": rng.choice(["interleaved", "half"]),
                "base": rng.choice([10000.0, 80000.0]), "pi": rng.choice([1.0, 2.0, 8.0, 25.0]), "orig": rng.choice([0, 4096]),
                "mscale": rng.choice([1.0, 1.25]), "far": _log(rng, max(N, 128), 1 << 20), "dtype": rng.choice(["bf16", "bf16", "f32"]) if N < 8192 else "bf16",
                "grad": rng.random() < 0.5}
    if op == "plan":
        R, P = _log(rng, 1, 512), rng.choice([16, 32, 64, 128])
        new = rng.choice([1, 1, 4, _log(rng, 2, 4000)])
        ctx = _log(rng, 1, 7000)
        return {"op": op, "R": R, "ctx": ctx, "new": new, "P": P, "width": -(-(ctx + new) // P) + rng.randrange(9)}
    if op == "append":
        Hkv, d = rng.choice([1, 2, 8, 32]), rng.choice([64, 96, 128, 256])
        return {"op": op, "T": _log(rng, 1, min(65536, 32768 * 32 * 128 // (Hkv * d))), "Hkv": Hkv, "d": d, "P": rng.choice([16, 32, 64, 128]),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    Hkv, d = rng.choice([1, 2, 8, 8, 32]), rng.choice([64, 128, 128, 256])
    group = rng.choice([1, 4, 8, 16] if Hkv < 32 else [1])
    new = rng.choice([1, 1, 1, rng.randrange(2, 9), _log(rng, 16, 512)])
    R = _log(rng, 1, 64 if new < 16 else 2)
    most = 24 * 32768 * 8 * 128 // (2 * R * Hkv * d)
    if new >= 16:
        most = min(most, 2 * 16384 * 512 * 64 * 128 // (2 * R * new * Hkv * group * d))
    ctx = max(new, _log(rng, 1, max(2, min(102400, most))))
    f32 = new < 16 and R * ctx * Hkv * group * d < (1 << 28) and rng.random() < 0.15
    return {"op": op, "R": R, "ctx": ctx, "new": new, "Hq": Hkv * group, "Hkv": Hkv, "d": rng.choice([d, 96]) if f32 else d,
            "P": rng.choice([16, 32, 64, 128]), "dtype": "f32" if f32 else "bf16"}


def _lengths(case):
    """(cached, new) tokens of each request: ragged, the same for every seed; the first request has the largest of both."""
    rng = random.Random("%d %d %d" % (case["R"], case["ctx"], case["new"]))
    plan = case["op"] == "plan"
    cached, new = [], []
    for r in range(case["R"]):
        n = case["new"] if r == 0 or case["new"] == 1 else rng.randint(1, case["new"])
        full = case["ctx"] if r == 0 else rng.randint(max(1, case["ctx"] // 4), case["ctx"])
        if plan:  # `ctx` is what is cached before the step
            cached.append(full if r % 3 else 0 if case["new"] > 1 and r else full)
        else:  # `ctx` counts the step's own tokens, which are cached already
            cached.append(max(0, full - n))
        new.append(n)
    return cached, new


def work(case):
    op = case["op"]
    if op == "rope":
        T, es = case["B"] * case["N"], 2 if case["dtype"] == "bf16" else 4
        passes, heads = 2 if case["grad"] else 1, case["Hq"] + case["Hkv"]
        return {"bytes": passes * (2 * T * heads * case["d"] * es + 4 * T), "flops": passes * 3 * T * heads * case["rot"]}
    if op == "plan":
        cached, new = _lengths(case)
        pages = sum(-(-(c + n) // case["P"]) - -(-c // case["P"]) for c, n in zip(cached, new))
        return {"bytes": 8 * case["R"] + 8 * pages + 4 * (2 * case["R"] + 1) + 8 * sum(new) + 12, "flops": 0}
    if op == "append":
        n, es = case["T"] * case["Hkv"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 4 * n * es + 2 * 1.25 * n + 8 * case["T"], "flops": 10 * n}
    cached, new = _lengths(case)
    es = 2 if case["dtype"] == "bf16" else 4
    held = sum(cached) + sum(new)
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    return {"bytes": 1.25 * held * case["Hkv"] * case["d"] + 2 * sum(new) * case["Hq"] * case["d"] * es + 4 * sum(-(-(c + n) // case["P"]) for c, n in zip(cached, new)),
            "flops": 4 * case["Hq"] * case["d"] * pairs}


# ---------------------------------------------------------------------------------------------------------- the cache's layout

def _places(d):
    """Byte in the sub-block and shift of the code of each (token, channel): for k and for v."""
    n = d // 32
    u = torch.arange(16).view(16, 1)
    x = torch.arange(d).view(1, d)
    j = x // 32
    # k: row u; four lanes of nG words, a word of eight codes per (lane, group); with eight groups odd rows swap halves
    word = (x % 32) // 8 * n + (j ^ (4 * (u & 1)) if n == 8 else j + 0 * u)
    k_byte = u * (d // 2) + 4 * word + (x % 8) // 2
    k_shift = 4 * (x % 2) + 0 * u
    # v: even tokens of eight before odd ones; eight lanes of nG half-words, four codes each, turned by the row
    row = (u & 8) + (u & 7) // 2 + 4 * (u & 1)
    turn = 2 * (row & 3) if n == 8 else 4 * (row // 2 & 1) if n == 4 else 0 * row
    v_byte = 10 * d + row * (d // 2) + ((x % 32) // 4 ^ turn) * 2 * n + 2 * j + (x % 4) // 2
    v_shift = 4 * (x % 2) + 0 * u
    return k_byte, k_shift, v_byte, v_shift, row.view(16)


def _tables(d):
    """The same as orders: position in the region's row of 16 d codes (low nibble first) of each (token, channel), and v's rows."""
    k_byte, k_shift, v_byte, v_shift, row = _places(d)
    k = (2 * k_byte + k_shift // 4).reshape(-1)
    v = (2 * (v_byte - 10 * d) + v_shift // 4).reshape(-1)
    return {"k": k.to(DEV), "v": v.to(DEV), "row": row.to(DEV)}


def _quantise(x):
    """Codes, scale and minimum of groups of 32 channels (last axis), all in IEEE fp32; the two are rounded to fp16."""
    g = x.float().clamp(-FP16_MAX, FP16_MAX).unflatten(-1, (-1, 32))
    low, high = g.amin(-1), g.amax(-1)
    scale, low = ((high - low) / 15).half(), low.half()
    s, m = scale.float().unsqueeze(-1), low.float().unsqueeze(-1)
    code = torch.where(s > 0, ((g - m) / s).round().clamp(0, 15), torch.zeros_like(g))
    return code.flatten(-2), scale, low


def _pack(k, v, t):
    """Sub-blocks of k, v [S, 16, d]."""
    S, _, d = k.shape
    out = torch.empty(S, 20 * d, dtype=torch.uint8, device=k.device)
    for x, at, order in ((k, 0, t["k"]), (v, 10 * d, t["v"])):
        code, scale, low = _quantise(x)
        nib = torch.empty(S, 16 * d, dtype=torch.uint8, device=k.device)
        nib[:, order] = code.reshape(S, -1).to(torch.uint8)
        out[:, at:at + 8 * d] = nib[:, 0::2] | nib[:, 1::2] << 4
        if at == 0:
            out[:, 8 * d:9 * d] = scale.reshape(S, -1).view(torch.uint8)
            out[:, 9 * d:10 * d] = low.reshape(S, -1).view(torch.uint8)
        else:
            pairs = torch.empty(S, 16, d // 32, 2, dtype=torch.float16, device=k.device)
            pairs[:, t["row"]] = torch.stack((scale, low), -1)
            out[:, 18 * d:] = pairs.reshape(S, -1).view(torch.uint8)
    return out


def _unpack(sub, d, t):
    """k, v in fp32, [..., 16, d], of sub-blocks [..., 20 d]."""
    def codes(region, order):
        nib = torch.stack((region & 15, region >> 4), -1).flatten(-2)
        return nib.index_select(-1, order).unflatten(-1, (16, d // 32, 32)).float()

    half = sub[..., 8 * d:10 * d].contiguous().view(torch.float16).float().unflatten(-1, (2, 16, d // 32))
    pair = sub[..., 18 * d:].contiguous().view(torch.float16).float().unflatten(-1, (16, d // 32, 2)).index_select(-3, t["row"])
    k = codes(sub[..., :8 * d], t["k"]) * half[..., 0, :, :].unsqueeze(-1) + half[..., 1, :, :].unsqueeze(-1)
    v = codes(sub[..., 10 * d:18 * d], t["v"]) * pair[..., 0].unsqueeze(-1) + pair[..., 1].unsqueeze(-1)
    return k.flatten(-2), v.flatten(-2)


# --------------------------------------------------------------------------------------------------------------------- inputs

def _turns(case):
    """Turns per token of each channel pair: the table that a program keeps for its model's positions."""
    r = case["rot"]
    theta = torch.tensor([case["base"] ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)
    if case["orig"]:
        keep = ((case["orig"] * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / case["pi"])
    else:
        theta = theta / case["pi"]
    return (theta / (2 * math.pi)).to(DEV)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if op == "rope":
        B, N, t = case["B"], case["N"], DTYPES[case["dtype"]]
        s["q"], s["k"] = ((0.5 * normal(B, N, case[h], case["d"])).to(t) for h in ("Hq", "Hkv"))
        start = torch.randint(0, case["far"] - N + 1, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        s["positions"] = start + torch.arange(N, dtype=torch.int32, device=DEV)
        s["freqs"] = _turns(case)
        if case["grad"]:
            s["dq"], s["dk"] = normal(*s["q"].shape).to(t), normal(*s["k"].shape).to(t)
            s["q"].requires_grad_()
            s["k"].requires_grad_()
        return s
    if op == "plan":
        cached, new = _lengths(case)
        P, R = case["P"], case["R"]
        held = [-(-c // P) for c in cached]
        most = sum(-(-(c + n) // P) for c, n in zip(cached, new)) + 17
        pages = torch.randperm(most, generator=g, device=DEV).int()
        s["table"] = torch.zeros(R, case["width"], dtype=torch.int32, device=DEV)
        col = torch.arange(case["width"], device=DEV).view(1, -1)
        full = col < torch.tensor(held, device=DEV).view(-1, 1)
        s["table"][full] = pages[:sum(held)]
        s["free"] = pages[sum(held):].clone()
        s["free_count"] = _int([most - sum(held)])
        s["cached"], s["new"], s["T"] = _int(cached), _int(new), sum(new)
        return s
    P, Hkv, d = case["P"], case["Hkv"], case["d"]
    s["tables"] = _tables(d)
    if op == "append":
        T, t = case["T"], DTYPES[case["dtype"]]
        loud = 1 + 3 * (torch.rand(Hkv, d, generator=g, device=DEV) < 0.05)  # k has a few loud channels
        s["k"], s["v"] = (normal(T, Hkv, d) * loud).to(t), normal(T, Hkv, d).to(t)
        n_pages = -(-T // P) + 3
        page = torch.randperm(n_pages, generator=g, device=DEV).int()
        at = torch.arange(T, device=DEV)
        s["slots"] = page[at // P] * P + (at % P).int()
        s["cache"] = torch.zeros(n_pages, Hkv, P // 16, 20 * d, dtype=torch.uint8, device=DEV)
        return s
    cached, new = _lengths(case)
    lens = [c + n for c, n in zip(cached, new)]
    held = [-(-n // P) for n in lens]
    n_pages = sum(held) + 2
    loud = 1 + 3 * (torch.rand(Hkv, 1, 1, d, generator=g, device=DEV) < 0.05)
    s["cache"] = torch.empty(n_pages, Hkv, P // 16, 20 * d, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (Hkv * P * d))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        k, v = normal(n, Hkv, P // 16 * 16, d).view(n, Hkv, P // 16, 16, d) * loud, normal(n, Hkv, P // 16, 16, d)
        s["cache"][p:p + n] = _pack(k.flatten(0, 2), v.flatten(0, 2), s["tables"]).view(n, Hkv, P // 16, 20 * d)
    pages = torch.randperm(n_pages, generator=g, device=DEV).int()
    s["table"] = torch.zeros(case["R"], max(held), dtype=torch.int32, device=DEV)
    full = torch.arange(max(held), device=DEV).view(1, -1) < torch.tensor(held, device=DEV).view(-1, 1)
    s["table"][full] = pages[:sum(held)]
    s["lens"], s["max_new"] = _int(lens), max(new)
    s["cu_new"] = _int([sum(new[:r]) for r in range(len(new) + 1)])
    s["q"] = (1.5 * normal(sum(new), case["Hq"], d)).to(DTYPES[case["dtype"]])
    return s


# ----------------------------------------------------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, case):
    """x [B, N, H, d] rotated; cos, sin [B, N, 1, rot/2], the magnitude in them."""
    y, rest = x.float(), case["rot"]
    if case["layout"] == "half":
        a, b = y[..., :rest // 2], y[..., rest // 2:rest]
        z = torch.cat((a * cos - b * sin, a * sin + b * cos, y[..., rest:]), -1)
    else:
        a, b = y[..., 0:rest:2], y[..., 1:rest:2]
        z = torch.cat((torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2), y[..., rest:]), -1)
    return z.to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double().unsqueeze(-1) * s["freqs"]
    angle = (2 * math.pi * (angle - angle.round())).unsqueeze(-2)
    cos, sin = (c["mscale"] * angle.cos()).float(), (c["mscale"] * angle.sin()).float()
    with torch.no_grad():
        out = [_rotate(s["q"], cos, sin, c), _rotate(s["k"], cos, sin, c)]
        if c["grad"]:  # the rotation's transpose: the other way round
            out += [_rotate(s["dq"], cos, -sin, c), _rotate(s["dk"], cos, -sin, c)]
    return out


def _plain_plan(s):
    P, T, table, count = s["case"]["P"], s["T"], s["table"], s["free_count"]
    before, after = -(-s["cached"] // P), -(-(s["cached"] + s["new"]) // P)
    need = after - before
    first = need.cumsum(0) - need
    cu = torch.cat((torch.zeros_like(count), s["new"].cumsum(0)))
    col = torch.arange(table.shape[1], device=DEV).view(1, -1)
    taken = (col >= before.view(-1, 1)) & (col < after.view(-1, 1))
    at = count - 1 - (first.view(-1, 1) + col - before.view(-1, 1))
    table.copy_(torch.where(taken, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    pos = s["cached"][r] + t - cu[r]
    slots = table[r, pos // P] * P + pos % P
    return [table, cu.int(), (s["cached"] + s["new"]), pos.int(), slots.int(), (count - need.sum()).int()]


def _plain_append(s):
    c, cache, slots = s["case"], s["cache"], s["slots"].long()
    d, P, H, T, tab = c["d"], c["P"], c["Hkv"], slots.numel(), s["tables"]
    page, u, n = slots // P, slots % 16, d // 32
    k, v = _quantise(s["k"]), _quantise(s["v"])

    def put(at, row, width, x):  # `width` bytes of row `row` of the region at `at`, for every token and head
        byte = at + row.view(T, 1, 1) * width + torch.arange(width, device=DEV)
        cache.index_put_((page.view(T, 1, 1), torch.arange(H, device=DEV).view(1, H, 1), (slots % P // 16).view(T, 1, 1), byte), x)

    def in_order(code, order, row):  # a token's codes where they lie in its row
        place = order.view(16, d)[u] - (row * d).view(T, 1)
        nib = torch.zeros(T, H, d, dtype=torch.uint8, device=DEV)
        nib.scatter_(-1, place.unsqueeze(1).expand(T, H, d), code.to(torch.uint8))
        return nib[..., 0::2] | nib[..., 1::2] << 4

    row = tab["row"][u]
    put(0, u, d // 2, in_order(k[0], tab["k"], u))
    put(8 * d, u, 2 * n, k[1].view(torch.uint8))
    put(9 * d, u, 2 * n, k[2].view(torch.uint8))
    put(10 * d, row, d // 2, in_order(v[0], tab["v"], row))
    put(18 * d, row, 4 * n, torch.stack((v[1], v[2]), -1).flatten(-2).view(torch.uint8))
    value = lambda code, scale, low: (code * scale.float().unsqueeze(-1) + low.float().unsqueeze(-1)).flatten(-2)  # noqa: E731
    return [value(x[0].unflatten(-1, (n, 32)), x[1], x[2]).to(s["k"].dtype) for x in (k, v)]


def _plain_attn(s):
    c, tab = s["case"], s["table"].long()
    R, H, d, n = c["R"], c["Hkv"], c["d"], s["max_new"]
    group = c["Hq"] // H
    k, v = _unpack(s["cache"][tab], d, s["tables"])                  # [R, pages, H, P/16, 16, d]
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(R, H, -1, d)
    v = v.permute(0, 2, 1, 3, 4, 5).reshape(R, H, -1, d)
    i = torch.arange(n, device=DEV).view(1, n)
    count = (s["cu_new"][1:] - s["cu_new"][:-1]).view(R, 1)
    at = (s["cu_new"][:-1].view(R, 1) + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(R, n, H, group, d).permute(0, 2, 1, 3, 4).reshape(R, H, n * group, d)
    score = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    score = score.view(R, H, n, group, -1)
    last = s["lens"].view(R, 1) - count + i                          # a token sees the keys up to its own place
    hidden = torch.arange(k.shape[2], device=DEV).view(1, 1, -1) > last.unsqueeze(-1)
    score.masked_fill_(hidden.view(R, 1, n, 1, -1), -math.inf)
    score = (score - score.amax(-1, keepdim=True)).exp_()
    score /= score.sum(-1, keepdim=True)
    o = score.view(R, H, n * group, -1) @ v
    o = o.view(R, H, n, group, d).permute(0, 2, 1, 3, 4).reshape(R, n, c["Hq"], d).to(s["q"].dtype)
    t = torch.arange(s["q"].shape[0], device=DEV, dtype=torch.int32)
    r = torch.searchsorted(s["cu_new"], t, right=True) - 1
    return [o[r, t - s["cu_new"][r]]]


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[c["op"]](s)
    from longlora_shifted_sparse_b200 import s2attn as s2
    if c["op"] == "rope":
        q, k = s2.rope(s["q"], s["k"], s["positions"], s["freqs"], layout=c["layout"], mscale=c["mscale"])
        if not c["grad"]:
            return [q, k]
        return [q.detach(), k.detach(), *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))]
    if c["op"] == "plan":
        p = s2.page_plan(s["cached"], s["new"], s["free"], s["free_count"], s["table"], c["P"], s["T"])
        return [s["table"], p.cu_new, p.lens, p.positions, p.slots, p.free_count]
    if c["op"] == "append":
        s2.cache4_append(s["k"], s["v"], s["cache"], s["slots"])
        return list(s2.cache4_read(s["cache"], s["slots"], s["k"].dtype))
    if "ws" not in s:
        s["ws"] = s2.cache4_workspace(s["q"].device)
    return [s2.cache4_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu_new"], s["max_new"], ws=s["ws"])]


# ----------------------------------------------------------------------------------------------------------------- exact forms

def _exact_rope(c, s):
    r, two_pi = c["rot"], 2 * math.pi
    theta = []
    for i in range(r // 2):
        f = math.exp(-2.0 * i / r * math.log(c["base"]))
        if c["orig"]:
            g = min(1.0, max(0.0, (c["orig"] * f / two_pi - 1.0) / 31.0))
            f = g * f + (1.0 - g) * f / c["pi"]
        else:
            f /= c["pi"]
        theta.append(f)
    phi = s["positions"].double()[..., None, None] * torch.tensor(theta, dtype=torch.float64, device=DEV)
    z = torch.polar(torch.full_like(phi, c["mscale"]), phi)

    def turn(x, z):
        y = x.detach().double().clone()
        even, odd = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
        w = torch.complex(y[..., even], y[..., odd]) * z
        y[..., even], y[..., odd] = w.real, w.imag
        return y

    out = [turn(s["q"], z), turn(s["k"], z)]
    return out + [turn(s["dq"], z.conj()), turn(s["dk"], z.conj())] if c["grad"] else out


def _exact_append(c, s):
    def held(x):  # the format's own roundings in fp32 and fp16, the value in 64 bits
        T, H, d = x.shape
        y = x.float().clamp(-FP16_MAX, FP16_MAX).reshape(T, H, d // 32, 32)
        top, low = y.max(-1, keepdim=True).values, y.min(-1, keepdim=True).values
        scale = torch.div(top - low, 15.0).half().float()
        low = low.half().float()
        code = torch.div(y - low, torch.where(scale == 0, torch.ones_like(scale), scale)).round().clamp(0, 15)
        code[(scale == 0).expand_as(code)] = 0
        return (low.double() + scale.double() * code.double()).reshape(T, H, d)

    return [held(s["k"]), held(s["v"])]


def _exact_attn(c, s):
    H, d, P, Hq = c["Hkv"], c["d"], c["P"], c["Hq"]
    k_byte, k_shift, v_byte, v_shift, row = (x.to(DEV) for x in _places(d))
    u, j = torch.arange(16, device=DEV).view(16, 1), torch.arange(d, device=DEV).view(1, d) // 32

    def half(sub, at):  # the fp16 number at byte `at`, from its bits
        bits = sub[..., at].int() | sub[..., at + 1].int() << 8
        sign, e, m = 1.0 - 2.0 * (bits >> 15), (bits >> 10) & 31, (bits & 1023).double()
        return sign * torch.where(e == 0, m * 2.0 ** -24, torch.ldexp(1024 + m, (e - 25).double()))

    n = d // 32
    cu, lens, out = s["cu_new"].tolist(), s["lens"].tolist(), []
    for r, length in enumerate(lens):
        q = s["q"][cu[r]:cu[r + 1]].double().view(-1, H, Hq // H, d)
        for_heads = []
        for h in range(H):
            sub = s["cache"][s["table"][r, :-(-length // P)].long(), h].view(-1, 20 * d)
            k = (sub[:, k_byte] >> k_shift.to(torch.uint8) & 15) * half(sub, 8 * d + 2 * (u * n + j)) + half(sub, 9 * d + 2 * (u * n + j))
            vp = 18 * d + 4 * (row.view(16, 1) * n + j)
            v = (sub[:, v_byte] >> v_shift.to(torch.uint8) & 15) * half(sub, vp) + half(sub, vp + 2)
            k, v = k.reshape(-1, d)[:length], v.reshape(-1, d)[:length]
            a = torch.einsum("igx,jx->gij", q[:, h], k) * d ** -0.5
            own_place = torch.arange(length - q.shape[0], length, device=DEV).view(-1, 1)
            a = torch.where(torch.arange(length, device=DEV) <= own_place, a, -torch.inf)
            for_heads.append(torch.einsum("gij,jx->igx", torch.softmax(a, -1), v))
        out.append(torch.stack(for_heads, 1).reshape(-1, Hq, d))
    return [torch.cat(out)]


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    with torch.no_grad():
        return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](case, s)
