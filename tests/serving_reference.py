"""Plain 64-bit forms of the serving operators, on CPU or GPU tensors, for their tests."""
from __future__ import annotations

import math

import torch


def freqs(rot, base=10000.0, pi_scale=1.0, original_len=0, slow=1.0, fast=32.0):
    """Radians a token of each pair, from the definition."""
    out = []
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        if original_len:
            keep = min(1.0, max(0.0, (theta * original_len / (2 * math.pi) - slow) / (fast - slow)))
            out.append(theta * keep + theta / pi_scale * (1 - keep))
        else:
            out.append(theta / pi_scale)
    return torch.tensor(out, dtype=torch.float64)


def rope(x, positions, theta, layout, mscale=1.0, inverse=False):
    """x [B, N, H, d]; positions [B, N]."""
    y = x.double().clone()
    r = 2 * theta.numel()
    phi = (positions.double().unsqueeze(-1) * theta.to(x.device)).unsqueeze(-2)
    c, s = mscale * phi.cos(), mscale * phi.sin() * (-1 if inverse else 1)
    even, odd = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = y[..., even].clone(), y[..., odd].clone()
    y[..., even], y[..., odd] = a * c - b * s, a * s + b * c
    return y


def quantised(x):
    """The value in 64 bits that the cache holds of finite x [T, H, d], and the groups' scales."""
    g = x.float().clamp(-65504, 65504).unflatten(-1, (-1, 32))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale, low = ((high - low) * (1 / 15)).half(), low.half().float()
    # a top value that would round beyond fp16 (65504 + half a step) takes the next smaller scale
    scale = torch.where(scale.double() * 15 + low.double() >= 65520, (scale.view(torch.int16) - 1).view(torch.float16), scale).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.where(scale > 0, ((g - low) / safe).round().clamp(0, 15), torch.zeros_like(g))
    return (code.double() * scale.double() + low.double()).flatten(-2), scale.squeeze(-1)


def attention(q, k, v, keys, scale):
    """One request: q [n, Hq, d]; k, v [L, Hkv, d] in 64 bits; row i sees keys[i] of them.
    Returns o, lse [n, Hq], and sum p |v| (for error bounds)."""
    n, Hq, d = q.shape
    H = k.shape[1]
    qd = q.double().view(n, H, Hq // H, d)
    s = torch.einsum("nhgd,lhd->nhgl", qd, k) * scale
    hidden = torch.arange(k.shape[0], device=q.device) >= torch.tensor(keys, device=q.device).view(-1, 1)
    s = s.masked_fill(hidden.view(n, 1, 1, -1), -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[0] else torch.full(s.shape[:-1], -math.inf, device=q.device, dtype=torch.float64)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse).unsqueeze(-1))
    p = p.masked_fill(hidden.view(n, 1, 1, -1), 0.0)  # hidden keys add nothing, whatever they hold

    def times(x):
        seen = torch.where(hidden.all(0).view(-1, 1, 1), torch.zeros_like(x), x)
        return torch.einsum("nhgl,lhd->nhgd", p, seen).reshape(n, Hq, d)

    return times(v), lse.reshape(n, Hq), times(v.abs())


def plan(cached, new, free, free_count, table, P, T):
    """The step's plan by loops over requests and tokens, on lists."""
    table = [list(r) for r in table]
    left, row, taken = min(max(free_count, 0), len(free)), 0, 0
    positions, slots = [0] * T, [-1] * T
    cu, lens, out = [], [], 0
    pages_before = 0
    for r, (c, n) in enumerate(zip(cached, new)):
        cu.append(row)
        if c < 0 or n < 0:
            lens.append(c)
            out += 1
            continue
        held, need = -(-c // P), -(-(c + n) // P)
        fits = need <= len(table[r])
        more = need - held if fits else 0
        ok = fits and (more == 0 or pages_before + more <= left) and (n == 0 or row + n <= T)
        if ok:
            for j in range(more):
                table[r][held + j] = free[left - 1 - pages_before - j]
            taken = pages_before + more if more else taken
        out += not ok
        for i in range(n):
            if row + i < T:
                positions[row + i] = c + i
                if ok:
                    slots[row + i] = table[r][(c + i) // P] * P + (c + i) % P
        pages_before += more
        row += n
        lens.append(c + n if ok else c)
    cu.append(row)
    return cu, lens, positions, slots, left - taken, out, table
