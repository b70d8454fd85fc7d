"""Plain 64-bit statements of the paged-cache operators, for the tests: nothing
of the library's arithmetic is used here."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def values(pool: torch.Tensor, scale) -> torch.Tensor:
    """float64 values of a pool [pages][tokens][heads][dim] of codes."""
    p = pool.cpu()
    if p.element_size() == 2:
        return p.view(torch.bfloat16).double()
    x = p.contiguous().view(E4M3).double()
    return x if scale is None else x * scale.cpu().double()[:, None]


def page_map(page, pool_pages, max_pages, cap, ctx, new, table, n_pages, free, state):
    """The page map in plain lists: (table, n_pages, free, state, cu, slots)."""
    table, free = [list(r) for r in table], list(free)
    head, count = state
    size = len(free)
    out, cu, slots, taken, pushed = [], [0], [], 0, []
    for r, (c, w, h) in enumerate(zip(ctx, new, n_pages)):
        if c < 0:
            pushed += table[r][:h]
            out.append(0)
            cu.append(cu[-1])
            continue
        want = -(-(c + w) // page)
        for j in range(h, want):
            table[r][j] = free[(head + taken) % size]
            taken += 1
        out.append(max(h, want))
        cu.append(cu[-1] + w)
        for p in range(c, c + w):
            g = table[r][p // page]
            slots.append(g * page + p % page if 0 <= g < pool_pages else -1)
    for i, p in enumerate(pushed):
        free[(head + count + i) % size] = p
    slots += [-1] * (cap - len(slots))
    return table, out, free, [(head + taken) % max(size, 1), count - taken + len(pushed)], cu, slots


def to_e4m3(x: torch.Tensor) -> torch.Tensor:
    """Codes of float64 values: nearest of the 8-bit grid, ties to even, saturated; by search
    over every finite code."""
    codes = torch.arange(127, dtype=torch.uint8)
    grid = codes.view(E4M3).double()                       # ascending, 0 .. 448
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a.flatten()).clamp(max=126).view(a.shape)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    even = torch.where(hi % 2 == 0, hi, lo)
    c = torch.where(up < down, hi, torch.where(down < up, lo, even))
    c = torch.where(torch.isnan(x), torch.full_like(c, 127), c)
    return (c | torch.where(torch.signbit(x), 128, 0)).to(torch.uint8)


def visible(masks, i, j):
    return j <= i if masks is None else bool((int(masks[i][j // 64]) >> (j % 64)) & 1)


def attention(q, k, v, ks, vs, table, ctx, cu, mask, scale, q_eps=0.0, p_eps=2.0 ** -8):
    """Outputs, log-sums and the largest error each may have, in float64:
      o        sum w V / sum w over the visible positions
      lse      log sum w
      tol      half a step of the bf16 output (2^-8 |o|); half a step of each weight
               (p_eps) against A = sum w |V| / sum w; the binary32 score sums, each off
               by d_p = ((dim + 8) 2^-24 + q_eps) scale sum |q K_p|, which moves its weight by
               up to exp(d_p) - 1 of it in numerator and denominator; and 2^-16 A for the
               exponentials, the running sums and the last division
      lse_tol  the same d_p, and the rounding of the sum and the logarithm
    Rows outside every request are NaN."""
    dim = q.shape[2]
    kv, vv, qd = values(k, ks), values(v, vs), q.cpu().double()
    heads, kvh = q.shape[1], k.shape[2]
    page = k.shape[1]
    o = torch.full(q.shape, math.nan, dtype=torch.float64)
    tol = torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    lse_tol = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    table, ctx, cu = table.cpu(), ctx.cpu().tolist(), cu.cpu().tolist()
    for r in range(len(ctx)):
        n = cu[r + 1] - cu[r]
        if n <= 0:
            continue
        end = ctx[r] + n
        pos = torch.arange(end)
        ids = table[r].long()[pos // page]
        kk, ve = kv[ids, pos % page], vv[ids, pos % page]             # [end, kvh, dim]
        masks = None if mask is None else mask[cu[r]:cu[r + 1]].cpu().tolist()
        for i in range(n):
            see = torch.tensor([p < ctx[r] or visible(masks, i, p - ctx[r]) for p in range(end)], dtype=torch.bool)
            kr, vr = kk[see], ve[see]
            for g in range(heads):
                h = g // (heads // kvh)
                row = qd[cu[r] + i, g]
                if kr.shape[0] == 0:
                    o[cu[r] + i, g], tol[cu[r] + i, g] = 0.0, 0.0
                    lse[cu[r] + i, g], lse_tol[cu[r] + i, g] = -math.inf, 0.0
                    continue
                s = kr[:, h] @ row * scale
                d = ((dim + 8) * 2.0 ** -24 + q_eps) * (kr[:, h].abs() @ row.abs()) * abs(scale)
                w = torch.softmax(s, 0)
                wd = torch.where(w > 0, w * torch.expm1(d), torch.zeros_like(w))
                z = w @ vr[:, h]
                av = vr[:, h].abs()
                o[cu[r] + i, g] = z
                tol[cu[r] + i, g] = (2.0 ** -8 * z.abs() + (p_eps + 2.0 ** -16) * (w @ av) + wd @ av + wd.sum() * z.abs()
                                     + 2.0 ** -133)
                l = torch.logsumexp(s, 0)
                lse[cu[r] + i, g] = l
                lse_tol[cu[r] + i, g] = wd.sum() + 2.0 ** -16 + 2.0 ** -22 * l.abs()
    return o, tol, lse, lse_tol


def tree_bits(parents):
    """Ancestor-or-self bits of nodes whose parents come before them (-1: the context)."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return bits


def mask_tensor(rows, words):
    t = torch.zeros(len(rows), words, dtype=torch.int64)
    for i, b in enumerate(rows):
        for w in range(words):
            x = (b >> (64 * w)) & ((1 << 64) - 1)
            t[i, w] = x - (1 << 64) if x >> 63 else x
    return t
