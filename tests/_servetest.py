"""Plain statements of the operators around a paged cache in a serving step, for the
tests: 64-bit numbers, Python's whole numbers and lists; nothing of the library's arithmetic is
used here."""
from __future__ import annotations

from decimal import Decimal, getcontext

import numpy as np
import torch

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def far_angles(pos, freq):
    """Angles of far positions, reduced to one turn in 60 digits."""
    getcontext().prec = 60
    out = torch.zeros(len(pos), len(freq), dtype=torch.float64)
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            t = Decimal(int(p)) * Decimal(float(f)) / (2 * PI)
            out[i, j] = float((t - t.to_integral_value()) * 2 * PI)
    return out


def angles(pos, freq, axes):
    """[n][frequencies] of positions [n_axes][n]."""
    pos = pos.double()
    f = torch.tensor([float(x) for x in freq], dtype=torch.float64)
    if axes is None:
        return pos[0][:, None] * f
    return pos[torch.tensor(axes, dtype=torch.long)].T * f


def rotated(x, norm, eps, angle, interleaved, amplitude):
    """float64 result for rows x [n][heads][dim], and how far a binary32 computation of it may be off:
    the norm's sum of dim squares, half of it in the root, the root and two products: (dim / 2 + 8) 2^-24
    of each channel; sine and cosine within 2^-21 (two units of the last place, and an
    angle of at most half a turn rounded to 24 bits: 2^-24 pi); two roundings and the amplitude's."""
    x = x.double()
    n = angle.shape[1]
    if norm is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * norm.double()
    grain = (x.shape[-1] / 2 + 8) * 2.0 ** -24 if norm is not None else 0.0
    y, off = x.clone(), x.abs() * grain
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    first = 2 * torch.arange(n) if interleaved else torch.arange(n)
    second = first + (1 if interleaved else n)
    a, b = x[..., first], x[..., second]
    y[..., first] = (a * c - b * s) * amplitude
    y[..., second] = (a * s + b * c) * amplitude
    either = (a.abs() + b.abs()) * abs(amplitude) * (grain + 2.0 ** -21 + 2.0 ** -22)
    off[..., first], off[..., second] = either, either
    return y, off


def bf16_tol(y, off):
    return off * (1 + 2.0 ** -7) + 2.0 ** -8 * y.abs() + 2.0 ** -133


def e4m3_tol(code, off):
    """Of a code that stands for a quotient `code` known within `off`: half a step of 4 significant bits
    (2^-4 of the value at most), 2^-10 among the smallest."""
    return off * (1 + 2.0 ** -3) + torch.maximum(2.0 ** -4 * code.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64))


# ---------------------------------------------------------------- verification

def _row(t, i):
    r = t[i].astype(np.float32)
    r = np.where(np.isnan(r), np.float32(0), r)
    return np.clip(r, np.float32(0), np.float32(1))


def _rest(p, q, c):
    return np.maximum((p.astype(np.float64) - np.float64(c) * q.astype(np.float64)).astype(np.float32), np.float32(0))


def _units(r):
    return np.rint(r.astype(np.float64) * 2.0 ** 44).astype(np.int64)


def verify(probs, draft, tokens, parents, uniform, cu, vocab, distinct):
    """(accepted, paths as lists of rows, next tokens) of well-formed requests."""
    accepted, paths, nxt = [], [], []
    for r in range(len(cu) - 1):
        a, n = cu[r], cu[r + 1] - cu[r]
        if n == 0:
            accepted.append(0)
            paths.append([])
            nxt.append(-1)
            continue
        here, path = 0, [a]
        p = _row(probs, a)
        q = None if draft is None else _row(draft, a)
        c, left, unseen, gone = 0.0, 1.0, 1.0, set()
        for i in range(1, n):
            par = i - 1 if parents is None else int(parents[a + i])
            if par != here:
                continue
            x, u = int(tokens[a + i]), float(uniform[a + i])
            if draft is None:
                w = 0.0 if x in gone else float(p[x])
                take = u * left < w
                if not take:
                    left = max(left - w, 0.0)
                    gone.add(x)
            else:
                rest = float(_rest(p[x:x + 1], q[x:x + 1], c)[0])
                take = u * float(q[x]) * left < rest * unseen
                if not take:
                    if unseen > 0:
                        c = float(np.float32(c + left / unseen))
                    if distinct:
                        unseen = max(unseen - float(q[x]), 0.0)
                    left = int(_units(_rest(p, q, c)).sum()) / 2.0 ** 44
            if take:
                here = i
                path.append(a + i)
                p = _row(probs, a + i)
                q = None if draft is None else _row(draft, a + i)
                c, left, unseen, gone = 0.0, 1.0, 1.0, set()
        w = _units(p if draft is None else _rest(p, q, c))
        for x in gone:
            w[x] = 0
        if w.sum() == 0:
            w = _units(p)
        total = int(w.sum())
        if total:
            t = min(int(np.floor(np.float64(uniform[a]) * np.float64(total))), total - 1)
            nxt.append(int(np.searchsorted(np.cumsum(w), t, side="right")))
        else:
            nxt.append(-1)
        accepted.append(len(path))
        paths.append(path)
    return accepted, paths, nxt


# ---------------------------------------------------------------- pages

def fork(page, pool, parents, ctx, table, have, free, state, trim):
    """(rows, page counts, lengths, ring, ring state, copies) in plain lists."""
    head, count = state
    free, size = list(free), len(free)
    n = len(ctx)
    parents = list(range(n)) if parents is None else parents
    groups = {}
    for s, r in enumerate(parents):
        if r >= 0 and ctx[r] >= 0:
            groups.setdefault(r, []).append(s)
    heir = {r: (r if r in kids else min(kids)) for r, kids in groups.items()}
    rows, lens, copies, taken = [], [], [], 0
    for s, r in enumerate(parents):
        copy = (-1, -1, 0)
        if r < 0 or ctx[r] < 0:
            rows.append([])
            lens.append(-1)
            copies.append(copy)
            continue
        whole, part = divmod(ctx[r], page)
        if heir[r] == s:
            row = table[r][:whole + (part > 0)] if trim else table[r][:have[r]]
        else:
            row = table[r][:whole]
            if part:
                new = free[(head + taken) % size]
                taken += 1
                copy = (table[r][whole], new, part)
                row = row + [new]
        rows.append(row)
        lens.append(ctx[r])
        copies.append(copy)
    before = {p for r in range(n) for p in table[r][:have[r]]}
    after = {p for row in rows for p in row}
    freed = sorted(before - after)
    for i, p in enumerate(freed):
        free[(head + count + i) % size] = p
    return rows, [len(r) for r in rows], lens, free, [(head + taken) % max(size, 1), count - taken + len(freed)], copies


def compact(pool, table, have):
    """(rows, ring's pages, moves)."""
    held = sorted({p for r, h in enumerate(have) for p in table[r][:h]})
    live = len(held)
    holes = sorted(set(range(live)) - set(held))
    far = [p for p in held if p >= live]
    to = dict(zip(far, holes))
    return [[to.get(p, p) for p in table[r][:h]] for r, h in enumerate(have)], list(range(live, pool)), list(zip(far, holes))
