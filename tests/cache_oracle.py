"""Appending to a paged cache, attention over it and keeping a path: the definitions in 64 bits, one
sequence after another, with bounds for a 32-bit evaluation in any order of summation."""
from __future__ import annotations

import numpy as np

from tests.ops_oracle import HALF, U

# what the split of a binary32 product drops, relative to the factors' magnitudes: the rests' product
# (2^-10 2^-10), and what the instruction cuts from each rest (2^-10 of 2^-10)
SPLIT = 3 * 2.0 ** -20


def place(table_row, slot, page, pages):
    """(page, slot in it), or None where there is none."""
    if not 0 <= slot < len(table_row) * page:
        return None
    p = int(table_row[slot // page])
    return (p, slot % page) if 0 <= p < pages else None


def append(k, v, q, kc, vc, table, starts, positions=None, counts=None, inv_freq=None, pairs=False):
    """New keys, values (caches' copies, binary64), queries, and the bounds of the keys and queries; flag."""
    k, v, kc, vc = (np.array(z, np.float64) for z in (k, v, kc, vc))
    b, n, hkv, d = k.shape
    bound_k = np.zeros_like(kc)
    out_q = bound_q = None
    if q is not None:
        q = np.array(q, np.float64)
        out_q, bound_q = np.zeros_like(q), np.zeros_like(q)
    pages, page = kc.shape[:2]
    flag = False

    def turn(x, pos):
        x = x.copy()
        err = np.zeros_like(x)
        if inv_freq is None or len(inv_freq) == 0:
            return x, err
        half = len(inv_freq)
        th = pos * np.asarray(inv_freq, np.float64)
        one = np.arange(0, 2 * half, 2) if pairs else np.arange(half)
        two = one + (1 if pairs else half)
        a, c = x[:, one].copy(), x[:, two].copy()
        x[:, one], x[:, two] = a * np.cos(th) - c * np.sin(th), c * np.cos(th) + a * np.sin(th)
        # the angle to 2^-22 with the functions' own error, then two products and a sum
        err[:, one] = err[:, two] = (np.abs(a) + np.abs(c)) * (2.0 ** -22 + 4 * U)
        return x, err

    for i in range(b):
        m = n if counts is None else int(counts[i])
        flag |= not 0 <= m <= n or int(starts[i]) < 0
        for t in range(min(max(m, 0), n)):
            pos = int(starts[i]) + t if positions is None else int(positions[i, t])
            if q is not None:
                out_q[i, t], bound_q[i, t] = turn(q[i, t], pos)
            at = place(table[i], int(starts[i]) + t, page, pages) if starts[i] >= 0 else None
            if at is None:
                flag = True
                continue
            kc[at], bound_k[at] = turn(k[i, t], pos)
            vc[at] = v[i, t]
    return dict(k=kc, v=vc, q=out_q, bk=bound_k, bq=bound_q, flag=flag)


def attend(q, kc, vc, table, lens, mask=None, counts=None, scale=None, kind="f32"):
    """out, lse and their bounds; flag."""
    q, kc, vc = (np.asarray(z, np.float64) for z in (q, kc, vc))
    b, n, hq, d = q.shape
    pages, page, hkv, _ = kc.shape
    g = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros(q.shape), np.full((b, n, hq), -np.inf)
    bout, blse = np.zeros(q.shape), np.zeros((b, n, hq))
    flag = False
    for i in range(b):
        room = len(table[i]) * page
        m = n if counts is None else int(counts[i])
        ln = int(lens[i])
        flag |= ln < 0 or not 0 <= m <= n or ln + m > room
        m, ln = min(max(m, 0), n), min(max(ln, 0), room)
        for t in range(m):
            see = list(range(ln))
            for j in range(m):
                sees = j <= t if mask is None else (mask[i] if mask.ndim == 3 else mask)[t, j]
                if sees and ln + j < room:
                    see.append(ln + j)
            at = [place(table[i], s, page, pages) for s in see]
            flag |= any(z is None for z in at)
            at = [z for z in at if z is not None]
            if not at:
                continue
            ps, ss = (np.array(z) for z in zip(*at))
            for h in range(hq):
                x, y = kc[ps, ss, h // g], vc[ps, ss, h // g]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (x @ q[i, t, h])
                    big = abs(scale) * (np.abs(x) @ np.abs(q[i, t, h]))
                    top = s.max()
                    if top == -np.inf:
                        continue
                    e = np.exp(s - top)
                    lse[i, t, h] = top + np.log(e.sum())
                    p = e / e.sum()
                    out[i, t, h] = np.where(p > 0, p, 0) @ y
                    # a matrix instruction may cut each sum (2 U); the scores' product with the scale and their difference
                    es = np.max(big) * (2 * (d + 4) * U + (SPLIT if kind == "f32" else 0)) + 8 * U * (np.abs(s).max() + 1)
                    terms = (len(at) / 4 + 64) * 2 * U       # a thread's sums, then a few joins
                    blse[i, t, h] = es + terms + 4 * U * abs(lse[i, t, h])
                    bout[i, t, h] = (p @ np.abs(y)) * (2 * es + 2 * terms + (SPLIT if kind == "f32" else HALF[kind]))
    return dict(out=out, lse=lse, bout=bout, blse=blse, flag=flag)


def keep(kc, vc, table, lens, path, kept, nodes=1 << 20):
    """The caches after the moves; flag."""
    kc, vc = np.array(kc), np.array(vc)
    pages, page = kc.shape[:2]
    flag = False
    for i in range(len(lens)):
        m = int(kept[i])
        flag |= not 0 <= m <= path.shape[1]
        m = min(max(m, 0), path.shape[1])
        old_k, old_v, before = kc.copy(), vc.copy(), -1
        for j in range(m):
            x = int(path[i, j])
            src = place(table[i], int(lens[i]) + x, page, pages) if lens[i] >= 0 else None
            dst = place(table[i], int(lens[i]) + j, page, pages) if lens[i] >= 0 else None
            if not before < x < nodes or src is None or dst is None:
                flag = True
                break
            kc[dst], vc[dst] = old_k[src], old_v[src]
            before = x
    return dict(k=kc, v=vc, flag=flag)
