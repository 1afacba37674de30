"""The operators' definitions in 64 bits, one element after another, with error bounds for a
32-bit evaluation in any order of summation."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # half an ulp of binary32, relative
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # rounding to the type, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def distill(x, t, idx, tau, scale=None, teacher_lse=None):
    """loss, lse, grad and the bounds of loss, lse and grad (binary64 arrays) for rows x [N, V]."""
    x, t = np.asarray(x, np.float64), np.asarray(t, np.float64)
    n, v = x.shape
    loss, lse = np.zeros(n), np.zeros(n)
    grad, bgrad = np.zeros((n, v)), np.zeros((n, v))
    bloss, blse = np.zeros(n), np.zeros(n)
    for r in range(n):
        y = x[r] / tau
        m = y.max()
        lse[r] = -np.inf if m == -np.inf else tau * (m + np.log(np.exp(y - m).sum()))
        big = np.abs(x[r][np.isfinite(x[r])]).max(initial=0.0) + (abs(lse[r]) if np.isfinite(lse[r]) else 0.0)
        # lse = m + tau ln s: a few roundings of its size, and ln s to s's relative error over tau
        blse[r] = 4 * U * (big + tau * (16 + np.log(v) + big / tau))
        keep = [k for k in range(idx.shape[1]) if 0 <= idx[r, k] < v]
        if not keep:
            continue
        tk = np.array([t[r, k] for k in keep]) / tau
        if teacher_lse is not None:
            L = teacher_lse[r] / tau
        elif tk.max() == -np.inf:
            continue
        else:
            L = tk.max() + np.log(np.exp(tk - tk.max()).sum())
        q = np.exp(tk - L)
        if not q.sum() or lse[r] == -np.inf:
            continue
        at = np.array([idx[r, k] for k in keep])
        logp = (x[r][at] - lse[r]) / tau
        some = q > 0
        with np.errstate(invalid="ignore"):
            terms = q[some] * (tk[some] - L - logp[some])
        loss[r] = tau * tau * terms.sum()
        tbig = np.abs(tk[np.isfinite(tk)]).max() + abs(L)
        # each term's factors carry a few roundings of their parts' sizes, and so does q
        parts = np.abs(tk[some]) + abs(L) + big / tau
        bloss[r] = 8 * U * tau * tau * (q[some] * (parts + 16) * (1 + tbig) * (1 + np.abs(terms / q[some]))).sum()
        s = 1.0 if scale is None else float(scale[r])
        p = np.exp((x[r] - lse[r]) / tau)
        S = q.sum()
        grad[r] = S * p
        rel = U * (16 + 4 * np.minimum(np.abs(y - lse[r] / tau), 200.0) + 4 * blse[r] / (tau * U) + 4 * tbig + np.log2(len(keep) + 1))
        bgrad[r] = S * p * rel
        for k, j in enumerate(at):
            grad[r, j] -= q[k]
            bgrad[r, j] += q[k] * U * (16 + 8 * tbig + len(keep))
        grad[r] *= s * tau
        bgrad[r] *= abs(s) * tau
    return dict(loss=loss, lse=lse, grad=grad, bloss=bloss, blse=blse, bgrad=bgrad)


def units(r):
    """A mass in whole units of 2^-40."""
    r = np.asarray(r, np.float32)
    with np.errstate(invalid="ignore"):
        r = np.where(r > 0, np.minimum(r, np.float32(1)), np.float32(0))
    return (r.astype(np.float64) * 2.0 ** 40).astype(np.int64)     # exact, then cut


def verify(p, q, tokens, u, us, lens=None):
    """accepted [B], tokens [B, D + 1], accept_p [B, D]; p, q, u, us as binary32 values."""
    b, d1, v = p.shape
    d = d1 - 1
    acc, out, share = np.zeros(b, int), np.full((b, d1), -1), np.zeros((b, d), np.float32)
    for r in range(b):
        m = d if lens is None else int(np.clip(lens[r], 0, d))

        def pq(i):
            tok = int(tokens[r, i])
            if not 0 <= tok < v:
                return np.float32(0), np.float32(0), False
            return p[r, i, tok], (np.float32(1) if q is None else q[r, i, tok]), True

        n = 0
        while n < m:
            pt, qt, _ = pq(n)
            if not np.float32(u[r, n]) * qt < pt:
                break
            n += 1
        for i in range(m):
            pt, qt, inside = pq(i)
            share[r, i] = 0 if not inside else np.float32(pt) / np.float32(qt) if pt < qt else 1
        row = p[r, n].astype(np.float32).copy()
        if n < m and q is not None:
            with np.errstate(invalid="ignore"):
                row = row - q[r, n].astype(np.float32)
        elif n < m and 0 <= int(tokens[r, n]) < v:
            row[int(tokens[r, n])] = 0
        c = np.cumsum(units(row))
        if c[-1] == 0:
            c = np.cumsum(units(p[r, n]))
        x = np.float32(us[r])
        U31 = min(int(np.float64(x) * 2 ** 31), 2 ** 31 - 1) if x > 0 else 0
        mark = U31 * int(c[-1]) >> 31
        acc[r] = n
        out[r, :n] = tokens[r, :n]
        out[r, n] = int(np.searchsorted(c, mark, side="right")) if c[-1] else -1
    return dict(accepted=acc, tokens=out, accept_p=share)


def _weights(a, x, resets, sigmoid):
    a, x = np.asarray(a, np.float64), np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            e = np.exp(-np.abs(a))
            w = np.where(a >= 0, 1 / (1 + e), e / (1 + e))
            cw = np.where(a >= 0, e / (1 + e), 1 / (1 + e))
        else:
            w, cw = a, np.ones_like(a)
        v = np.where(cw == 0, 0, cw * x) if sigmoid else x
    wr = w if resets is None else np.where(np.asarray(resets)[..., None] != 0, 0, w)
    return wr, w, cw, v


def _weigh(w, h):
    with np.errstate(invalid="ignore"):
        return np.where(w == 0, 0, w * h)


def scan(a, x, h0=None, resets=None, sigmoid=False, reverse=False):
    """h, last and their bounds."""
    if reverse:
        f = lambda z: None if z is None else np.asarray(z)[:, ::-1]
        got = scan(f(a), f(x), h0, f(resets), sigmoid)
        return dict(got, h=got["h"][:, ::-1], bh=got["bh"][:, ::-1])
    w, _, _, v = _weights(a, x, resets, sigmoid)
    b, t, c = w.shape
    h = np.zeros((b, c)) if h0 is None else np.asarray(h0, np.float64)
    e = np.zeros((b, c))
    hs, es = np.zeros((b, t, c)), np.zeros((b, t, c))
    for i in range(t):
        with np.errstate(invalid="ignore"):
            # a step rounds each product and sum, and the gates carry a few roundings each
            e = _weigh(np.abs(w[:, i]), e) + 16 * U * (np.abs(_weigh(w[:, i], h)) + np.abs(v[:, i]))
            h = _weigh(w[:, i], h) + v[:, i]
        hs[:, i], es[:, i] = h, e
    return dict(h=hs, last=h, bh=es, blast=e)


def scan_backward(a, x, h, gh, h0=None, resets=None, glast=None, sigmoid=False, reverse=False):
    """grad_a, grad_x, grad_h0 and their bounds, from the given (stored) h."""
    if reverse:
        f = lambda z: None if z is None else np.asarray(z)[:, ::-1]
        got = scan_backward(f(a), f(x), f(h), f(gh), h0, f(resets), glast, sigmoid)
        return {k: (z if "h0" in k else z[:, ::-1]) for k, z in got.items()}
    if x is None:
        x = np.zeros_like(np.asarray(a, np.float64))
    wr, w, cw, _ = _weights(a, x, resets, sigmoid)
    x = np.asarray(x, np.float64)
    b, t, c = wr.shape
    h, gh = np.asarray(h, np.float64), np.asarray(gh, np.float64)
    start = np.zeros((b, c)) if h0 is None else np.asarray(h0, np.float64)
    carry = np.zeros((b, c)) if glast is None else np.asarray(glast, np.float64)
    e = np.zeros((b, c))
    out = {k: np.zeros((b, t, c)) for k in ("grad_a", "grad_x", "bgrad_a", "bgrad_x")}
    for i in range(t - 1, -1, -1):
        g = gh[:, i] + carry
        eg = e + 16 * U * (np.abs(gh[:, i]) + np.abs(carry))
        before = h[:, i - 1] if i else start
        if resets is not None:
            before = np.where(np.asarray(resets)[:, i, None] != 0, 0, before)
        if sigmoid:
            ww = w[:, i] * cw[:, i]
            with np.errstate(invalid="ignore"):
                out["grad_a"][:, i] = np.where(ww == 0, 0, g * (before - x[:, i]) * ww)
                out["bgrad_a"][:, i] = np.where(ww == 0, 0, (eg + 32 * U * np.abs(g)) * (np.abs(before) + np.abs(x[:, i])) * ww)
            out["grad_x"][:, i] = _weigh(cw[:, i], g)
            out["bgrad_x"][:, i] = _weigh(cw[:, i], eg + 16 * U * np.abs(g))
        else:
            zero = False if resets is None else np.asarray(resets)[:, i, None] != 0
            with np.errstate(invalid="ignore"):
                out["grad_a"][:, i] = np.where(zero, 0, g * before)
                out["bgrad_a"][:, i] = np.where(zero, 0, (eg + 16 * U * np.abs(g)) * np.abs(before))
            out["grad_x"][:, i], out["bgrad_x"][:, i] = g, eg
        carry = _weigh(wr[:, i], g)
        e = _weigh(np.abs(wr[:, i]), eg) + 16 * U * np.abs(carry)
    return dict(out, grad_h0=carry, bgrad_h0=e)


def close(got, want, bound, kind="f32"):
    """Every element within its bound plus the rounding to its type; non-finite ones alike."""
    got, want, bound = (np.asarray(z, np.float64) for z in (got, want, bound))
    fine = np.isfinite(want)
    same = np.where(np.isnan(want), np.isnan(got), got == want)
    assert same[~fine].all(), "non-finite values differ"
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
        lim = bound * 1.01 + HALF[kind] * 1.01 * (np.abs(want) + bound) + TINY[kind]
    bad = fine & ~(off <= lim)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside their bound; worst {np.max(off[bad] / lim[bad]):.3g} "
                           f"times, at {np.argwhere(bad)[:4].tolist()}: {got[bad][:4]} for {want[bad][:4]}")
