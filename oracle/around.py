"""Plain 64-bit reference of the operators around the experts: the norm with the
residual's addition and the sum over a token's experts, 8-bit results, routing,
and the choice of the next token.  Loops and numpy only; nothing of the package.
"""
from __future__ import annotations

import numpy as np

# the magnitudes of e4m3 by code: 4 exponent bits with bias 7, 3 bits below; code 127 is no number
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def state(x, gates=None, residual=None):
    """residual + the sum of each token's rows: (h, the sum of the terms' magnitudes); a row of gate 0 takes no part."""
    x = np.asarray(x, np.float64)
    if gates is None:
        gates = np.ones((x.shape[0], 1))
    gates = np.asarray(gates, np.float64)
    T, k = gates.shape
    h = np.zeros((T, x.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(h)
    for t in range(T):
        for j in range(k):
            if gates[t, j] != 0:
                with np.errstate(invalid="ignore"):
                    h[t] += gates[t, j] * x[t * k + j]
                    size[t] += np.abs(gates[t, j] * x[t * k + j])
    return h, size


def rms_norm(h, weight=None, eps=1e-6):
    with np.errstate(invalid="ignore", over="ignore"):
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        return y if weight is None else y * np.asarray(weight, np.float64)


def to_e4m3(a):
    """The nearest e4m3 number, halves to the even code, 448 at most."""
    m = np.minimum(np.abs(a), 448.0)
    at = np.clip(np.searchsorted(E4M3, m), 1, 126)
    low, high = E4M3[at - 1], E4M3[at]
    up = (m - low > high - m) | ((m - low == high - m) & (at % 2 == 0))
    return np.copysign(np.where(up, high, low), a)


def fp8(y, block):
    """y [T, D] in e4m3 with a scale for each block (0: the row): (values [T, D], scales [T, blocks], bytes of scales or None)."""
    T, D = y.shape
    n = block or D
    out, scales, powers = np.empty_like(y), [], []
    for d in range(0, D, n):
        part = y[:, d:d + n]
        bad = ~np.isfinite(part).all(1)
        top = np.where(bad, 1.0, np.abs(part).max(1))
        if block == 32:
            s = np.full(T, 1)
            for p in range(1, 255):
                s = np.where(top > 448 * 2.0 ** (s - 127), np.minimum(p + 1, 254), s)
            unit = np.exp2(s - 127.0)
            powers.append(np.where(bad, 255, s))
        else:
            with np.errstate(under="ignore"):
                unit = np.maximum((top / 448).astype(np.float32), np.float32(2.0 ** -126)).astype(np.float64)
        with np.errstate(invalid="ignore"):
            out[:, d:d + n] = np.where(bad[:, None], np.nan, to_e4m3(part / unit[:, None]) * unit[:, None])
        scales.append(np.where(bad, np.nan, unit))
    return out, np.stack(scales, 1), np.stack(powers, 1) if powers else None


def route(logits, k, bias=None, sigmoid=False, n_groups=1, top_groups=1, group_best=2, renormalise=False, scale=1.0,
          requests=None):
    """(ids int [T, k], gates [T, k], how many rows were refused)"""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids, gates, refused = np.full((T, k), -1), np.zeros((T, k)), 0
    for t in range(T):
        if requests is not None and requests[t] < 0:
            continue
        l = logits[t]
        if np.isnan(l).any() or (l == np.inf).any():
            refused += 1
            continue
        there = l > -np.inf
        if not there.any():
            continue
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        c = l.copy() if bias is None else np.where(there, s + np.asarray(bias, np.float64), -np.inf)
        if np.isnan(c).any() or (c == np.inf).any():
            refused += 1
            continue
        there = c > -np.inf
        by = c if bias is not None else s
        if n_groups > 1:
            n = E // n_groups
            value = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                best = np.sort(by[g * n:(g + 1) * n][there[g * n:(g + 1) * n]])[::-1][:group_best]
                if best.size:
                    value[g] = best.sum()
            order = [g for g in np.argsort(-value, kind="stable") if value[g] > -np.inf][:top_groups]
            there &= np.isin(np.arange(E) // n, order)
        free = np.flatnonzero(there)
        pick = free[np.argsort(-c[free], kind="stable")][:k]
        g = s[pick]
        if renormalise and g.sum() > 0:
            g = g / g.sum()
        ids[t, :pick.size], gates[t, :pick.size] = pick, scale * g
    return ids, gates, refused


def kept(l, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (indices that stay, rising; their weights), or None for a row that has no distribution."""
    l = np.asarray(l, np.float64)
    if np.isnan(l).any() or (l == np.inf).any() or not (l > -np.inf).any() or not temperature >= 0 or np.isnan([top_p, min_p]).any():
        return None
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if temperature == 0:
        return order[:1], np.ones(1)
    if top_k > 0:
        order = order[:top_k]
    w = np.exp((l[order] - l.max()) / temperature)
    stays = w >= min(min_p, 1.0)
    order, w = order[stays], w[stays]
    if top_p < 1:
        upto = np.cumsum(w)
        n = 1 + int(np.searchsorted(upto, top_p * upto[-1]))
        order, w = order[:n], w[:n]
    by_index = np.argsort(order)
    return order[by_index], w[by_index]


def sample(l, u, **how):
    """One row: (token, ln of its probability), (-1, NaN) where there is no distribution."""
    got = kept(l, **how)
    if got is None or np.isnan(u):
        return -1, np.nan
    at, w = got
    upto = np.cumsum(w)
    i = int(np.searchsorted(upto, min(max(u, 0.0), 1.0) * upto[-1], side="right"))
    i = min(i, int(np.flatnonzero(w > 0)[-1]))
    return int(at[i]), float(np.log(w[i] / upto[-1]))
