"""Plain 64-bit reference of the operators around the experts: the step plan of
a paged cache, norms and rotation of queries and keys, the 4-bit cache's
format, and attention over it.  Loops and numpy only; nothing of the package.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MOST_SCALE = {"bf16": 252, "fp16": 140}
BITS = {"bf16": 8, "fp16": 11}
FINEST = {"bf16": -133, "fp16": -24}      # exponent of the smallest subnormal


def plan(ctx, new, free, table, block_size, max_tokens):
    """One step: (table, slots, positions, requests, cu_q, kv_lens, n_free); the
    free list is popped from its end."""
    table = np.array(table, np.int32)
    free = list(free)
    slots, positions, requests, cu = [], [], [], [0]
    for i, (c, n) in enumerate(zip(ctx, new)):
        for j in range(-(-c // block_size), -(-(c + n) // block_size)):
            table[i, j] = free.pop()
        for p in range(c, c + n):
            slots.append(int(table[i, p // block_size]) * block_size + p % block_size)
            positions.append(p)
            requests.append(i)
        cu.append(cu[-1] + n)
    pad = max_tokens - len(slots)
    i32 = lambda v: np.array(v, np.int32)
    return (table, i32(slots + [-1] * pad), i32(positions + [0] * pad), i32(requests + [-1] * pad), i32(cu),
            i32([c + n for c, n in zip(ctx, new)]), len(free))


def round_to(x, dtype: str):
    """float64 to the nearest bf16 / fp16 value (halves to even), as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.frexp(np.where(np.isfinite(x), x, 1.0))[1]
        q = np.ldexp(1.0, np.maximum(e - BITS[dtype], FINEST[dtype]))
        y = np.rint(x / q) * q
        top = 65504.0 if dtype == "fp16" else (2.0 - 2.0 ** -7) * 2.0 ** 127
        return np.where(np.isfinite(x), np.where(np.abs(y) > top, np.copysign(np.inf, x), y), x)


def norm_rope(x, w, rope, rot, eps=1e-6, neighbours=False):
    """x [T, H, D], w [D] or None, rope [T, rot] (cosines, sines): unrounded float64."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if not rot:
        return y
    half = rot // 2
    c, s = (np.asarray(rope, np.float64)[:, None, i * half:(i + 1) * half] for i in (0, 1))
    out = y.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, half), slice(half, rot))
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def quantise(x, dtype: str):
    """x [..., D] -> (codes uint8 [..., D], scales uint8 [..., D/32])."""
    b = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.frexp(np.where(top > 0, top, 1.0) / 7.0)      # top / 7 = m 2^e, m in [0.5, 1)
    s = e[1] - (e[0] == 0.5)                              # the smallest power of two that is >= top / 7
    # division by 7 rounds: settle the border exactly
    s = np.where(top > 7.0 * np.ldexp(1.0, s), s + 1, s)
    s = np.where(top <= 7.0 * np.ldexp(1.0, s - 1), s - 1, s)
    s = np.where(top > 0, s, -126)
    s = np.clip(s + 127, 1, MOST_SCALE[dtype])
    a = np.abs(b) / np.ldexp(1.0, s - 127)[..., None]
    off = np.abs(a[..., None] - E2M1)
    code = off.argmin(-1)                                 # the lower of two equally near
    tie = np.take_along_axis(off, np.minimum(code + 1, 7)[..., None], -1)[..., 0] == off.min(-1)
    code = np.where(tie & (code % 2 == 1) & (code < 7), code + 1, code)
    code = code + 8 * np.signbit(np.asarray(x, np.float64).reshape(b.shape))
    s = np.where(bad, 255, s)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(np.shape(x)).astype(np.uint8), s.astype(np.uint8)


def values(codes, scales):
    """What codes [..., D] and scales [..., D/32] stand for, float64."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(codes.shape)


def pages(codes_k, scales_k, codes_v, scales_v):
    """Rows [..., bs, D] of codes and [..., bs, D/32] of scales to records uint8 [..., bytes]."""
    flat = lambda a: a.reshape(*a.shape[:-2], -1)
    pack = lambda c: flat(c[..., 0::2] | (c[..., 1::2] << 4))
    return np.concatenate([pack(codes_k), pack(codes_v), flat(scales_k), flat(scales_v)], -1)


def split_pages(data, bs, dim):
    """Records to (codes_k, scales_k, codes_v, scales_v), each [..., bs, :]."""
    n, m = bs * dim // 2, bs * dim // 32
    rows = lambda a: a.reshape(*a.shape[:-1], bs, -1)
    two = lambda a: np.stack([a & 15, a >> 4], -1).reshape(*a.shape[:-1], -1)
    return (two(rows(data[..., :n])), rows(data[..., 2 * n:2 * n + m]), two(rows(data[..., n:2 * n])),
            rows(data[..., 2 * n + m:]))


def attention(q, data, bs, table, kv_lens, cu_q, scale):
    """q [T, H, D] float64, data uint8 [n_blocks, Hk, bytes].  Returns (out, lse,
    weight): weight[t, h, d] = sum softmax |v|, what errors of the weights scale
    with.  A block outside the cache hides its tokens; hidden tokens take no
    part, whatever they hold."""
    T, H, D = q.shape
    nb, Hk, _ = data.shape
    out, weight = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    cu = list(range(len(kv_lens) + 1)) if cu_q is None else list(cu_q)
    for r, n in enumerate(kv_lens):
        a, b = cu[r], cu[r + 1]
        n = min(n, table.shape[1] * bs)
        if n <= 0 or a == b:
            continue
        blocks = table[r, :-(-n // bs)]
        there = np.repeat((blocks >= 0) & (blocks < nb), bs)[:n]
        page = data[np.clip(blocks, 0, nb - 1)]
        kc, ks, vc, vs = split_pages(page, bs, D)
        for h in range(Hk):
            k = values(kc[:, h], ks[:, h]).reshape(-1, D)[:n]
            v = values(vc[:, h], vs[:, h]).reshape(-1, D)[:n]
            for t in range(a, b):
                sees = there & (np.arange(n) <= n - (b - a) + (t - a))
                if not sees.any():
                    continue
                for j in range(h * (H // Hk), (h + 1) * (H // Hk)):
                    with np.errstate(all="ignore"):
                        z = scale * (k[sees] @ q[t, j])
                        top = z.max()
                        p = np.exp(z - top)
                        lse[t, j] = top + np.log(p.sum())
                        out[t, j] = (p / p.sum()) @ v[sees]
                        weight[t, j] = (p / p.sum()) @ np.abs(v[sees])
    return out, lse, weight
