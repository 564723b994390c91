"""Plain CPU oracle of the attention side of a decode step (numpy, 64 bits): block tables,
norm and rotation with the cache append, attention over the paged cache.  Definitions only,
written from the formulas in include/w12.h; shares no code with the library.

Caches are passed as float64 arrays of the values they stand for, in the library's layout:
k [n_pages, n_kv_heads, page_size, head_dim], v [n_pages, n_kv_heads, head_dim, page_size].
"""
from __future__ import annotations

import numpy as np


def offsets_ok(off, m: int) -> bool:
    off = [int(o) for o in off]
    return off[0] >= 0 and off[-1] <= m and all(a <= b for a, b in zip(off, off[1:]))


def kv_plan(page: int, table, held, ring, state, length, off, m: int):
    """One w12_kv_plan, request by request.  Returns (kv_len, pos, slot) and updates table,
    held, ring and state (numpy int32 arrays) in place."""
    n, (_, max_pages), n_pages = len(length), table.shape, len(ring)
    kv_len = np.full(n, -1, np.int32)
    pos = np.full(m, -1, np.int32)
    slot = np.full(m, -1, np.int32)
    head, count = int(state[0]), int(state[1])
    if not (0 <= head < n_pages and 0 <= count <= n_pages) or not offsets_ok(off, m):
        return kv_len, pos, slot
    rows = [int(off[r + 1]) - int(off[r]) for r in range(n)]
    valid = [int(length[r]) >= 0 and 0 <= int(held[r]) <= max_pages
             and int(length[r]) + rows[r] <= max_pages * page for r in range(n)]
    want = [-(-(int(length[r]) + rows[r]) // page) if valid[r] else int(held[r]) for r in range(n)]
    back = [int(table[r, i]) for r in range(n) if valid[r] for i in range(want[r], int(held[r]))]
    if count + len(back) > n_pages:
        return kv_len, pos, slot
    for i, p in enumerate(back):
        ring[(head + count + i) % n_pages] = p
    count += len(back)
    stopped = False
    for r in range(n):
        if not valid[r]:
            continue
        need = max(0, want[r] - int(held[r]))
        if need and (stopped or need > count):
            stopped = True
            continue
        for i in range(need):
            table[r, held[r] + i] = ring[head]
            head, count = (head + 1) % n_pages, count - 1
        held[r] = want[r]
        kv_len[r] = int(length[r]) + rows[r]
        for i in range(rows[r]):
            p = int(length[r]) + i
            pos[off[r] + i] = p
            g = int(table[r, p // page])
            slot[off[r] + i] = g * page + p % page if 0 <= g < n_pages else -1
    state[0], state[1] = head, count
    return kv_len, pos, slot


def rotated_heads(x, weight, eps: float, freq, pos, interleaved: bool):
    """x [m, h, d] float64 -> (normed and turned heads, |a| + |b| of each value's pair)."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    rot = 2 * len(freq)
    mag = np.abs(x)
    if rot:
        ang = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)[None, :]
        c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
        ia = np.arange(rot // 2) * (2 if interleaved else 1)
        ib = ia + (1 if interleaved else rot // 2)
        a, b = x[..., ia].copy(), x[..., ib].copy()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return x, mag


def attention(q, k, v, table, kv_len, off, scale: float):
    """q [m, hq, d]; returns (out, tol) float64 [m, hq, d]; rows of no request stay NaN in
    both.  tol is the error allowance of an FP32 evaluation with BF16 weights and a BF16
    result (see attention_tolerance)."""
    m, hq, d = q.shape
    n_pages, hkv, page, _ = k.shape
    out = np.full((m, hq, d), np.nan)
    tol = np.full((m, hq, d), np.nan)
    for r in range(len(kv_len)):
        a, b, length = int(off[r]), int(off[r + 1]), int(kv_len[r])
        if a == b:
            continue
        if not 0 <= length <= table.shape[1] * page:
            tol[a:b] = 0.0
            continue
        ids = np.asarray(table[r, :-(-length // page)], np.int64)
        good = (ids >= 0) & (ids < n_pages)
        at = np.where(good, ids, 0)
        ok = np.repeat(good, page)[:length]
        kk = k[at].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :length]
        vv = v[at].transpose(1, 0, 3, 2).reshape(hkv, -1, d)[:, :length]
        for i in range(b - a):
            end = length - (b - a) + i + 1
            if end <= 0:
                out[a + i] = tol[a + i] = 0.0
                continue
            if not ok[:end].all():
                tol[a + i] = 0.0
                continue
            for h in range(hq):
                kh, vh = kk[h // (hq // hkv), :end], vv[h // (hq // hkv), :end]
                with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                    s = kh @ q[a + i, h] * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[a + i, h] = w @ vh
                    mags = np.abs(kh) @ np.abs(q[a + i, h])
                    big = np.abs(scale) * mags[np.isfinite(mags)].max(initial=0.0)
                    tol[a + i, h] = attention_tolerance(out[a + i, h], w @ np.abs(vh), big, end, d)
    return out, tol


def attention_tolerance(o, wv, big: float, t: int, d: int):
    """Allowance per output value.  A score of d exact products summed in FP32 in any order is
    off by at most d 2^-23 of the sum of magnitudes (big, largest over the tokens), its scaling
    and exp2 by 2^-20 relative; numerator and denominator each see it.  Weights rounded to BF16
    are off by 2^-8 each, the FP32 sums over t tokens by t 2^-23, both relative to wv = sum of
    w |v|.  The result is rounded to BF16: 2^-8 of it."""
    delta = d * 2.0 ** -23 * big + 2.0 ** -20
    return 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * np.expm1(delta) + t * 2.0 ** -23) * wv * (1 + 2.0 ** -7) + 1e-37
