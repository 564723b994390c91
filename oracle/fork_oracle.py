"""Plain CPU oracle of several continuations of one prompt (numpy, 64 bits): block tables whose
pages requests share, the copies and moves of pages, the choice of the beams that go on.
Definitions only, written from include/w12.h; shares no code with the library."""
from __future__ import annotations

import numpy as np

from oracle.kv_oracle import offsets_ok


def kv_fork(page: int, table, held, ring, state, refs, parent, length, off, m: int):
    """One w12_kv_fork, request by request.  Returns (kv_len, pos, slot, copies) and updates table,
    held, ring, state and refs [n_pages] (numpy int32 arrays) in place."""
    n, (max_req, max_pages), n_pages = len(length), table.shape, len(ring)
    kv_len, pos, slot = np.full(n, -1, np.int32), np.full(m, -1, np.int32), np.full(m, -1, np.int32)
    copies = np.tile(np.array([-1, -1, 0, 0], np.int32), (n, 1))
    refused = kv_len.copy(), pos.copy(), slot.copy(), copies.copy()
    head, count = int(state[0]), int(state[1])
    if not (0 <= head < n_pages and 0 <= count <= n_pages and state[2] == 0) or not offsets_ok(off, m):
        return refused
    old, had = table.copy(), [int(h) if 0 <= h <= max_pages else 0 for h in held]
    parent = list(range(n)) if parent is None else [int(p) for p in parent]
    rows = [int(off[r + 1]) - int(off[r]) for r in range(n)]
    served, takes, writer = [], [], []
    for r in range(n):
        p, length_r = parent[r], int(length[r])
        ok = 0 <= held[r] <= max_pages and length_r >= 0 and length_r + rows[r] <= max_pages * page
        ok = ok and (p == -1 or (0 <= p < max_req and 0 <= held[p] <= max_pages))
        ok = ok and -(-length_r // page) <= (0 if p == -1 else int(held[p]))
        served.append(ok)
        takes.append([int(old[p, c]) for c in range(-(-length_r // page))] if ok
                     else [int(old[r, c]) for c in range(had[r])])
        writer.append(ok and length_r % page > 0 and rows[r] > 0)
    good = lambda x: 0 <= x < n_pages
    # holders after the call, those that will write into their last page not among them
    after = refs.astype(np.int64).copy()
    for r in range(n):
        for c in range(had[r]):
            if good(old[r, c]):
                after[old[r, c]] -= 1
        for x in takes[r][:-1] if writer[r] else takes[r]:
            if good(x):
                after[x] += 1
    lone = after.copy()
    new = [list(t) for t in takes]
    need, kept = [], set()
    for r in range(n):
        copy = False
        if writer[r]:
            x = takes[r][-1]
            copy = bool(good(x) and (lone[x] != 0 or x in kept))
            if not copy and good(x):
                kept.add(x)
                after[x] += 1
            copies[r] = [x, -1 if copy else x, length[r] % page if copy else 0, 0]
        want = -(-(int(length[r]) + rows[r]) // page) if served[r] else len(takes[r])
        need.append((copy, want - len(takes[r])))
    total = sum(c + k for c, k in need)
    back = []
    for c in range(max_pages):
        for r in range(n):
            if c < had[r] and good(old[r, c]) and after[old[r, c]] == 0 and int(old[r, c]) not in back:
                if not (c < len(takes[r]) and takes[r][c] == old[r, c]):
                    back.append(int(old[r, c]))
    if total > count or count + len(back) > n_pages:
        return refused
    for r in range(n):
        copy, more = need[r]
        got = [int(ring[(head + i) % n_pages]) for i in range(copy + more)]
        head, count = (head + copy + more) % n_pages, count - copy - more
        if copy:
            new[r][-1] = copies[r][1] = got[0]
        new[r] += got[copy:]
        for x in got:
            after[x] += 1
    for i, x in enumerate(back):
        ring[(head + count + i) % n_pages] = x
    state[0], state[1] = head, count + len(back)
    refs[:] = after
    for r in range(n):
        if served[r]:
            table[r, :len(new[r])] = new[r]
            held[r] = len(new[r])
            kv_len[r] = int(length[r]) + rows[r]
            for i in range(rows[r]):
                p = int(length[r]) + i
                pos[off[r] + i] = p
                if good(new[r][p // page]):
                    slot[off[r] + i] = new[r][p // page] * page + p % page
    return kv_len, pos, slot, copies


def kv_copy(k, v, copies):
    """k [..., n_pages, heads, page, dim] and v [..., n_pages, heads, dim, page] in place."""
    n_pages, page = k.shape[-4], k.shape[-2]
    for src, dst, tokens, _ in np.asarray(copies):
        if tokens < 1 or src == dst or not (0 <= src < n_pages and 0 <= dst < n_pages):
            continue
        t = min(page, -(-int(tokens) // 16) * 16)
        k[..., dst, :, :t, :] = k[..., src, :, :t, :]
        v[..., dst, :, :, :t] = v[..., src, :, :, :t]


def kv_compact(page: int, table, held, ring, state, refs, first: int, n_clear: int):
    """One w12_kv_compact.  Returns (moves, moved) and updates the arrays in place."""
    n_pages, max_pages = len(ring), table.shape[1]
    moves = np.tile(np.array([-1, -1, 0, 0], np.int32), (n_clear, 1))
    inside = lambda x: first <= x < first + n_clear
    live = [x for x in range(n_pages) if inside(x) and refs[x] > 0]
    free = [x for x in range(n_pages) if not inside(x) and refs[x] <= 0]
    if len(live) > len(free):
        return moves, -1
    to = dict(zip(live, free))
    for x, y in to.items():
        moves[x - first] = [x, y, page, 0]
        refs[y], refs[x] = refs[x], 0
    for r in range(table.shape[0]):
        if 0 <= held[r] <= max_pages:
            for c in range(int(held[r])):
                table[r, c] = to.get(int(table[r, c]), int(table[r, c]))
    left = free[len(live):] + list(range(first, first + n_clear))
    ring[:len(left)] = left
    state[0], state[1] = 0, len(left)
    return moves, len(live)


def beam_select(logits, scores, off, k: int, max_beams: int = 64):
    """logits [n, vocab] and scores [n] float64.  Returns (parent, token, score float64) [n_grp, k], and
    the smallest difference between scores of two rows that the choice or its order turned on
    (differences of rows with equal logits do not count: inf if there is none)."""
    n, n_grp = len(logits), len(off) - 1
    parent, token = np.full((n_grp, k), -1, np.int32), np.full((n_grp, k), -1, np.int32)
    if not offsets_ok(off, n) or any(int(b) - int(a) > max_beams for a, b in zip(off, off[1:])):
        return parent, token, np.full((n_grp, k), np.nan), np.inf
    score, close = np.full((n_grp, k), -np.inf), np.inf
    with np.errstate(all="ignore"):
        for g in range(n_grp):
            best = []
            for r in range(int(off[g]), int(off[g + 1])):
                x = np.asarray(logits[r], np.float64)
                top = x.max()
                lse = top + np.log(np.exp(x - top).sum())
                rank = np.where(np.isnan(x), -np.inf, x)
                order = np.argsort(-rank, kind="stable")[:k]
                s = scores[r] + (rank[order] - lse)
                best += [(-np.inf if np.isnan(v) else v, r, int(t)) for v, t in zip(s, order)]
            best.sort(key=lambda b: -b[0])     # stable: lower rows first, a row's in its own order
            for j, (v, r, t) in enumerate(best[:k]):
                parent[g, j], token[g, j], score[g, j] = r, t, v
            for (v, r, _), (w, q, _) in zip(best[:k], best[1:k + 1]):
                if r != q and np.isfinite(v) and np.isfinite(w) and not (
                        scores[r] == scores[q] and np.array_equal(logits[r], logits[q])):
                    close = min(close, v - w)
    return parent, token, score, close
