"""Shared pages without a GPU: pins of the oracle, and the refusals of the C calls, which come
before any HIP call."""
import ctypes

import numpy as np
import pytest

import lossless_bit_weight_w12_amd as w12
from lossless_bit_weight_w12_amd import w12 as B
from oracle import fork_oracle as fo

FAKE = 0x10000          # non-null, aligned, never dereferenced (validation fails first)
NULL, SHAPE, RANGE, FORMAT, WS, ALIGN = -1, -2, -3, -4, -5, -7


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(w12.lib_path()):
        from lossless_bit_weight_w12_amd import build
        build.build(verbose=False)
    return w12.lib()


# ------------------------------------------------------------------------------ the oracle
def pool(n_pages, max_req, max_pages, head=0):
    return [np.full((max_req, max_pages), -1, np.int32), np.zeros(max_req, np.int32),
            ((np.arange(n_pages) - head) % n_pages).astype(np.int32), np.array([head, n_pages, 0, 0], np.int32),
            np.zeros(n_pages, np.int32)]


def counted(p):
    """Counts are those of the tables, and every page is free or held."""
    table, held, ring, state, refs = p
    want = np.zeros_like(refs)
    for r, h in enumerate(held):
        for x in table[r, :h]:
            want[x] += 1
    free = [int(ring[(state[0] + i) % len(ring)]) for i in range(state[1])]
    return (want == refs).all() and sorted(free + np.flatnonzero(want).tolist()) == list(range(len(ring)))


def test_fork_worked_example():
    """A prompt of 20 tokens (pages 0, 1) in row 3; requests 0 .. 2 continue it with a row each:
    page 0 is shared, page 1 copied for all three (row 3 still holds it)."""
    p = pool(10, 4, 4)
    table, held, ring, state, refs = p
    kv_len, pos, slot, copies = fo.kv_fork(16, *p, [0, 1, 2, -1], [0, 0, 0, 0], [0, 0, 0, 0, 20], 20)
    assert kv_len.tolist() == [0, 0, 0, 20] and table[3, :2].tolist() == [0, 1] and state.tolist() == [2, 8, 0, 0]
    kv_len, pos, slot, copies = fo.kv_fork(16, *p, [3, 3, 3], [20, 20, 20], [0, 1, 2, 3], 3)
    assert table[:, :2].tolist() == [[0, 2], [0, 3], [0, 4], [0, 1]] and held.tolist() == [2, 2, 2, 2]
    assert copies.tolist() == [[1, 2, 4, 0], [1, 3, 4, 0], [1, 4, 4, 0]]
    assert slot.tolist() == [2 * 16 + 4, 3 * 16 + 4, 4 * 16 + 4] and refs[:5].tolist() == [4, 1, 1, 1, 1]
    # beam 1 goes on three times: request 0 keeps its page (nobody else holds it), 2 and 4 are given back
    kv_len, pos, slot, copies = fo.kv_fork(16, *p, [1, 1, 1], [21, 21, 21], [0, 1, 2, 3], 3)
    assert copies.tolist() == [[3, 3, 0, 0], [3, 5, 5, 0], [3, 6, 5, 0]]
    assert table[:, :2].tolist() == [[0, 3], [0, 5], [0, 6], [0, 1]] and slot.tolist() == [3 * 16 + 5, 5 * 16 + 5, 6 * 16 + 5]
    assert [int(ring[(state[0] + i) % 10]) for i in range(state[1])] == [7, 8, 9, 2, 4] and counted(p)
    # without rows nothing is written: the last page is shared too; row 3 is released
    fo.kv_fork(16, *p, [2, 2, 2, -1], [20, 18, 16, 0], [0, 0, 0, 0, 0], 0)
    assert table[:3, :2].tolist() == [[0, 6], [0, 6], [0, 6]] and held.tolist() == [2, 2, 1, 0]
    assert refs[[0, 6]].tolist() == [3, 2] and counted(p)


def test_fork_is_whole_or_nothing():
    p = pool(3, 3, 4)
    before = [x.copy() for x in p]
    out = fo.kv_fork(16, *p, None, [0, 0, 0], [0, 20, 40, 41], 41)
    assert (out[0] == -1).all() and all((a == b).all() for a, b in zip(p, before))
    out = fo.kv_fork(16, *p, None, [0, 0, 0], [0, 20, 20, 36], 36)
    assert out[0].tolist() == [20, 0, 16] and counted(p)


def test_fork_conserves_pages():
    g = np.random.default_rng(5)
    p, tokens = pool(80, 9, 12, head=7), np.zeros(9, int)
    done = 0
    for _ in range(150):
        n = int(g.integers(1, 10))
        parent = g.integers(-1, 9, n)
        length = [0 if q < 0 else int(g.integers(0, tokens[q] + 1)) for q in parent]
        rows = g.integers(0, 30, n)
        out = fo.kv_fork(16, *p, parent, length, np.concatenate([[0], np.cumsum(rows)]), int(rows.sum()))
        assert counted(p)
        if (out[0] >= 0).any():
            tokens[:n] = np.where(out[0] >= 0, out[0], tokens[:n])
            done += 1
    assert done > 40


def test_compact_worked_example():
    table = np.array([[0, 5, 7], [0, 4, -1]], np.int32)
    held = np.array([3, 2], np.int32)
    ring, state = np.array([1, 2, 3, 6, 9, 9, 9, 9], np.int32), np.array([0, 4, 0, 0], np.int32)
    refs = np.array([2, 0, 0, 0, 1, 1, 0, 1], np.int32)
    moves, moved = fo.kv_compact(16, table, held, ring, state, refs, 5, 3)
    assert moved == 2 and moves.tolist() == [[5, 1, 16, 0], [-1, -1, 0, 0], [7, 2, 16, 0]]
    assert table.tolist() == [[0, 1, 2], [0, 4, -1]] and refs.tolist() == [2, 1, 1, 0, 1, 0, 0, 0]
    assert state.tolist() == [0, 4, 0, 0] and ring[:4].tolist() == [3, 5, 6, 7]
    assert fo.kv_compact(16, table, held, ring, state, refs, 0, 7)[1] == -1


def test_copy_worked_example():
    k, v = np.arange(3 * 32.).reshape(3, 1, 32, 1), np.arange(3 * 32.).reshape(3, 1, 1, 32)
    fo.kv_copy(k, v, [[0, 2, 3, 0], [1, 1, 5, 0], [0, 3, 4, 0]])
    assert k[2, 0, :, 0].tolist() == list(range(16)) + list(range(80, 96)) and v[2, 0, 0].tolist() == k[2, 0, :, 0].tolist()


# ------------------------------------------------------------------------------- C refusals
def pages(**kw):
    p = B.W12Pages()
    p.n_pages, p.page_size, p.max_req, p.max_pages = 100, 16, 8, 20
    p.table = p.held = p.ring = p.state = FAKE
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


def kv(**kw):
    d = B.W12Kv()
    d.n_pages, d.page_size, d.n_kv_heads, d.head_dim, d.dtype = 100, 16, 8, 128, 0
    d.k_scale = d.v_scale = 1.0
    d.k = d.v = FAKE
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("change,status", [
    (dict(p=None), NULL), (dict(refs=None), NULL), (dict(len=None), NULL), (dict(off=None), NULL),
    (dict(kv_len=None), NULL), (dict(copies=None), NULL), (dict(pos=None), NULL), (dict(slot=None), NULL),
    (dict(p=pages(table=None)), NULL), (dict(p=pages(page_size=24)), SHAPE), (dict(p=pages(n_pages=0)), SHAPE),
    (dict(p=pages(max_pages=0)), SHAPE), (dict(p=pages(max_req=4097)), SHAPE),
    (dict(p=pages(max_pages=(1 << 26) + 1)), SHAPE), (dict(n=0), RANGE), (dict(n=9), RANGE),
    (dict(m=(1 << 20) + 1), RANGE), (dict(copies=FAKE + 8), ALIGN), (dict(parent=FAKE + 2), ALIGN),
    (dict(refs=FAKE + 1), ALIGN)])
def test_fork_refuses(L, change, status):
    a = dict(p=pages(), refs=FAKE, parent=FAKE, len=FAKE, off=FAKE, n=4, m=5, kv_len=FAKE, pos=FAKE, slot=FAKE,
             copies=FAKE)
    a.update(change)
    assert L.w12_kv_fork(*a.values(), None) == status


@pytest.mark.parametrize("layers,n,copies,n_copies,status", [
    (None, 1, FAKE, 1, NULL), ([kv()], 1, None, 1, NULL), ([kv(k=None)], 1, FAKE, 1, NULL), ([kv()], 0, FAKE, 1, RANGE),
    ([kv()] * 1025, 1025, FAKE, 1, RANGE), ([kv()], 1, FAKE, (1 << 22) + 1, RANGE), ([kv()], 1, FAKE + 4, 1, ALIGN),
    ([kv(), kv(v=FAKE + 8)], 2, FAKE, 1, ALIGN), ([kv(), kv(head_dim=64)], 2, FAKE, 1, SHAPE),
    ([kv(), kv(n_pages=99)], 2, FAKE, 1, SHAPE), ([kv(), kv(dtype=1)], 2, FAKE, 1, SHAPE),
    ([kv(n_kv_heads=0)], 1, FAKE, 1, SHAPE), ([kv(dtype=2)], 1, FAKE, 1, FORMAT), ([kv()], 1, None, 0, 0)])
def test_copy_refuses(L, layers, n, copies, n_copies, status):
    d = (B.W12Kv * len(layers))(*layers) if layers else None
    assert L.w12_kv_copy(d, n, copies, n_copies, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(p=None), NULL), (dict(refs=None), NULL), (dict(moves=None), NULL), (dict(moved=None), NULL),
    (dict(p=pages(page_size=8)), SHAPE), (dict(n=0), RANGE), (dict(n=101), RANGE), (dict(first=91), RANGE),
    (dict(first=0xfffffff8, n=16), RANGE), (dict(moves=FAKE + 8), ALIGN), (dict(moved=FAKE + 2), ALIGN)])
def test_compact_refuses(L, change, status):
    a = dict(p=pages(), refs=FAKE, first=90, n=10, moves=FAKE, moved=FAKE)
    a.update(change)
    assert L.w12_kv_compact(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(kv=None), NULL), (dict(table=None), NULL), (dict(kv_len=None), NULL), (dict(off=None), NULL),
    (dict(grp_off=None), NULL), (dict(grp_len=None), NULL), (dict(ws=None), NULL), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(kv=kv(k=None)), NULL), (dict(kv=kv(head_dim=96)), SHAPE),
    (dict(heads=41), SHAPE), (dict(q_stride=5112), SHAPE), (dict(out_stride=5121), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(n_req=0), RANGE), (dict(n_req=4097), RANGE), (dict(n_grp=0), RANGE), (dict(n_grp=4097), RANGE),
    (dict(m=3277), RANGE), (dict(max_pages=1 << 25), RANGE), (dict(scale=float("inf")), FORMAT), (dict(scale=float("nan")), FORMAT),
    (dict(kv=kv(dtype=1, k_scale=0.0)), FORMAT), (dict(ws_bytes=-1), WS), (dict(q=FAKE + 8), ALIGN),
    (dict(ws=FAKE + 16), ALIGN), (dict(grp_off=FAKE + 2), ALIGN), (dict(m=0, q=None, out=None), 0)])
def test_attn_shared_refuses(L, change, status):
    a = dict(q=FAKE, q_stride=5120, m=24, heads=40, kv=kv(), table=FAKE, max_pages=600, kv_len=FAKE, off=FAKE, n_req=24,
             grp_off=FAKE, grp_len=FAKE, n_grp=6, scale=0.1, out=FAKE, out_stride=5120, ws=FAKE, ws_bytes=0)
    a["ws_bytes"] = L.w12_attn_shared_ws_bytes(24, 40, 128) + change.pop("ws_bytes", 0)
    a.update(change)
    a["kv"] = ctypes.byref(a["kv"]) if a["kv"] is not None else None
    assert L.w12_attn_shared(*a.values(), None) == status


def test_attn_shared_workspace_bytes(L):
    """None for calls that are none; more for more rows and wider heads."""
    f = L.w12_attn_shared_ws_bytes
    assert f(1, 0, 128) == f(1, 1025, 128) == f(1, 40, 96) == f(3277, 40, 128) == 0
    assert 0 < f(1, 1, 64) < f(2, 1, 64) < f(2, 1, 128) and f(1 << 17, 1, 256) > 0


# ---------------------------------------------------------------------------------- the beams
def test_beam_oracle_worked_example():
    """Two rows of three tokens: probabilities 1/2, 1/4, 1/4 and 1/8, 3/4, 1/8; prior scores log 1/2 and
    log 1/3: the pairs' probabilities are 1/4, 1/8, 1/8 and 1/24, 1/4, 1/24."""
    x = np.log(np.array([[2.0, 1, 1], [1, 6, 1]]))
    parent, token, score, _ = fo.beam_select(x, np.log([1 / 2, 1 / 3]), [0, 2, 2], 5)
    assert parent[0].tolist() in ([0, 1, 0, 0, 1], [1, 0, 0, 0, 1]) and sorted(token[0, :2].tolist()) == [0, 1]
    assert token[0, 2:].tolist() == [1, 2, 0] and np.allclose(np.exp(score[0]), [1 / 4, 1 / 4, 1 / 8, 1 / 8, 1 / 24])
    assert (parent[1] == -1).all() and (token[1] == -1).all() and (score[1] == -np.inf).all()


def test_beam_oracle_ties_and_what_is_no_number():
    x = np.zeros((3, 4))
    parent, token, _, close = fo.beam_select(x, np.zeros(3), [0, 3], 6)
    assert parent[0].tolist() == [0, 0, 0, 0, 1, 1] and token[0].tolist() == [0, 1, 2, 3, 0, 1] and close == np.inf
    x[0, 2], x[1, 1] = np.nan, -np.inf
    parent, token, score, _ = fo.beam_select(x, [9.0, 0.0, -1.0], [0, 3], 11)
    assert parent[0].tolist() == [1, 1, 1, 2, 2, 2, 2, 0, 0, 0, 0] and token[0].tolist() == [0, 2, 3, 0, 1, 2, 3, 0, 1, 3, 2]
    assert np.isinf(score[0, 7:]).all()


def test_beam_oracle_against_torch():
    import torch
    g = np.random.default_rng(3)
    x, s = g.standard_normal((7, 301)) * 3, g.standard_normal(7)
    parent, token, score, close = fo.beam_select(x, s, [0, 3, 7], 9)
    p = torch.log_softmax(torch.from_numpy(x), -1) + torch.from_numpy(s)[:, None]
    for i, (a, b) in enumerate([(0, 3), (3, 7)]):
        v, at = torch.topk(p[a:b].reshape(-1), 9)
        assert np.allclose(score[i], v.numpy(), atol=1e-12)
        assert (parent[i] == a + at.numpy() // 301).all() and (token[i] == at.numpy() % 301).all()
    assert 0 < close < 1


@pytest.mark.parametrize("change,status", [
    (dict(grp_off=None), NULL), (dict(parent=None), NULL), (dict(token=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), NULL), (dict(logits=None), NULL), (dict(scores=None), NULL), (dict(vocab=0), SHAPE),
    (dict(vocab=(1 << 21) + 1, stride=1 << 22), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(vocab=3), SHAPE),
    (dict(stride=999), SHAPE), (dict(stride=1 << 40), SHAPE), (dict(n=4097), RANGE), (dict(n_grp=0), RANGE),
    (dict(n_grp=4097), RANGE), (dict(dtype=2), FORMAT), (dict(ws_bytes=-1), WS), (dict(logits=FAKE + 2), ALIGN),
    (dict(ws=FAKE + 8), ALIGN), (dict(scores=FAKE + 1), ALIGN)])
def test_beam_select_refuses(L, change, status):
    a = dict(logits=FAKE, dtype=1, stride=1000, n=8, vocab=1000, scores=FAKE, grp_off=FAKE, n_grp=2, k=4, parent=FAKE,
             token=FAKE, out=FAKE, ws=FAKE, ws_bytes=0)
    a["ws_bytes"] = L.w12_beam_ws_bytes(8, 1000, 4) + change.pop("ws_bytes", 0)
    a.update(change)
    assert L.w12_beam_select(*a.values(), None) == status


def test_beam_workspace_bytes(L):
    f = L.w12_beam_ws_bytes
    assert f(4097, 10, 1) == f(1, 0, 1) == f(1, (1 << 21) + 1, 1) == f(1, 10, 0) == f(1, 100, 65) == 0
    assert 16384 < f(1, 10, 1) < f(2, 10, 1) <= f(2, 10, 2) < f(2, 100000, 2) and f(4096, 1 << 21, 64) > 0
