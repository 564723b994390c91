"""Shared pages on the GPU against the oracle: all whole numbers, so everything is equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from oracle import fork_oracle as fo  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
NAMES = ("kv_len", "pos", "slot", "copies", "table", "held", "ring", "state", "refs")


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int32)).to(DEV)


def cpu(t):
    return t.cpu().numpy()


class Pool:
    """Shared pages on the device and the oracle's copy of them."""

    def __init__(self, n_pages, page, max_req, max_pages, head=0):
        self.pt = w12.page_table(n_pages, page, max_req, max_pages, DEV, shared=True)
        self.pt.ring.copy_(torch.roll(self.pt.ring, head))
        self.pt.state[0] = head
        self.page = page
        self.ref = [cpu(t).copy() for t in self.arrays()]

    def arrays(self):
        return self.pt.table, self.pt.held, self.pt.ring, self.pt.state, self.pt.refs[:self.pt.n_pages]

    def fork(self, parent, length, off, m):
        got = w12.kv_fork(self.pt, None if parent is None else i32(parent), i32(length), i32(off), m)
        want = fo.kv_fork(self.page, *self.ref, parent, length, off, m)
        self.same(NAMES[:4], got, want)
        return want

    def same(self, names, got, want):
        for name, a, b in zip(names, got, want):
            assert np.array_equal(cpu(a), b), name
        for name, a, b in zip(NAMES[4:], self.arrays(), self.ref):
            assert np.array_equal(cpu(a), b), name
        assert not self.pt.refs[self.pt.n_pages:3 * self.pt.n_pages].any(), "words of a call under way"

    def compact(self, first, n_clear):
        moves, moved = w12.kv_compact(self.pt, first, n_clear)
        ring = cpu(self.pt.ring)
        want, n = fo.kv_compact(self.page, *self.ref, first, n_clear)
        left = self.ref[3][1]
        self.ref[2][left:] = ring[left:]
        self.same(("moves", "moved"), (moves, moved), (want, np.array([n])))
        return want, n


def offsets(rows, start=0):
    return np.concatenate([[start], start + np.cumsum(rows)]).astype(np.int64)


@pytest.mark.parametrize("max_req,page,max_pages,n_pages,most", [
    (1, 16, 4, 9, 30), (5, 16, 12, 60, 40), (24, 16, 70, 900, 60), (33, 64, 200, 900, 90), (130, 256, 5, 500, 300),
    (256, 16, 40, 4000, 50), (300, 16, 33, 4000, 40), (1030, 32, 9, 5000, 60)])
def test_fork_follows_random_parents(max_req, page, max_pages, n_pages, most):
    """Random parents, lengths and rows: forks, trims, releases, admissions and refusals in one."""
    g = np.random.default_rng(max_req + page)
    p = Pool(n_pages, page, max_req, max_pages, head=n_pages // 3)
    tokens, done = np.zeros(max_req, np.int64), 0
    for step in range(14):
        n = max_req if step % 3 else int(g.integers(1, max_req + 1))
        some = g.integers(0, max_req, max(1, max_req // 3))
        parent = np.where(g.random(n) < 0.5, np.arange(n), g.choice(some, n))
        parent[g.random(n) < 0.1] = -1
        length = np.where(parent < 0, 0, g.integers(0, tokens[parent] + 1))
        whole = g.random(n) < 0.6
        length = np.where(whole & (parent >= 0), tokens[parent], length)
        rows = g.integers(0, most, n) * (g.random(n) < 0.7)
        rows = np.minimum(rows, max_pages * page - length)
        start = int(g.integers(0, 3))
        off = offsets(rows, start)
        out = p.fork(parent, length, off, int(off[-1]) + int(g.integers(0, 3)))
        if (out[0] >= 0).any():
            tokens[:n] = np.where(out[0] >= 0, out[0], tokens[:n])
            done += 1
        else:   # too few pages: some go
            drop = np.where(np.arange(max_req) % 2 == 0, -1, np.arange(max_req))
            keep = np.where(drop < 0, 0, tokens)
            p.fork(drop, keep, np.zeros(max_req + 1, np.int64), 0)
            tokens = keep
    assert done > 3


@pytest.mark.parametrize("n_req,max_pages", [(4, 30), (64, 520), (4096, 3), (7, 40000)])
def test_fork_reorders_beams(n_req, max_pages):
    """Every request becomes another one, some several times, at once."""
    page, n_pages = 16, min(n_req * max_pages + 2 * n_req, 90000)
    g = np.random.default_rng(n_req)
    p = Pool(n_pages, page, n_req, max_pages, head=1)
    cap = min((max_pages - 1) * page, (n_pages // n_req - 2) * page, w12.MAX_KV_ROWS // n_req)
    rows = g.integers(1, cap, n_req)
    p.fork(None, np.zeros(n_req), offsets(rows), int(rows.sum()))
    tokens = rows
    for _ in range(3):
        parent = g.permutation(n_req)
        parent[::3] = parent[0]
        out = p.fork(parent, tokens[parent], np.arange(n_req + 1), n_req)
        assert (out[0] == tokens[parent] + 1).all()
        tokens = tokens[parent] + 1


@pytest.mark.parametrize("n_req,max_pages", [(256, 9000), (4096, 600)])
def test_fork_of_more_columns_than_fit_at_once(n_req, max_pages):
    """A few requests hold almost every column, so that a workgroup takes its columns in turns."""
    g = np.random.default_rng(n_req + 1)
    n_pages = 8 * max_pages + 4 * n_req
    p = Pool(n_pages, 16, n_req, max_pages, head=n_pages - 5)
    rows = g.integers(1, 20, n_req)
    long = g.permutation(n_req)[:3]
    rows[long] = 16 * max_pages - g.integers(20, 40, 3)
    p.fork(None, np.zeros(n_req), offsets(rows), int(rows.sum()))
    tokens = rows
    for i in range(3):
        parent = np.arange(n_req)
        some = g.permutation(n_req)[:n_req // 3]
        parent[some] = long[i]
        parent[long[(i + 1) % 3]] = some[0]
        length = np.minimum(tokens[parent], g.integers(1, 16 * max_pages, n_req)) if i == 1 else tokens[parent]
        out = p.fork(parent, length, np.arange(n_req + 1), n_req)
        assert (out[0] == length + 1).all()
        tokens = length + 1
        long = some[:3]


def test_fork_refuses_a_request():
    """Lengths, parents and counts that are none refuse their request alone."""
    p = Pool(60, 16, 8, 5)
    p.fork(None, [0] * 8, offsets([20] * 8), 160)
    out = p.fork([0, 9, 2, -2, -1, 5, 6, 1], [-1, 5, 33, 0, 1, 17, 60, 20], offsets([1, 1, 1, 1, 1, 1, 21, 1]), 28)
    assert out[0].tolist() == [-1, -1, -1, -1, -1, 18, -1, 21]
    p.pt.held[2] = p.ref[1][2] = -1
    p.pt.held[3] = p.ref[1][3] = 6
    out = p.fork([0, 1, 2, 3, 2, 3, 6, 7], [20] * 8, offsets([1] * 8), 8)
    assert out[0].tolist() == [21, 21, -1, -1, -1, -1, 21, 21]


@pytest.mark.parametrize("off,state", [([0, 2, 1, 3], None), ([-1, 0, 0, 0], None), ([0, 0, 0, 4], None),
                                       ([0, 1, 2, 3], [60, 5, 0, 0]), ([0, 1, 2, 3], [0, -1, 0, 0]),
                                       ([0, 1, 2, 3], [0, 61, 0, 0]), ([0, 1, 2, 3], [0, 40, 5, 0])])
def test_fork_refuses_what_is_no_pool(off, state):
    p = Pool(60, 16, 3, 5)
    p.fork(None, [0, 0, 0], [0, 20, 40, 60], 60)
    if state is not None:
        p.pt.state.copy_(i32(state))
        p.ref[3][:] = state
    out = p.fork([1, 1, 1], [20, 20, 20], off, 3)
    assert (out[0] == -1).all()


def test_fork_is_captured_and_replayed():
    """A step of beam search in a graph, replayed with other parents."""
    n, page = 8, 16
    g = np.random.default_rng(0)
    p = Pool(200, page, n, 12)
    rows = g.integers(20, 90, n)
    p.fork(None, np.zeros(n), offsets(rows), int(rows.sum()))
    parent, length, off = i32(np.arange(n)), i32(rows), i32(np.arange(n + 1))
    out = [torch.empty(s, dtype=torch.int32, device=DEV) for s in (n, n, n, (n, 4))]
    call = lambda: w12.kv_fork(p.pt, parent, length, off, n, *out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    tokens = rows
    for step in range(5):
        chosen = g.integers(0, n, n)
        parent.copy_(i32(chosen))
        length.copy_(i32(tokens[chosen]))
        graph.replay()
        want = fo.kv_fork(page, *p.ref, chosen, tokens[chosen], np.arange(n + 1), n)
        p.same(NAMES[:4], out, want)
        tokens = want[0].astype(np.int64)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page,heads,dim,layers", [(16, 8, 128, 3), (32, 1, 64, 1), (64, 3, 256, 2), (256, 2, 128, 1),
                                                   (16, 5, 64, 130), (256, 5, 256, 1)])
def test_copies_of_all_layers(page, heads, dim, layers, f8):
    g = np.random.default_rng(page + dim)
    n_pages = 11
    bits = lambda *s: torch.from_numpy(g.integers(0, 256 if f8 else 65536, s).astype(np.uint8 if f8 else np.uint16).view(np.uint8 if f8 else np.int16))
    k, v = bits(layers, n_pages, heads, page, dim), bits(layers, n_pages, heads, dim, page)
    copies = np.array([[0, 5, 1, 0], [0, 6, page, 7], [1, 7, page // 2 + 1, 0], [2, 2, 9, 0], [-1, -1, 0, 0], [3, 8, 0, 0],
                       [n_pages, 8, 3, 0], [3, n_pages, 3, 0], [-1, 9, 3, 0], [4, 10, page + 100, 0], [4, 9, -3, 0]], np.int32)
    dk, dv = k.to(DEV), v.to(DEV)
    t = F8 if f8 else torch.bfloat16
    w12.kv_copy([w12.KvCache(a.view(t), b.view(t)) for a, b in zip(dk, dv)], i32(copies))
    wk, wv = k.numpy().copy(), v.numpy().copy()
    fo.kv_copy(wk, wv, copies)
    assert np.array_equal(cpu(dk), wk) and np.array_equal(cpu(dv), wv)


def test_copies_beyond_32_bits():
    """Pages whose offset within a cache passes 2^32 bytes."""
    n_pages, heads, dim, page = 140000, 8, 128, 16
    k, v = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((n_pages, heads, page, dim), (n_pages, heads, dim, page)))
    ends = torch.arange(heads * page * dim, device=DEV).bfloat16()
    for i in (3, n_pages - 2):
        k[i], v[i] = (ends + i % 7).view(heads, page, dim), (ends - i % 5).view(heads, dim, page)
    w12.kv_copy([w12.KvCache(k, v)], i32([[n_pages - 2, 5, 16, 0], [3, n_pages - 1, 16, 0]]))
    assert torch.equal(k[5], k[n_pages - 2]) and torch.equal(v[5], v[n_pages - 2])
    assert torch.equal(k[n_pages - 1], k[3]) and torch.equal(v[n_pages - 1], v[3])


def test_copies_of_none():
    k = torch.ones((1, 3, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    v = torch.ones((1, 3, 2, 64, 16), dtype=torch.bfloat16, device=DEV)
    w12.kv_copy([w12.KvCache(k[0], v[0])], torch.empty((0, 4), dtype=torch.int32, device=DEV))
    assert (k == 1).all()


@pytest.mark.parametrize("n_pages,max_req,max_pages,page", [(9, 1, 4, 16), (300, 7, 20, 16), (5000, 260, 30, 64),
                                                           (70001, 33, 3000, 16)])
def test_compact_clears_a_range(n_pages, max_req, max_pages, page):
    g = np.random.default_rng(n_pages)
    p = Pool(n_pages, page, max_req, max_pages, head=n_pages // 2)
    most = max(1, min(max_pages, n_pages // (2 * max_req)) * page - page + 1)
    rows = g.integers(0, most, max_req)
    off = offsets(rows)
    assert (p.fork(None, np.zeros(max_req), off, int(off[-1]))[0] == rows).all()
    parent = np.arange(max_req)
    parent[max_req // 2:] = 0
    p.fork(parent, p_len(p, parent, rows), np.zeros(max_req + 1, np.int64), 0)
    for first, n in ((n_pages // 2, n_pages - n_pages // 2), (0, n_pages // 3), (n_pages // 4, 1), (0, n_pages),
                     (n_pages - 1, 1), (n_pages // 3, n_pages // 3)):
        before = [x.copy() for x in p.ref]
        moves, moved = p.compact(first, n)
        if moved < 0:
            assert all(np.array_equal(a, b) for a, b in zip(before, p.ref))
        # (and the pool goes on)
        p.fork(None, p_len(p, np.arange(max_req), rows), np.zeros(max_req + 1, np.int64), 0)


def held_tokens(p):
    return p.ref[1].astype(np.int64) * p.page


def p_len(p, parent, tokens):
    return np.minimum(tokens[parent], held_tokens(p)[parent])


def test_a_smaller_pool_after_the_range_is_cleared():
    p = Pool(100, 16, 4, 10)
    p.fork(None, [0] * 4, offsets([100, 50, 70, 3]), 223)
    moves, moved = p.compact(40, 60)
    small = w12.page_table(40, 16, 4, 10, DEV, shared=True)
    small.table.copy_(p.pt.table), small.held.copy_(p.pt.held), small.ring.copy_(p.pt.ring[:40])
    small.refs[:40] = p.pt.refs[:40]
    small.state.copy_(p.pt.state)
    small.state[1] -= 60
    kv_len, pos, slot, copies = w12.kv_fork(small, None, i32([100, 50, 70, 3]), i32([0, 30, 60, 90, 120]), 120)
    assert cpu(kv_len).tolist() == [130, 80, 100, 33] and cpu(slot).max() < 40 * 16
    free = [int(small.ring[(int(small.state[0]) + i) % 40]) for i in range(int(small.state[1]))]
    used = [int(x) for r in range(4) for x in small.table[r, :int(small.held[r])]]
    assert sorted(free + used) == list(range(40))
