"""The attention side of a decode step on the GPU against its 64-bit oracle: block tables and
slot maps (exact), norm and rotation with the cache append, attention over the paged cache."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from oracle import kv_oracle as ko  # noqa: E402
from tests.gpu_util import say  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int32)).to(DEV)


def host(t):
    return t.double().cpu().numpy()


def normal(g, shape, dtype=torch.bfloat16, scale=1.0):
    x = torch.from_numpy(g.standard_normal(shape, dtype=np.float32) * np.float32(scale))
    return x.to(dtype).to(DEV)


# ---------------------------------------------------------------------------- block tables
class Pool:
    """A page table on the device and the oracle's copy of it."""

    def __init__(self, n_pages, page, max_req, max_pages, head=0):
        self.pt = w12.page_table(n_pages, page, max_req, max_pages, DEV)
        self.pt.state[0] = head
        self.page = page
        self.ref = [t.cpu().numpy().copy() for t in (self.pt.table, self.pt.held, self.pt.ring, self.pt.state)]

    def step(self, length, off, m):
        got = w12.kv_plan(self.pt, i32(length), i32(off), m)
        want = ko.kv_plan(self.page, *self.ref, length, off, m)
        self.same(got, want)
        return want

    def same(self, got, want):
        for name, a, b in zip(("kv_len", "pos", "slot", "table", "held", "ring", "state"),
                              list(got) + [self.pt.table, self.pt.held, self.pt.ring, self.pt.state],
                              list(want) + self.ref):
            assert np.array_equal(a.cpu().numpy(), b), name


def offsets(rows, start=0):
    return np.concatenate([[start], start + np.cumsum(rows)]).astype(np.int64)


@pytest.mark.parametrize("n,page,max_pages,n_pages,top", [
    (1, 16, 4, 5, 60), (3, 16, 9, 20, 140), (24, 16, 40, 700, 600), (24, 64, 12, 100, 700),
    (65, 128, 5, 200, 600), (257, 16, 20, 1500, 300), (1024, 32, 4, 3000, 128), (1025, 256, 3, 2500, 700),
    (4096, 16, 3, 9000, 45)])
def test_plan_follows_random_lengths(n, page, max_pages, n_pages, top):
    """Twelve steps: lengths grow, shrink and vanish, some do not fit the table, the pool runs
    dry; a batch may begin and end with rows of no request."""
    say("plan", n, page, max_pages, n_pages)
    g = np.random.default_rng([7, n, page])
    p = Pool(n_pages, page, n, max_pages, head=int(g.integers(0, n_pages)))
    for step in range(12):
        rows = g.integers(0, 6 if step % 3 else 40, n) * g.integers(0, 2, n)
        length = g.integers(0, top, n) * (g.random(n) < 0.8)
        if step == 11:
            rows[:], length[:] = 0, 0
        off = offsets(rows, step % 4)
        p.step(length, off, int(off[-1]) + step % 3)
    assert int(p.pt.state[1]) == n_pages


def test_plan_refuses_single_requests():
    """Negative length, a length past the table, counts out of range: the others are served."""
    p = Pool(40, 16, 6, 5)
    p.step([10, 20, 30, 40, 50, 60], offsets([1, 1, 1, 1, 1, 1]), 6)
    p.pt.held[4] = -2
    p.ref[1][4] = -2
    p.pt.held[5] = 6
    p.ref[1][5] = 6
    want = p.step([11, -1, 80, 79, 5, 5], offsets([1, 1, 1, 1, 1, 1]), 6)
    assert want[0].tolist() == [12, -1, -1, 80, -1, -1]
    p.step([2147483647, 0, 0, 0, 0, 0], offsets([3, 0, 0, 0, 0, 0]), 3)


@pytest.mark.parametrize("off,m", [([-1, 2, 3], 3), ([0, 2, 1], 3), ([0, 2, 4], 3), ([3, 2, 3], 3)])
def test_plan_refuses_offsets(off, m):
    p = Pool(10, 16, 2, 4)
    p.step([5, 6], [0, 1, 2], 2)
    want = p.step([6, 7], off, m)
    assert want[0].tolist() == [-1, -1] and (want[1] == -1).all()


@pytest.mark.parametrize("state", [(-1, 3), (10, 3), (0, 11), (0, -1), (3, 10)])
def test_plan_refuses_states(state):
    """Heads and counts no ring has, and a count that leaves no room for what comes back."""
    p = Pool(10, 16, 2, 4)
    p.step([30, 40], [0, 0, 0], 0)
    for i in (0, 1):
        p.pt.state[i] = state[i]
        p.ref[3][i] = state[i]
    want = p.step([0, 0], [0, 0, 1], 1)
    assert want[0].tolist() == [-1, -1]


def test_plan_pages_move_within_a_call():
    """The pool is empty: what request 1 gives back, request 0 takes in the same call."""
    p = Pool(6, 16, 2, 6, head=4)
    p.step([16, 80], [0, 0, 0], 0)
    want = p.step([64, 20], [0, 1, 2], 2)
    assert want[0].tolist() == [-1, 21] and p.ref[1].tolist() == [1, 2]   # 3 free, 4 wanted
    want = p.step([48, 20], [0, 16, 17], 17)
    assert want[0].tolist() == [64, 21]


def test_plan_needs_past_2_to_the_30_pages():
    """Requests of 2^26 pages each: from the 16th on the sums of their needs saturate, and a sum equals
    the one before it; all the same every request that needs pages is refused."""
    n = 19
    p = w12.page_table(64, 16, n, 1 << 26, DEV)
    p.held[3] = 4      # the one request that needs nothing, behind refused ones
    p.state[1] = 60
    length = np.full(n, (1 << 30) - 1)
    length[3] = 60
    kv_len, pos, slot = w12.kv_plan(p, i32(length), i32(np.arange(n + 1)), n)
    want = np.full(n, -1)
    want[3] = 61
    assert np.array_equal(kv_len.cpu().numpy(), want)
    want[3] = 60
    assert np.array_equal(pos.cpu().numpy(), want)
    assert (slot == -1).all()      # (its table names no page)
    assert p.held.tolist() == [0, 0, 0, 4] + [0] * 15 and p.state.tolist() == [0, 60, 0, 0]
    assert p.ring.tolist() == list(range(64))
    assert int(p.table.max()) == -1


def test_plan_large_tables():
    """64 prompts of up to 4000 tokens at once, then everything back; and a bad page id in the
    table gives no slot."""
    g = np.random.default_rng(5)
    rows = g.integers(1, 4000, 64)
    p = Pool(20000, 16, 64, 256, head=19990)
    p.step(np.zeros(64, int), offsets(rows), int(rows.sum()) + 5)
    p.step(rows, offsets([1] * 64), 64)
    p.pt.table[3, 0] = 20000
    p.ref[0][3, 0] = 20000
    p.step(np.ones(64, int), offsets([2] * 64), 128)
    p.step(np.zeros(64, int), offsets([0] * 64), 0)


# ------------------------------------------------------------------------ norm and rotation
def rope_case(g, m, hq, hkv, d, page, f8, norm, per=3, far=1 << 20):
    """Inputs with rows of several requests: consecutive slots inside each, in shuffled pages."""
    n = -(-m // per)
    each = (page + per - 2) // page + 1
    n_pages = n * each + 1
    perm = g.permutation(n_pages)
    start = g.integers(0, far, n)
    r, i = np.arange(m) // per, np.arange(m) % per
    logical = start % page
    slot = perm[r * each + (logical[r] + i) // page] * page + (logical[r] + i) % page
    c = w12.KvCache(normal(g, (n_pages, hkv, page, d), F8 if f8 else torch.bfloat16),
                    normal(g, (n_pages, hkv, d, page), F8 if f8 else torch.bfloat16),
                    *((0.03125, 0.0117) if f8 else (1.0, 1.0)))
    q, k, v = (normal(g, (m, h, d), scale=2.0) for h in (hq, hkv, hkv))
    w = [normal(g, (d,)) if norm else None for _ in range(2)]
    return q, k, v, c, w, (start[r] + i).astype(np.int64), slot.astype(np.int64)


def check_rope(q, k, v, before, after, q_out, w, freq, eps, inter, pos, slot, scales, f8, skip=()):
    """q_out and the cache places of every row against the oracle; all other places unchanged.
    FP32 norm and rotation are off by at most 2^-18 of the pair's magnitudes (the sum of
    squares, root, division and products: below 16 roundings; sine and cosine of an angle
    known to 2^-25 of a turn: 2^-21; two products and a sum), then half a step of the type."""
    half = 2.0 ** -8
    live = np.array([i for i in range(len(pos)) if pos[i] >= 0 and i not in skip], int)
    y, mag = ko.rotated_heads(host(q)[live], None if w[0] is None else host(w[0]), eps, freq, pos[live], inter)
    assert (np.abs(host(q_out)[live] - y) <= half * np.abs(y) * (1 + half) + 2.0 ** -18 * mag).all()
    kb, vb = (host(x) for x in before)
    ka, va = (host(x) for x in after)
    page = kb.shape[2]
    yk, mk = ko.rotated_heads(host(k)[live], None if w[1] is None else host(w[1]), eps, freq, pos[live], inter)
    n_slots = kb.shape[0] * page
    seen_k, seen_v = np.zeros(kb.shape, bool), np.zeros(vb.shape, bool)
    for j, i in enumerate(live):
        if not 0 <= slot[i] < n_slots:
            continue
        p, o = divmod(int(slot[i]), page)
        seen_k[p, :, o], seen_v[p, :, :, o] = True, True
        gk, gv, ev = ka[p, :, o], va[p, :, :, o], host(v)[i]
        if f8:
            # E4M3: half a step 2^-4 of a normal value, 2^-10 of a subnormal one
            want = np.clip(yk[j] / scales[0], -448, 448)
            assert (np.abs(gk - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + 2.0 ** -17 * mk[j] / scales[0]).all()
            want = np.clip(ev / np.float32(scales[1]), -448, 448)
            assert (np.abs(gv - want) <= 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -10).all()
        else:
            assert (np.abs(gk - yk[j]) <= half * np.abs(yk[j]) * (1 + half) + 2.0 ** -18 * mk[j]).all()
            assert np.array_equal(gv, ev)
    assert np.array_equal(np.where(seen_k, 0, ka), np.where(seen_k, 0, kb))
    assert np.array_equal(np.where(seen_v, 0, va), np.where(seen_v, 0, vb))


ROPE = [  # m, hq, hkv, d, rot, interleaved, norm, f8, page, rows per request
    (1, 40, 8, 128, 128, False, True, False, 16, 1),
    (1, 1, 1, 64, 64, False, False, True, 16, 1),
    (7, 5, 1, 64, 32, True, True, False, 32, 3),
    (24, 40, 8, 128, 128, False, True, True, 16, 1),
    (120, 40, 8, 128, 128, False, True, True, 16, 5),
    (33, 6, 2, 256, 256, False, True, False, 64, 11),
    (33, 3, 3, 256, 128, True, False, True, 128, 33),
    (50, 28, 4, 128, 96, False, True, False, 256, 17),
    (50, 28, 4, 128, 48, True, True, True, 16, 50),
    (19, 12, 4, 64, 16, False, True, True, 16, 4),
    (300, 16, 16, 64, 64, True, True, False, 16, 100),
    (1031, 10, 2, 128, 128, False, True, False, 16, 600),
    (1031, 10, 2, 128, 0, False, True, True, 32, 77),
]


@pytest.mark.parametrize("m,hq,hkv,d,rot,inter,norm,f8,page,per", ROPE)
def test_qk_rope(m, hq, hkv, d, rot, inter, norm, f8, page, per):
    say("qk_rope", m, hq, hkv, d, rot, inter, norm, f8, page, per)
    g = np.random.default_rng([11, m, hq, d, rot])
    q, k, v, c, w, pos, slot = rope_case(g, m, hq, hkv, d, page, f8, norm, per)
    freq = 1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))
    before = c.k.clone(), c.v.clone()
    r = w12.Rope(torch.from_numpy(freq).to(DEV) if rot else None, *w, eps=1e-5, interleaved=inter)
    out = w12.qk_rope(q, k, v, c, r, i32(pos), i32(slot))
    check_rope(q, k, v, before, (c.k, c.v), out, w, freq, 1e-5, inter, pos, slot, (c.k_scale, c.v_scale), f8)


@pytest.mark.parametrize("f8", [False, True])
def test_qk_rope_strided_in_place_and_padded(f8):
    """q, k, v as columns of one buffer, q turned in place; rows without a position are left
    alone, rows without a slot (-1, or past the pool) still get their q."""
    g = np.random.default_rng(12)
    m, hq, hkv, d, page = 29, 6, 2, 128, 16
    _, _, _, c, w, pos, slot = rope_case(g, m, hq, hkv, d, page, f8, True)
    buf = normal(g, (m, (hq + 2 * hkv) * d + 24))
    q = buf[:, :hq * d].unflatten(1, (hq, d))
    k = buf[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = buf[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    q0, rest0 = q.clone(), buf[:, hq * d:].clone()
    pos[[0, 13, 28]] = [-1, -5, -2147483648]
    slot[[3, 4, 5]] = [-1, c.k.shape[0] * page, 2147483647]
    freq = 1e4 ** (-np.arange(64) / 64)
    before = c.k.clone(), c.v.clone()
    r = w12.Rope(torch.from_numpy(freq).to(DEV), *w)
    w12.qk_rope(q, k, v, c, r, i32(pos), i32(slot), q)
    check_rope(q0, k, v, before, (c.k, c.v), q, w, freq, 1e-6, False, pos, slot, (c.k_scale, c.v_scale), f8)
    assert torch.equal(q[[0, 13, 28]], q0[[0, 13, 28]]) and torch.equal(buf[:, hq * d:], rest0)


def test_qk_rope_far_positions():
    """Angles of positions up to 2^31 - 1: known to 2^31 2^-53 of a turn and its products."""
    g = np.random.default_rng(13)
    q, k, v, c, w, pos, slot = rope_case(g, 8, 2, 1, 64, 16, False, False, per=1)
    pos[:] = [0, 1, 2147483647, 2147483646, 1 << 24, (1 << 24) + 1, 123456789, 1 << 30]
    freq = 1e4 ** (-np.arange(32) / 32)
    out = w12.qk_rope(q, k, v, c, w12.Rope(torch.from_numpy(freq).to(DEV)), i32(pos), i32(slot))
    y, mag = ko.rotated_heads(host(q), None, 0.0, freq, pos, False)
    assert (np.abs(host(out) - y) <= 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(y) + 2.0 ** -18 * mag).all()
    assert torch.equal(out[0], q[0])


@pytest.mark.parametrize("f8", [False, True])
def test_qk_rope_non_finite_rows_stay_apart(f8):
    """A row of NaN or infinity spoils its own heads and no other row; E4M3 saturates."""
    g = np.random.default_rng(14)
    m, hq, hkv, d = 6, 4, 2, 128
    q, k, v, c, w, pos, slot = rope_case(g, m, hq, hkv, d, 16, f8, True, per=1)
    freq = 1e4 ** (-np.arange(64) / 64)
    r = w12.Rope(torch.from_numpy(freq).to(DEV), *w)
    clean = w12.KvCache(c.k.clone(), c.v.clone(), c.k_scale, c.v_scale)
    ref = w12.qk_rope(q, k, v, clean, r, i32(pos), i32(slot))
    q[2, 1, 5], k[2, 0, 7], v[2, 1, 9] = float("nan"), float("inf"), float("nan")
    v[3, 0, :4] = torch.tensor([float("inf"), -float("inf"), 3e38, -3e38])
    out = w12.qk_rope(q, k, v, c, r, i32(pos), i32(slot))
    assert torch.isnan(out[2, 1]).all() and torch.equal(out[2, 0], ref[2, 0])
    for i in (0, 1, 3, 4, 5):
        assert torch.equal(out[i], ref[i])
    p, o = divmod(int(slot[2]), 16)
    assert torch.isnan(c.k[p, 0, o].float()).any() and torch.isnan(c.v[p, 1, 9, o].float())
    p, o = divmod(int(slot[3]), 16)
    got = c.v[p, 0, :4, o].float().cpu().tolist()
    assert got == ([448.0, -448.0, 448.0, -448.0] if f8 else
                   [float("inf"), -float("inf")] + torch.tensor([3e38, -3e38]).bfloat16().float().tolist())


def test_qk_rope_zero_row_without_eps():
    """x = 0 with eps = 0: 0 / 0, as the formula has it; with eps it is zero."""
    g = np.random.default_rng(15)
    q, k, v, c, w, pos, slot = rope_case(g, 2, 1, 1, 64, 16, False, True, per=1)
    q[0] = 0
    for eps, check in ((0.0, torch.isnan), (1e-6, lambda t: t == 0)):
        assert check(w12.qk_rope(q, k, v, c, w12.Rope(None, *w, eps=eps), i32(pos), i32(slot))[0]).all()


# ---------------------------------------------------------------------------------- attention
class Ctx:
    """A filled cache with block tables in shuffled pages, and queries."""

    def __init__(self, g, lens, rows, hq, hkv, d, page, f8=False, start=0, tail=0, extra=2, peak=2.0, scales=None):
        need = [-(-max(0, x) // page) for x in lens]
        self.n_pages = sum(need) + 3
        dt = F8 if f8 else torch.bfloat16
        self.c = w12.KvCache(normal(g, (self.n_pages, hkv, page, d), dt), normal(g, (self.n_pages, hkv, d, page), dt),
                             *(scales or ((0.5, 0.25) if f8 else (1.0, 1.0))))
        perm = g.permutation(self.n_pages)
        self.table = np.full((len(lens), max(max(need), 1) + extra), -1, np.int32)
        a = 0
        for r, x in enumerate(need):
            self.table[r, :x] = perm[a:a + x]
            a += x
        self.off = offsets(rows, start)
        self.m = int(self.off[-1]) + tail
        self.lens = list(lens)
        self.q = normal(g, (self.m, hq, d), scale=peak)
        self.out = torch.full((self.m, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        self.d = d

    def run(self, **kw):
        kw.setdefault("out", self.out)
        return w12.attn_paged(self.q, self.c, i32(self.table), i32(self.lens), i32(self.off), **kw)

    def check(self, out=None, scale=None):
        got = host(self.run(scale=scale) if out is None else out)
        k = host(self.c.k) * self.c.k_scale
        v = host(self.c.v) * self.c.v_scale
        want, tol = ko.attention(host(self.q), k, v, self.table, self.lens, self.off,
                                 self.d ** -0.5 if scale is None else scale)
        mine = np.zeros(self.m, bool)
        mine[self.off[0]:self.off[-1]] = True
        assert (got[~mine] == 7.0).all(), "rows of no request were written"
        fine = np.isfinite(want[mine])
        assert np.array_equal(np.isfinite(got[mine]), fine)
        err = np.abs(got[mine] - want[mine])[fine]
        assert (err <= tol[mine][fine]).all(), float((err / tol[mine][fine]).max())
        return got


ATTN = [  # lens, rows, hq, hkv, d, page, f8
    ([1], [1], 40, 8, 128, 16, False),
    ([17], [1], 40, 8, 128, 16, False),
    ([1, 2, 15, 16, 17, 31, 32, 33], [1] * 8, 5, 1, 128, 16, False),
    ([63, 64, 65, 127, 128, 129, 0, 5], [1, 2, 3, 4, 5, 1, 1, 0], 8, 8, 128, 16, False),
    ([300], [1], 16, 1, 64, 32, False),
    ([300, 41], [3, 5], 17, 1, 64, 16, False),
    ([1000, 3, 511], [2, 3, 7], 12, 4, 256, 64, False),
    ([2500], [1], 8, 1, 256, 128, False),
    ([700, 700], [16, 16], 40, 8, 128, 256, False),
    ([260], [130], 6, 2, 128, 16, False),
    ([70], [70], 3, 3, 64, 16, False),
    ([5000], [1], 4, 2, 128, 16, False),
    ([17], [1], 40, 8, 128, 16, True),
    ([1, 2, 15, 16, 17, 31, 32, 33], [1] * 8, 5, 1, 128, 16, True),
    ([63, 64, 65, 127, 128, 129, 0, 5], [1, 2, 3, 4, 5, 1, 1, 0], 8, 8, 64, 16, True),
    ([1000, 3, 511], [2, 3, 7], 12, 4, 256, 64, True),
    ([700, 700], [16, 16], 40, 8, 128, 256, True),
    ([3000, 900], [5, 5], 14, 2, 64, 32, True),
    ([333], [90], 7, 1, 128, 32, True),
    ([777, 778], [40, 33], 4, 2, 256, 32, False),
    ([50], [2], 128, 1, 64, 16, False),
    ([2000], [3], 96, 1, 128, 16, True),
    ([9000, 5000], [16, 9], 40, 8, 128, 16, False),
    ([9000, 5000], [16, 9], 40, 8, 128, 16, True),
    ([6000, 4000], [4, 4], 32, 4, 256, 64, False),
]


@pytest.mark.parametrize("lens,rows,hq,hkv,d,page,f8", ATTN)
def test_attention(lens, rows, hq, hkv, d, page, f8):
    say("attn", lens, rows, hq, hkv, d, page, f8)
    Ctx(np.random.default_rng([21, sum(lens), d]), lens, rows, hq, hkv, d, page, f8, start=1, tail=2).check()


SHARED = [  # lens, rows, hq, hkv, d, page: several tiles of query rows read a cache together
    ([9000, 5000], [40, 33], 32, 8, 128, 64),
    ([9000, 3, 5000, 0, 64, 65], [40, 2, 60, 0, 64, 65], 32, 8, 128, 128),
    ([1000], [40], 8, 2, 128, 64),
    ([200, 129], [160, 129], 3, 3, 128, 256),
    ([20000], [16], 64, 4, 128, 64),
    ([9000, 8000, 300], [20, 7, 3], 16, 4, 256, 16),
    ([9000, 0, 1, 6000], [3, 0, 1, 50], 36, 3, 256, 256),
    ([5000, 4000], [64, 100], 4, 4, 256, 64),
    ([33, 31, 96], [5, 31, 9], 5, 1, 256, 32),
]


@pytest.mark.parametrize("lens,rows,hq,hkv,d,page", SHARED)
def test_attention_of_shared_tiles(lens, rows, hq, hkv, d, page):
    say("attention of shared tiles", lens, rows, hq, hkv, d, page)
    Ctx(np.random.default_rng([29, lens[0], rows[0], d]), lens, rows, hq, hkv, d, page, start=1, tail=2).check()


@pytest.mark.parametrize("lens,rows,hq,hkv,d,page", [
    ([5000, 4500, 130], [40, 50, 12], 32, 8, 128, 64), ([9000, 8000, 130], [20, 7, 3], 16, 4, 256, 16)])
def test_attention_of_shared_tiles_ignores_what_lies_behind(lens, rows, hq, hkv, d, page):
    """NaN in every free place, an infinite value that only the last row sees, a page that is none
    and a length that is none: each reaches its own rows only."""
    say("attention of shared tiles, what lies behind", lens, rows, d)
    x = Ctx(np.random.default_rng([30, d]), lens, rows, hq, hkv, d, page)
    clean = x.run().clone()
    k, v = x.c.k.view(torch.int16), x.c.v.view(torch.int16)
    used = np.zeros((x.n_pages, page), bool)
    for r, n in enumerate(lens):
        t = np.arange(n)
        used[x.table[r, t // page], t % page] = True
    free = torch.from_numpy(~used).to(DEV)
    k.copy_(torch.where(free[:, None, :, None], 0x7fc0, k))
    v.copy_(torch.where(free[:, None, None, :], 0x7fc0, v))
    assert torch.equal(x.run(), clean)
    x.check()
    last = lens[0] - 1
    v[int(x.table[0, last // page]), :, 3, last % page] = 0x7f80
    got, keep = x.run().clone(), torch.ones_like(clean, dtype=torch.bool)
    assert not torch.isfinite(got[rows[0] - 1, :, 3].float()).any()
    keep[rows[0] - 1, :, 3] = False
    assert torch.equal(got[keep], clean[keep])
    x.table[0, 70 // page] = x.n_pages
    x.lens[2] = -1
    got = x.check()     # (the pieces of request 1 differ now, and so may its last bits)
    mine = slice(rows[0], rows[0] + rows[1])
    assert np.isfinite(got[mine]).all() and np.isnan(got[:rows[0]]).all() and np.isnan(got[mine.stop:]).all()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_many_requests(d, f8):
    """300 requests, lengths 0 to 400, up to 4 rows, some requests without rows."""
    g = np.random.default_rng([22, d])
    rows = g.integers(0, 5, 300)
    Ctx(g, g.integers(0, 400, 300), rows, 4, 2, d, 16, f8).check()


def test_attention_most_requests():
    """4096 requests, most without rows or tokens, a few long ones among them."""
    g = np.random.default_rng(32)
    rows = (g.random(4096) < 0.05).astype(int) * g.integers(1, 4, 4096)
    lens = np.where(g.random(4096) < 0.5, 0, g.integers(0, 40, 4096))
    lens[[7, 2000, 4095]], rows[[7, 2000, 4095]] = [3000, 1, 1500], [2, 1, 20]
    Ctx(g, lens, rows, 2, 1, 64, 16, extra=0).check()


@pytest.mark.parametrize("f8", [False, True])
def test_attention_queries_stay_apart(f8):
    """NaN and infinity in one query row: the others are as they were, bit for bit."""
    g = np.random.default_rng(33)
    x = Ctx(g, [200, 70], [5, 2], 10, 2, 128, 16, f8)
    clean = x.run().clone()
    x.q[2, 3, 7], x.q[6, 0, 0] = float("nan"), float("inf")
    got = x.run()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[2, 3], keep[6, 0] = False, False
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[2, 3]).all()


def test_attention_longest_table():
    """A length of 2^24 tokens through a table whose pages repeat: 16 different pages, so the
    result is that of 256 tokens (every weight 2^16 times)."""
    g = np.random.default_rng(34)
    x = Ctx(g, [256], [1], 2, 1, 64, 16, peak=1.0)
    want, tol = ko.attention(host(x.q), host(x.c.k), host(x.c.v), x.table, x.lens, x.off, 0.125)
    x.table = np.tile(x.table[:, :16], (1, 1 << 16))
    x.lens = [1 << 24]
    # 2^18 units over 1024 waves: a lane adds 16 weights of each of 256 units, then waves and
    # pieces; below 2^13 roundings of 2^-23 (tol allows 256) of a sum of w |v| <= max |v|
    assert (np.abs(host(x.run()) - want) <= tol + 2.0 ** -10 * np.abs(host(x.c.v)).max()).all()


def test_attention_rows_before_the_first_token():
    """kv_len smaller than the number of rows: the first rows see nothing and are zero."""
    got = Ctx(np.random.default_rng(23), [3, 0, 1], [6, 2, 70], 5, 1, 128, 16).check()
    assert (got[:3] == 0).all() and (got[6:8] == 0).all() and (got[8:77] == 0).all() and (got[77] != 0).any()


@pytest.mark.parametrize("f8", [False, True])
def test_attention_ignores_what_lies_behind(f8):
    """NaN and infinity in every free place, in the tails of pages, and in new tokens that
    later rows see but earlier ones do not."""
    g = np.random.default_rng(24)
    x = Ctx(g, [37, 130, 64], [1, 5, 3], 10, 2, 128, 16, f8)
    k, v = x.c.k.view(torch.uint8 if f8 else torch.int16), x.c.v.view(torch.uint8 if f8 else torch.int16)
    used = np.zeros((x.n_pages, 16), bool)
    for r, n in enumerate(x.lens):
        for t in range(n):
            used[x.table[r, t // 16], t % 16] = True
    free = torch.from_numpy(~used).to(DEV)
    bad = 0x7f if f8 else 0x7fc0
    k.copy_(torch.where(free[:, None, :, None], bad, k))
    v.copy_(torch.where(free[:, None, None, :], bad, v))
    x.check()
    clean = x.run().clone()
    # the last token of request 1 is spoiled: its last row alone sees it
    p, o = x.table[1, 129 // 16], 129 % 16
    v[int(p), :, 3, o] = 0x7f if f8 else 0x7f80
    got = x.run()
    assert not torch.isfinite(got[5, :, 3].float()).any()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[5, :, 3] = False
    assert torch.equal(got[keep], clean[keep])
    # and its key as well
    k[int(p), :, o] = bad
    got = x.run()
    assert torch.isnan(got[5].float()).all()
    keep[5] = False
    assert torch.equal(got[keep], clean[keep])


def test_attention_infinite_scores():
    """Keys of -inf direction give weight 0; a row whose scores are all -inf is 0 / 0."""
    g = np.random.default_rng(25)
    x = Ctx(g, [40, 20], [1, 1], 2, 1, 64, 16)
    x.q.abs_()
    for t in range(5, 40):
        x.c.k[int(x.table[0, t // 16]), :, t % 16] = -float("inf")
    for t in range(20):
        x.c.k[int(x.table[1, t // 16]), :, t % 16] = -float("inf")
    got = x.check()
    assert np.isfinite(got[0]).all() and np.isnan(got[1]).all()


@pytest.mark.parametrize("n", [40, 4000])
def test_attention_broken_requests(n):
    """kv_len out of range and table entries out of range give NaN to the rows concerned."""
    g = np.random.default_rng(26)
    x = Ctx(g, [n, n, n, n, n], [2, 2, 2, 2, 2], 4, 2, 64, 16)
    x.lens[1], x.lens[3] = -1, x.table.shape[1] * 16 + 1
    x.table[2, 1] = x.n_pages
    x.table[4, (n - 1) // 16] = -1
    got = x.check()
    assert [bool(np.isnan(got[2 * r:2 * r + 2]).all()) for r in range(5)] == [False, True, True, True, True]


@pytest.mark.parametrize("off", [[-1, 2, 3], [0, 2, 1], [0, 2, 9], [3, 2, 3]])
def test_attention_broken_offsets(off):
    x = Ctx(np.random.default_rng(27), [20, 30], [2, 2], 4, 2, 64, 16)
    x.off = np.array(off)
    assert torch.isnan(x.run().float()).all()


def test_attention_strides_and_scale():
    """q and out as columns of wider buffers; what lies between stays; another scale, and 0."""
    g = np.random.default_rng(28)
    x = Ctx(g, [100, 33], [2, 3], 6, 2, 128, 16)
    wide, room = normal(g, (5, 1000)), torch.full((5, 904), 7.0, dtype=torch.bfloat16, device=DEV)
    x.q = wide[:, 200:968].unflatten(1, (6, 128))
    out = room[:, 8:776].unflatten(1, (6, 128))
    for s in (None, 0.3, -0.05, 0.0):
        x.check(x.run(out=out, scale=s), s)
        assert (room[:, :8] == 7).all() and (room[:, 776:] == 7).all()


def test_attention_long_context_is_joined():
    """One request over many workgroups, several heads and rows; and the same bits each time."""
    x = Ctx(np.random.default_rng(29), [20011], [2], 4, 1, 128, 16)
    a = x.run().clone()
    x.check(a)
    for _ in range(5):
        assert torch.equal(x.run(out=torch.zeros_like(a)), a)


def test_attention_ragged_lengths():
    """Short and very long requests together, in every cache type."""
    for f8 in (False, True):
        Ctx(np.random.default_rng(30), [9000, 1, 70, 4097, 2, 0, 333], [1, 1, 4, 2, 1, 1, 1], 8, 2, 64, 32, f8).check()


def test_attention_places_past_32_bits():
    """A pool of more than 2^32 bytes: pages at its far end (offsets in 64 bits)."""
    hkv, d, page = 8, 256, 256
    n_pages = (1 << 32) // (hkv * d * page * 2) + 70
    c = w12.kv_cache(n_pages, page, hkv, d, device=DEV)
    g = np.random.default_rng(31)
    ids = [n_pages - 1, 0, n_pages - 3]
    c.k[ids] = normal(g, (3, hkv, page, d))
    c.v[ids] = normal(g, (3, hkv, d, page))
    q = normal(g, (2, 8, d))
    table = np.array([ids], np.int32)
    pos = np.array([600, 601])
    slot = ids[2] * page + pos - 512
    knew, vnew = normal(g, (2, hkv, d)), normal(g, (2, hkv, d))
    w12.qk_rope(q, knew, vnew, c, w12.Rope(), i32(pos), i32(slot))
    assert torch.equal(c.k[ids[2], :, 88], knew[0]) and torch.equal(c.v[ids[2], :, :, 89], vnew[1])
    got = host(w12.attn_paged(q, c, i32(table), i32([602]), i32([0, 2])))
    want, tol = ko.attention(host(q), host(c.k[ids]), host(c.v[ids]), np.array([[0, 1, 2]]), [602], [0, 2], d ** -0.5)
    assert (np.abs(got - want) <= tol).all()
    del c
    torch.cuda.empty_cache()


# -------------------------------------------------------------------- streams, graphs, together
def test_two_streams_at_once():
    g = np.random.default_rng(41)
    xs = [Ctx(g, [8000, 5], [1, 2], 8, 1, 128, 16) for _ in range(2)]
    want = [x.run().clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    args = [(i32(x.table), i32(x.lens), i32(x.off)) for x in xs]
    outs = [torch.zeros_like(x.out) for x in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, s, a, o in zip(xs, streams, args, outs):
            with torch.cuda.stream(s):
                w12.attn_paged(x.q, x.c, *a, out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[:3], w[:3])


def chain(g, n=5, hq=8, hkv=2, d=64, page=16, f8=False):
    """One layer's attention side for n requests of up to 3 rows, as a serving loop has it."""
    rows = 1 + g.integers(0, 3, n)
    m = int(rows.sum())
    pt = w12.page_table(200, page, n, 30, DEV)
    c = w12.kv_cache(200, page, hkv, d, F8 if f8 else torch.bfloat16, *((0.0625, 0.0625) if f8 else ()), device=DEV)
    freq = 1e4 ** (-np.arange(d // 2) / (d // 2))
    w = [normal(g, (d,)), normal(g, (d,))]
    rope = w12.Rope(torch.from_numpy(freq).to(DEV), *w)
    return rows, m, pt, c, freq, w, rope


@pytest.mark.parametrize("f8", [False, True])
def test_serving_loop_together(f8):
    """kv_plan, qk_rope and attn_paged over steps of a serving loop with rejected drafts and a
    request that ends, against an oracle that keeps every request's tokens in a list (the
    stored keys and values are taken from the cache, so only this step's error counts)."""
    g = np.random.default_rng([42, f8])
    n, hq, hkv, d, page = 5, 8, 2, 64, 16
    rows, m, pt, c, freq, w, rope = chain(g, n, hq, hkv, d, page, f8)
    length = np.zeros(n, np.int64)
    toks = [[] for _ in range(n)]     # per request: (raw k, raw v) in order
    for step in range(12):
        rows = g.integers(0, 20, n) if step == 0 else 1 + g.integers(0, 5, n)
        if step == 6:
            length[2], rows[2], toks[2] = 0, 0, []      # request 2 ends
        off = offsets(rows)
        m = int(off[-1])
        q, k, v = (normal(g, (m, h, d)) for h in (hq, hkv, hkv))
        kv_len, pos, slot = w12.kv_plan(pt, i32(length), i32(off), m)
        qr = w12.qk_rope(q, k, v, c, rope, pos, slot)
        out = w12.attn_paged(qr, c, pt.table, kv_len, i32(off))
        assert kv_len.cpu().tolist() == (length + rows).tolist()
        for r in range(n):
            toks[r] = toks[r][:length[r]] + [(host(k)[i], host(v)[i]) for i in range(off[r], off[r + 1])]
        # the cache holds exactly these tokens, turned by their positions
        tab, kc, vc = pt.table.cpu().numpy(), host(c.k) * c.k_scale, host(c.v) * c.v_scale
        step_of = 2.0 ** -4 if f8 else 2.0 ** -8
        for r in range(n):
            for t, (kr, vr) in enumerate(toks[r]):
                y, mag = ko.rotated_heads(kr[None], host(w[1]), 1e-6, freq, [t], False)
                p, o = tab[r, t // page], t % page
                small = 2.0 ** -10 * 0.0625 if f8 else 0.0
                assert (np.abs(kc[p, :, o] - y[0]) <= step_of * np.abs(y[0]) * (1 + step_of) + 2.0 ** -16 * mag[0] + small).all()
                assert (np.abs(vc[p, :, :, o] - vr) <= (step_of if f8 else 0) * np.abs(vr) + small).all()
        want, tol = ko.attention(host(qr), kc, vc, tab, length + rows, off, d ** -0.5)
        assert (np.abs(host(out) - want) <= tol).all()
        length = np.maximum(0, length + rows - g.integers(0, 3, n) * (rows > 2))   # some drafts rejected
    length[:] = 0
    w12.kv_plan(pt, i32(length), i32([0] * (n + 1)), 0)
    assert int(pt.state[1]) == pt.n_pages and sorted(pt.ring.cpu().tolist()) == list(range(pt.n_pages))


def test_captured_step_replays():
    """The three calls captured into a graph (prepared and plain), replayed with new lengths,
    eager work in between: every replay gives the eager result."""
    g = np.random.default_rng(43)
    n, hq, hkv, d = 5, 8, 2, 64
    rows, m, pt, c, freq, w, rope = chain(g, n, hq, hkv, d)
    q, k, v = (normal(g, (m, h, d)) for h in (hq, hkv, hkv))
    off = i32(offsets(rows))
    length = i32(np.zeros(n))
    kv_len, pos, slot = i32(np.zeros(n)), i32(np.zeros(m)), i32(np.zeros(m))
    qr, out, out2 = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    calls = []

    def step():
        w12.kv_plan(pt, length, off, m, kv_len, pos, slot)
        w12.qk_rope(q, k, v, c, rope, pos, slot, qr)
        w12.attn_paged(qr, c, pt.table, kv_len, off, out=out)
        for f in calls:
            f()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls.append(w12.prepare_attn_paged(qr, c, pt.table, kv_len, off, out2, ws=w12.attn_workspace(DEV)))
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(6):
        length.copy_(i32(g.integers(0, 400, n)))
        q.copy_(normal(g, (m, hq, d)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (kv_len, pos, slot, qr, out, out2)]
        # the same step again, eagerly: the tables already fit, so nothing moves
        w12.kv_plan(pt, length, off, m, kv_len, pos, slot)
        w12.qk_rope(q, k, v, c, rope, pos, slot, qr)
        w12.attn_paged(qr, c, pt.table, kv_len, off, out=out)
        torch.cuda.synchronize()
        for a, b in zip(got, (kv_len, pos, slot, qr, out, out)):
            assert torch.equal(a, b)


def test_refusals_on_the_device():
    """Wrong types, shapes and overlaps are refused before any launch."""
    x = Ctx(np.random.default_rng(44), [20], [2], 4, 2, 64, 16)
    t, l, o = i32(x.table), i32(x.lens), i32(x.off)
    ok = lambda **kw: w12.attn_paged(**{**dict(q=x.q, cache=x.c, table=t, kv_len=l, req_off=o), **kw})
    ok()
    for kw in (dict(table=t.long()), dict(kv_len=l.long()), dict(req_off=o[:1]), dict(q=x.q.float()), dict(q=x.q[0]),
               dict(q=x.q[..., :32]), dict(q=x.q.transpose(0, 1)), dict(out=x.q), dict(out=x.out[:1]),
               dict(table=t[0]), dict(table=t.cpu()), dict(ws=torch.zeros(64, device=DEV)),
               dict(cache=w12.KvCache(x.c.k, x.c.k)), dict(cache=w12.KvCache(x.c.k.half(), x.c.v.half())),
               dict(q=x.q[:1].expand(2, 4, 64))):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(ws=torch.zeros(4096, dtype=torch.uint8, device=DEV)), dict(scale=float("nan")),
               dict(q=torch.zeros(2, 3, 64, dtype=torch.bfloat16, device=DEV)),
               dict(cache=w12.KvCache(x.c.k, x.c.v, 2.0))):
        with pytest.raises(w12.W12Error):
            ok(**kw)
    pt = w12.page_table(4, 16, 2, 3, DEV)
    with pytest.raises(ValueError):
        w12.kv_plan(pt, l, o, 2, kv_len=l)
    with pytest.raises(ValueError):
        w12.kv_plan(pt, l, o, 2, slot=pt.ring[:2])
    with pytest.raises(w12.W12Error):
        w12.kv_plan(pt, i32([0, 0, 0]), i32([0, 0, 0, 0]), 0)
    k = x.q[:, :2].contiguous()
    with pytest.raises(ValueError):
        w12.qk_rope(x.q, k, k[:1], x.c, w12.Rope(), i32([0, 1]), i32([0, 1]))
    with pytest.raises(ValueError):
        w12.qk_rope(x.q, k, k, x.c, w12.Rope(torch.zeros(32, device=DEV)), i32([0, 1]), i32([0, 1]))
    with pytest.raises(w12.W12Error):
        w12.qk_rope(x.q, k, k, x.c, w12.Rope(torch.zeros(4, device=DEV, dtype=torch.float64)), i32([0, 1]), i32([0, 1]))


def test_empty_batches():
    x = Ctx(np.random.default_rng(45), [20], [0], 4, 2, 64, 16)
    assert x.m == 0 and x.run().shape == (0, 4, 64)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert w12.qk_rope(q, q[:, :2], q[:, :2], x.c, w12.Rope(), i32([]), i32([])).shape == (0, 4, 64)
