"""Attention of requests that share their first tokens, on the GPU against the 64-bit oracle of the
attention (each request by itself), with the oracle's allowance: the parts' join adds two FP32
roundings per part and two exponentials, which the allowance's 2^-20 of each weight and 2^-23 per token hold."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_kv import DEV, F8, Ctx, i32, normal  # noqa: E402

pytestmark = pytest.mark.gpu


class Group(Ctx):
    """groups: (shared tokens, lengths, rows) per group, lengths in all.  Requests of a group hold its
    first request's pages for the shared tokens' full pages; other requests' entries of whole shared
    units are no pages at all where `own` is false (they are not read)."""

    def __init__(self, g, groups, hq, hkv, d, page, f8=False, only_first=True, **kw):
        lens = [x for _, ls, _ in groups for x in ls]
        rows = [x for _, _, rs in groups for x in rs]
        super().__init__(g, lens, rows, hq, hkv, d, page, f8, **kw)
        self.grp_off = np.concatenate([[0], np.cumsum([len(ls) for _, ls, _ in groups])])
        self.grp_len = [s for s, _, _ in groups]
        self.seen = self.table.copy()    # what the kernel is given
        for (s, ls, rs), a in zip(groups, self.grp_off):
            live = [r for r in range(a, a + len(ls)) if rows[r] and lens[r] >= 0]
            if len(live) < 2:
                continue
            full = max(0, s) // page
            self.table[a:a + len(ls), :full] = self.table[live[0], :full]
            self.seen[a:a + len(ls), :full] = self.table[live[0], :full]
            least = min([s] + [lens[r] - rows[r] + 1 for r in live])
            unread = max(0, least) // 64 * 64 // page if only_first else 0
            for r in live[1:]:
                self.seen[r, :unread] = -1
            if full * page < s:
                self.grp_len[list(self.grp_off).index(a)] = full * page

    def run(self, **kw):
        kw.setdefault("out", self.out)
        return w12.attn_shared(self.q, self.c, i32(self.seen), i32(self.lens), i32(self.off), i32(self.grp_off),
                               i32(self.grp_len), **kw)


def beams(n, shared, own, rows):
    return shared, [shared + own + 7 * i for i in range(n)], [rows] * n


CASES = [  # groups, hq, hkv, d, page, f8
    ([beams(4, 304, 1, 1)], 40, 8, 128, 16, False),
    ([beams(4, 304, 1, 1)], 40, 8, 128, 16, True),
    ([beams(2, 64, 1, 1)], 1, 1, 64, 16, False),
    ([beams(2, 63, 1, 1)], 2, 1, 64, 16, False),
    ([beams(2, 128, 0, 1)], 3, 1, 128, 64, False),          # no token but the shared ones
    ([beams(9, 1024, 5, 1), beams(1, 500, 3, 2), beams(3, 0, 40, 4)], 10, 2, 128, 32, False),
    ([beams(33, 700, 5, 5)], 16, 2, 128, 16, False),         # 1320 query rows: several tiles
    ([beams(13, 2048, 9, 5)], 10, 2, 64, 16, True),
    ([beams(7, 640, 20, 3)], 12, 4, 256, 64, False),
    ([beams(40, 640, 20, 3)], 12, 4, 256, 64, False),
    ([beams(40, 640, 20, 3)], 12, 4, 256, 64, True),
    ([beams(64, 8000, 20, 1)], 40, 8, 128, 16, False),
    ([beams(64, 8000, 20, 2)], 5, 1, 128, 256, True),
    ([beams(3, 20000, 900, 2)], 8, 1, 128, 16, False),
    ([beams(5, 192, 1, 8), (0, [5, 0, 900], [1, 1, 9]), beams(2, 256, 300, 16)], 16, 1, 64, 128, False),
    ([beams(20, 130, 3, 16)], 4, 4, 128, 16, False),
]


@pytest.mark.parametrize("groups,hq,hkv,d,page,f8", CASES)
def test_attention_over_shared_tokens(groups, hq, hkv, d, page, f8):
    say("attn_shared", [(s, len(x), r[0]) for s, x, r in groups], hq, hkv, d, page, f8)
    x = Group(np.random.default_rng([51, d, len(groups)]), groups, hq, hkv, d, page, f8, start=1, tail=2)
    got = x.check()
    for _ in range(3):
        assert np.array_equal(x.run(out=torch.full_like(x.out, 7.0)).double().cpu().numpy(), got), "same inputs, other bits"


@pytest.mark.parametrize("rows", [33, 64, 65, 96, 127, 128, 129, 160, 256, 257, 290, 513])
@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True), (256, False)])
def test_numbers_of_query_rows(rows, d, f8):
    """Around the borders of the tiles, with tokens that are no whole number of steps."""
    n = 3
    each = [rows // n + (i < rows % n) for i in range(n)]
    x = Group(np.random.default_rng([52, rows]), [(832, [832 + max(each) + 3 * i for i in range(n)], each)], 1, 1, d, 16, f8)
    x.check()


@pytest.mark.parametrize("shared", [64, 65, 127, 128, 192, 256, 320, 1088, 4096 + 64])
@pytest.mark.parametrize("d,f8", [(64, True), (128, False), (128, True), (256, True)])
def test_numbers_of_shared_tokens(shared, d, f8):
    x = Group(np.random.default_rng([53, shared]), [beams(6, shared, 2, 7)], 2, 1, d, 16, f8)
    x.check()


def test_many_groups():
    """300 groups of 0 to 5 requests, and 4096 requests in 1000 groups, most without rows."""
    g = np.random.default_rng(54)
    groups = []
    for i in range(300):
        n, s = int(g.integers(0, 6)), int(g.integers(0, 300))
        groups.append((s, [s + int(g.integers(1, 60)) for _ in range(n)], g.integers(0, 4, n).tolist()))
    Group(g, groups, 4, 2, 64, 16).check()
    groups = []
    for i in range(1024):
        s = int(g.integers(0, 200)) * (i % 50 == 0)
        groups.append((s, [s + int(g.integers(0, 9)) for _ in range(4)], (g.random(4) < 0.1).astype(int).tolist()))
    Group(g, groups, 2, 1, 64, 16, extra=0).check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [128, 256])
def test_rows_that_see_less_than_what_is_shared(d, f8):
    """Lengths below the shared tokens and more rows than tokens: shared is what every row sees."""
    g = np.random.default_rng(55)
    Group(g, [(640, [640, 300, 700], [1, 2, 3]), (100, [3, 200], [6, 1]), (64, [64, 70], [2, 3])], 5, 1, d, 16, f8).check()


@pytest.mark.parametrize("f8", [False, True])
def test_what_lies_behind(f8):
    """NaN in every free place; an infinite value that the last of a request's rows alone sees."""
    x = Group(np.random.default_rng(56), [beams(4, 208, 20, 5), beams(2, 64, 6, 3)], 10, 2, 128, 16, f8, only_first=False)
    k, v = x.c.k.view(torch.uint8 if f8 else torch.int16), x.c.v.view(torch.uint8 if f8 else torch.int16)
    used = np.zeros((x.n_pages, 16), bool)
    for r, n in enumerate(x.lens):
        t = np.arange(n)
        used[x.table[r, t // 16], t % 16] = True
    free = torch.from_numpy(~used).to(DEV)
    bad = 0x7f if f8 else 0x7fc0
    k.copy_(torch.where(free[:, None, :, None], bad, k))
    v.copy_(torch.where(free[:, None, None, :], bad, v))
    clean = x.run().clone()
    x.check()
    last = x.lens[1] - 1
    v[int(x.table[1, last // 16]), :, 3, last % 16] = 0x7f if f8 else 0x7f80
    got, keep = x.run(), torch.ones_like(clean, dtype=torch.bool)
    assert not torch.isfinite(got[9, :, 3].float()).any()
    keep[9, :, 3] = False
    assert torch.equal(got[keep], clean[keep])
    k[int(x.table[1, last // 16]), :, last % 16] = bad
    got = x.run()
    keep[9] = False
    assert torch.isnan(got[9].float()).all() and torch.equal(got[keep], clean[keep])
    # a shared value that is not finite reaches every row of its group
    v[int(x.table[0, 3]), :, 5, 2] = 0x7f if f8 else 0x7f80
    got = x.run().float()
    assert not torch.isfinite(got[:20, :, 5]).any() and torch.isfinite(got[20:]).all()


def test_queries_stay_apart():
    x = Group(np.random.default_rng(57), [beams(5, 256, 20, 5)], 10, 2, 128, 16)
    clean = x.run().clone()
    x.q[2, 3, 7], x.q[20, 0, 0] = float("nan"), float("inf")
    got, keep = x.run(), torch.ones_like(clean, dtype=torch.bool)
    keep[2, 3], keep[20, 0] = False, False
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[2, 3]).all()


def test_infinite_scores():
    """Keys of -inf direction in the shared tokens have weight 0; a row whose scores are all -inf is 0 / 0."""
    x = Group(np.random.default_rng(58), [(128, [140, 150], [1, 1]), (128, [128, 128], [1, 1])], 2, 1, 64, 16)
    x.q.abs_()
    for t in list(range(0, 64)) + [130]:
        x.c.k[int(x.table[0, t // 16]), :, t % 16] = -float("inf")
    for t in range(128):
        x.c.k[int(x.table[2, t // 16]), :, t % 16] = -float("inf")
    got = x.check()
    assert np.isfinite(got[:2]).all() and np.isnan(got[2:]).all()


def test_broken_requests():
    """Lengths that are none: NaN for their rows, and the group goes on, also without its first; pages that
    are none: their own request, or the whole group."""
    say("attn_shared, broken requests")
    groups = [beams(4, 320, 20, 2), beams(3, 320, 20, 2), beams(2, 320, 20, 2), beams(2, 64, 100, 1)]
    x = Group(np.random.default_rng(59), groups, 4, 2, 64, 16, only_first=False)
    x.lens[0], x.lens[2], x.lens[5] = -1, x.table.shape[1] * 16 + 1, -1
    x.seen[0, :20] = -1
    x.seen[7:9, 2] = x.table[7:9, 2] = x.n_pages
    x.seen[10, 8] = x.table[10, 8] = -7
    got = x.check()
    nan = [bool(np.isnan(got[x.off[r]:x.off[r + 1]]).all()) for r in range(11)]
    assert nan == [True, False, True, False, False, True, False, True, True, False, True]


@pytest.mark.parametrize("off,grp", [([-1, 2, 3], [0, 2]), ([0, 2, 1], [0, 2]), ([0, 2, 9], [0, 2]), ([0, 2, 4], [0, 1]),
                                     ([0, 2, 4], [1, 2]), ([0, 2, 4], [0, 3, 2]), ([0, 2, 4], [0, 3]), ([0, 2, 4], [0, -1, 2])])
def test_tables_that_are_none(off, grp):
    x = Group(np.random.default_rng(60), [beams(2, 64, 9, 2)], 4, 2, 64, 16)
    x.off, x.grp_off, x.grp_len = np.array(off), np.array(grp), [64] * (len(grp) - 1)
    assert torch.isnan(x.run().float()).all()


def test_strides_and_scale():
    x = Group(np.random.default_rng(61), [beams(3, 128, 9, 2)], 6, 2, 128, 16)
    wide, room = normal(np.random.default_rng(1), (6, 1000)), torch.full((6, 904), 7.0, dtype=torch.bfloat16, device=DEV)
    x.q = wide[:, 200:968].unflatten(1, (6, 128))
    out = room[:, 8:776].unflatten(1, (6, 128))
    for s in (None, 0.3, -0.05, 0.0):
        x.check(x.run(out=out, scale=s), s)
        assert (room[:, :8] == 7).all() and (room[:, 776:] == 7).all()


def test_a_longest_table():
    """2^24 shared tokens through a table whose pages repeat: the result is that of 256 tokens."""
    from oracle import kv_oracle as ko
    x = Group(np.random.default_rng(62), [(256, [256, 256], [1, 1])], 2, 1, 64, 16, peak=1.0)
    host = lambda t: t.double().cpu().numpy()
    want, tol = ko.attention(host(x.q), host(x.c.k), host(x.c.v), x.table, x.lens, x.off, 0.125)
    x.seen = np.tile(x.table[:, :16], (1, 1 << 16))
    x.lens, x.grp_len = [1 << 24] * 2, [1 << 24]
    # (sums of 2^24 weights: a lane adds 8 of each unit, its pieces and lanes are joined; below 2^13 roundings
    # of 2^-23 beside those that tol allows for 256 tokens)
    assert (np.abs(host(x.run()) - want) <= tol + 2.0 ** -10 * np.abs(host(x.c.v)).max()).all()


@pytest.mark.parametrize("n,f8", [(3, False), (40, False), (40, True)])
def test_pages_beyond_32_bits(n, f8):
    """Pages whose offset within the cache passes 2^32 bytes: the bits of the same pages at its start."""
    x = Group(np.random.default_rng(66), [beams(n, 400, 30, 1)], 8, 8, 128, 16, f8, only_first=False)
    want = x.run().clone()
    small, total = x.c, 280000 if f8 else 140000
    k, v = (torch.empty((total, *t.shape[1:]), dtype=t.dtype, device=DEV) for t in (small.k, small.v))
    at = total - small.k.shape[0]
    k[at:].view(torch.uint8).copy_(small.k.view(torch.uint8))
    v[at:].view(torch.uint8).copy_(small.v.view(torch.uint8))
    x.c = w12.KvCache(k, v, small.k_scale, small.v_scale)
    x.seen = np.where(x.seen >= 0, x.seen + at, x.seen)
    assert torch.equal(x.run(out=torch.full_like(want, 7)), want)


def test_streams_and_captured_graphs():
    """Two streams at once, and two graphs replayed beside eager calls: no workspace is shared."""
    g = np.random.default_rng(63)
    xs = [Group(g, [beams(12, 2000 + 700 * i, 30, 1)], 8, 1, 128, 16) for i in range(2)]
    want = [x.run().clone() for x in xs]
    args = [(x.q, x.c, i32(x.seen), i32(x.lens), i32(x.off), i32(x.grp_off), i32(x.grp_len)) for x in xs]
    outs = [torch.zeros_like(x.out) for x in xs]
    streams, graphs = [torch.cuda.Stream() for _ in xs], []
    torch.cuda.synchronize()
    for _ in range(10):
        for a, s, o in zip(args, streams, outs):
            with torch.cuda.stream(s):
                w12.attn_shared(*a, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for a, o in zip(args, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w12.attn_shared(*a, out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = w12.attn_shared(*args[0])
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs + [eager], want + [want[0]]))


def test_no_rows():
    x = Group(np.random.default_rng(64), [(64, [70, 70], [0, 0])], 2, 1, 64, 16)
    assert x.run().shape == (0, 2, 64)
    x = Group(np.random.default_rng(64), [(64, [70, 70], [0, 0])], 2, 1, 64, 16, start=2, tail=1)
    assert (x.run() == 7).all()


def test_as_many_rows_as_there_may_be():
    """2^17 query rows of 64 requests, compared with the attention that shares nothing."""
    g = np.random.default_rng(65)
    x = Group(g, [beams(16, 512, 70, 64) for _ in range(4)], 32, 2, 64, 16, only_first=False)
    assert x.m * 32 == w12.MAX_SHARED_ROWS
    got, ref = x.run().float(), w12.attn_paged(x.q, x.c, i32(x.table), i32(x.lens), i32(x.off)).float()
    # each is its FP32 result rounded to BF16 and has BF16 weights: 2 (2^-8 + 2^-8) of the largest value
    assert (got - ref).abs().max() <= 4 * 2.0 ** -8 * float(x.c.v.float().abs().max())
    assert (got - ref).norm() <= 0.01 * ref.norm()
