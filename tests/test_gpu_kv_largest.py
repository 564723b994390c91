"""The cache calls at their largest numbers of rows and heads, checked on samples."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from oracle import kv_oracle as ko  # noqa: E402
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_attn_counts import REL, column  # noqa: E402
from tests.test_gpu_kv import Ctx, check_rope, host, i32, normal  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_most_rows_through_plan_and_rope():
    """2^20 rows of two prompts: positions and slots exact, the heads of a sample of rows against the
    oracle, values of every token in place."""
    say("2^20 rows")
    m, page, d = w12.MAX_KV_ROWS, 256, 64
    rows = [700_000, m - 700_000]
    n_pages = sum(-(-r // page) for r in rows) + 3
    pt = w12.page_table(n_pages, page, 2, 2 + rows[0] // page + 1, DEV)
    kv_len, pos, slot = w12.kv_plan(pt, i32([5, 0]), i32([0, rows[0], m]), m)
    assert kv_len.cpu().tolist() == [rows[0] + 5, rows[1]]
    p = np.concatenate([np.arange(rows[0]) + 5, np.arange(rows[1])])
    tab = pt.table.cpu().numpy()
    s = tab[np.repeat([0, 1], rows), p // page].astype(np.int64) * page + p % page
    assert np.array_equal(pos.cpu().numpy(), p) and np.array_equal(slot.cpu().numpy(), s)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    q, k, v = (torch.randn((m, 1, d), generator=g, device=DEV).bfloat16() for _ in range(3))
    c = w12.kv_cache(n_pages, page, 1, d, device=DEV)
    freq = 1e4 ** (-np.arange(d // 2) / (d // 2))
    out = w12.qk_rope(q, k, v, c, w12.Rope(torch.from_numpy(freq).to(DEV)), pos, slot)
    assert torch.equal(c.v.permute(0, 3, 1, 2).reshape(-1, 1, d)[slot.long()], v)
    at = np.unique(np.concatenate([[0, 1, rows[0] - 1, rows[0], m - 1], np.random.default_rng(1).integers(0, m, 3000)]))
    for x, y in ((q, out), (k, c.k.permute(0, 2, 1, 3).reshape(-1, 1, d)[slot.long()])):
        want, mag = ko.rotated_heads(host(x[at]), None, 0.0, freq, p[at], False)
        assert (np.abs(host(y[at]) - want) <= 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want) + 2.0 ** -18 * mag).all()


def test_most_heads():
    """1024 query heads over 1 and over 1024 key heads, turned and attending."""
    say("1024 heads")
    g = np.random.default_rng(99)
    for hkv, d, f8 in ((1, 64, False), (1024, 64, True), (2, 256, False)):
        m, page = 3, 16
        x = Ctx(g, [33, 20], [2, 1], 1024, hkv, d, page, f8)
        x.check()
        pos, slot = np.array([31, 32, 19]), None
        slot = x.table[[0, 0, 1], pos // page].astype(np.int64) * page + pos % page
        k, v = normal(g, (m, hkv, d)), normal(g, (m, hkv, d))
        freq = 1e4 ** (-np.arange(d // 2) / (d // 2))
        before = x.c.k.clone(), x.c.v.clone()
        out = w12.qk_rope(x.q, k, v, x.c, w12.Rope(torch.from_numpy(freq).to(DEV)), i32(pos), i32(slot))
        check_rope(x.q, k, v, before, (x.c.k, x.c.v), out, [None, None], freq, 1e-6, False, pos, slot,
                   (x.c.k_scale, x.c.v_scale), f8)


@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", [(200_001, 1, 1, 64, 16, False), (60_000, 4, 1, 128, 64, False),
                                                   (60_000, 4, 1, 128, 32, True), (40_000, 2, 1, 256, 64, False)])
def test_attention_of_long_prompts(rows, hq, hkv, d, page, f8):
    """A prompt over its own tokens, and a short one behind it, with q = 0: shares of tokens, on a sample of
    rows."""
    say("long prompt", rows, hq, d, f8)
    lens, n_rows = [rows + 70, 40], [rows, 40]
    x = Ctx(np.random.default_rng(100), lens, n_rows, hq, hkv, d, page, f8, scales=(1.0, 1.0))
    x.q.zero_()
    v = np.zeros((x.n_pages, hkv, d, page), np.float32)
    for r, n in enumerate(lens):
        t = np.arange(n)
        v[x.table[r, t // page], 0, column(t, r, 0, d, 16), t % page] = 1
    x.c.v.copy_(torch.from_numpy(v).to(x.c.v.dtype).to(DEV))
    out = x.run()
    g = np.random.default_rng(101)
    for r, i in [(0, int(i)) for i in (0, 1, 15, 16, 31, 32, rows - 1, *g.integers(0, rows, 60))] + [(1, i) for i in range(40)]:
        end = lens[r] - n_rows[r] + i + 1
        want = np.bincount(column(np.arange(end), r, 0, d, 16), minlength=d) / end
        got = host(out[(rows if r else 0) + i])
        assert (np.abs(got - want) <= REL * want).all(), (r, i)


def test_fewer_requests_than_table_rows():
    """A call on the first requests of a larger table leaves the others' pages alone."""
    from tests.test_gpu_kv import Pool, offsets
    g = np.random.default_rng(102)
    p = Pool(400, 16, 300, 12, head=390)
    p.step(g.integers(0, 15, 300), offsets([1] * 300), 300)
    for n in (3, 256, 257, 1):
        for _ in range(3):
            p.step(g.integers(0, 170, n), offsets(g.integers(0, 9, n)), 9 * n)
    x = Ctx(g, [40, 100, 7], [2, 1, 3], 4, 2, 64, 16)
    want = x.run().clone()
    x.table = np.concatenate([x.table, np.full((5, x.table.shape[1]), x.n_pages, np.int32)])
    assert torch.equal(x.run(out=torch.full_like(want, 7.0)), want)
