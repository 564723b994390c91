"""The attention's split and join, to the unit: with q = 0 every weight is exactly 1, and values that
are 1 for some tokens and 0 for the others make every output a count over a length, so a unit
of tokens that is left out, taken twice or given to another row, head or request shows.  And values
that are the same for all tokens come back as they are."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from tests.gpu_util import say  # noqa: E402

gpu = pytest.mark.gpu
DEV = "cuda:0"
# FP32: v_scale / len is off by 2^-24 of itself and its product with the count by 2^-24; then BF16, 2^-8.
REL = 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -22


def column(t, r, h, d, run):
    """The dimension in which token t of request r is 1 in head h: runs of `run` tokens in turn."""
    return (np.asarray(t) // run + 5 * r + 3 * h) % d


def counts(lens, rows, hq, hkv, d, run, drop=None, twice=None):
    """Per row and query head the share of its tokens in each dimension; drop and twice are (request,
    first token, end) of tokens to leave out or to take twice."""
    out = np.zeros((sum(rows), hq, d))
    a = 0
    for r, (n, k) in enumerate(zip(lens, rows)):
        w = np.ones(n)
        for what, by in ((drop, -1), (twice, 1)):
            if what and what[0] == r:
                w[what[1]:what[2]] += by
        for i in range(k):
            end = n - k + i + 1
            if end <= 0:
                continue
            for h in range(hkv):
                c = np.bincount(column(np.arange(end), r, h, d, run), w[:end], d) / w[:end].sum()
                out[a + i, h * (hq // hkv):(h + 1) * (hq // hkv)] = c
        a += k
    return out


@pytest.mark.parametrize("lens,d,unit", [([20011], 128, 32), ([9000, 8000], 256, 32), ([5000, 3], 64, 64), ([131072], 128, 32)])
def test_counts_see_every_unit(lens, d, unit):
    """What the check below would let pass: no unit left out, none taken twice."""
    want = counts(lens, [1] * len(lens), 1, 1, d, 16)
    last = lens[0] // unit
    for u in {0, 1, 2, last // 3, last // 2, last - 2, last - 1}:
        span = (0, u * unit, min((u + 1) * unit, lens[0]))
        for kind in ("drop", "twice"):
            got = counts(lens, [1] * len(lens), 1, 1, d, 16, **{kind: span})
            assert not (np.abs(got - want) <= REL * want).all(), (u, kind)


def run_counts(lens, rows, hq, hkv, d, page, f8, run, extra=1):
    from tests.test_gpu_kv import Ctx
    say("attention counts", lens[:8], rows[:8], hq, hkv, d, page, f8, run)
    g = np.random.default_rng([91, len(lens), d, run])
    scales = (0.5, 0.25) if f8 else (1.0, 1.0)
    x = Ctx(g, lens, rows, hq, hkv, d, page, f8, start=1, tail=1, extra=extra, scales=scales)
    x.q.zero_()
    v = np.zeros((x.n_pages, hkv, d, page), np.float32)
    for r, n in enumerate(lens):
        t = np.arange(n)
        for h in range(hkv):
            v[x.table[r, t // page], h, column(t, r, h, d, run), t % page] = 1
    x.c.v.copy_(torch.from_numpy(v).to(x.c.v.dtype).to(DEV))
    got = x.run().double().cpu().numpy()
    want = counts(lens, rows, hq, hkv, d, run) * scales[1]
    m = sum(rows)
    assert (got[0] == 7).all() and (got[1 + m:] == 7).all()
    err = np.abs(got[1:1 + m] - want)
    assert (err <= REL * want).all(), np.argwhere(err > REL * want)[:5].tolist()


FORMS = [  # rows of a request, hq, hkv, d, page, f8: every kernel form
    (1, 4, 2, 64, 16, False),       # one tile, units of 64
    (7, 10, 2, 64, 16, False),      # tiles of 32
    (2, 8, 2, 128, 16, False),      # one tile, units of 32
    (5, 10, 2, 128, 16, False),     # tiles of 32, units of 32
    (16, 10, 2, 128, 16, False),    # tiles of 32, units of 64
    (30, 10, 2, 128, 64, False),    # the same staged, where the table is wide enough
    (1, 6, 2, 256, 64, False),      # one tile
    (4, 16, 2, 256, 64, False),     # several, staged where the table is wide enough
    (1, 4, 2, 64, 16, True),
    (6, 10, 2, 64, 16, True),
    (2, 8, 2, 128, 32, True),
    (6, 10, 2, 128, 16, True),
    (3, 4, 2, 256, 64, True),
    (5, 16, 2, 256, 16, True),
]


@gpu
@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", FORMS)
@pytest.mark.parametrize("lens", [[20011], [9000, 1, 70, 4097, 2, 0, 333], [64, 40000, 31, 32, 33, 100], [3000, 8192, 8191, 4096, 7]])
def test_attention_counts(lens, rows, hq, hkv, d, page, f8):
    """Long, ragged and brief requests: items cut by one border, by both, and by many."""
    run_counts(lens, [rows] * len(lens), hq, hkv, d, page, f8, 16)


@gpu
@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", FORMS)
def test_attention_counts_single_tokens(rows, hq, hkv, d, page, f8):
    """Every token by itself (an output counts at most 100 of them), in a table of 131072 tokens."""
    n = 90 * d
    run_counts([n, n // 3, 17], [rows, 1, rows], hq, hkv, d, page, f8, 1, extra=131072 // page - (-(-n // page)))


@gpu
@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (256, False), (64, True), (128, True), (256, True)])
def test_attention_counts_many_requests(d, f8):
    """300 brief requests between long ones."""
    g = np.random.default_rng([92, d])
    lens = [int(n) for n in g.integers(0, 130, 300)]
    for r, n in ((0, 5000), (77, 2500), (78, 12000), (299, 3333)):
        lens[r] = n
    run_counts(lens, [int(k) for k in g.integers(0, 4, 300)], 4, 2, d, 16, f8, 16)


@gpu
@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True), (256, True)])
def test_attention_counts_longest(d, f8):
    run_counts([131001], [1], 2, 1, d, 16, f8, 16)


@gpu
@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", [
    (16, 40, 8, 64, 16, False), (16, 40, 8, 128, 16, False), (16, 40, 8, 128, 16, True), (30, 40, 8, 128, 64, False),
    (7, 64, 8, 256, 64, False), (7, 64, 8, 256, 16, True), (130, 24, 8, 64, 32, True)])
def test_attention_counts_items_of_several_tiles(rows, hq, hkv, d, page, f8):
    """Work enough that tiles of a head form one item (16 units for each of 256 workgroups)."""
    run_counts([20011, 5000, 70, 3], [rows, rows, min(rows, 70), 2], hq, hkv, d, page, f8, 16)


@gpu
@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", FORMS)
@pytest.mark.parametrize("lens", [[64, 3, 2, 300], [3000, 1, 777, 4096]])
def test_attention_of_equal_values(lens, rows, hq, hkv, d, page, f8):
    """Values that depend on head and dimension alone are what every row gets, exactly: the weights add
    up to their divisor.  (Both sums have at most t + 3 units + 64 additions and fadings of 2^-24 each,
    for t <= 4096 below 2^-10 together, and a BF16 value's neighbour begins 2^-9 away.)  Scores: one
    token's 0, all others such that their weight lies just below the middle of two BF16 values."""
    from tests.test_gpu_kv import Ctx
    say("attention of equal values", lens, rows, hq, hkv, d, page, f8)
    g = np.random.default_rng([93, lens[0], d])
    x = Ctx(g, lens, [rows] * len(lens), hq, hkv, d, page, f8)
    x.q.zero_()
    x.q[..., 5] = 1
    k = np.zeros((x.n_pages, hkv, page, d), np.float32)
    k[..., 5] = -1
    for r in range(len(lens)):
        k[x.table[r, 0], :, 1 % min(lens[r], page), 5] = 0
    x.c.k.copy_(torch.from_numpy(k).to(x.c.k.dtype).to(DEV))
    value = torch.from_numpy(g.standard_normal((hkv, d)).astype(np.float32)).to(x.c.v.dtype).to(DEV)
    x.c.v.copy_(value[None, :, :, None].expand(x.n_pages, hkv, d, page))
    weight = 0.5 * (1 + 0.98 * 2.0 ** -8)
    got = x.run(scale=-float(np.log(weight)) / x.c.k_scale)
    want = (value.float() * x.c.v_scale).bfloat16().repeat_interleave(hq // hkv, 0)
    a = 0
    for n in lens:
        for i in range(rows):
            assert torch.equal(got[a + i], want if n - rows + i >= 0 else torch.zeros_like(want)), (n, i)
        a += rows
