"""Attention with scores so large that their scaled value has few or no bits left below 1: only their
distance from the largest counts, and that is exact here."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_attn_counts import FORMS  # noqa: E402
from tests.test_gpu_kv import Ctx  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def filled(g, lens, rows, hq, hkv, d, page, f8, keys, values, query):
    """Heads whose queries are `query` {dimension: value}, with keys(r, t) {dimension: values} and
    values(r, t) per token, the same in every dimension."""
    x = Ctx(g, lens, [rows] * len(lens), hq, hkv, d, page, f8, scales=(1.0, 1.0))
    x.q.zero_()
    for i, q in query.items():
        x.q[..., i] = q
    k, v = np.zeros((x.n_pages, hkv, page, d), np.float32), np.zeros((x.n_pages, hkv, d, page), np.float32)
    for r, n in enumerate(lens):
        t = np.arange(n)
        at = x.table[r, t // page], t % page
        for i, kk in keys(r, t).items():
            k[at[0], :, at[1], i] = kk[:, None]
        v[at[0], :, :, at[1]] = values(r, t)[:, None, None]
    x.c.k.copy_(torch.from_numpy(k).to(x.c.k.dtype).to(DEV))
    x.c.v.copy_(torch.from_numpy(v).to(x.c.v.dtype).to(DEV))
    return x


LENS = [300, 5000, 33]


@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", FORMS)
def test_attention_scores_half_apart(rows, hq, hkv, d, page, f8):
    """Scores 2^22, 2^22 + 1/2 and 2^22 + 1 (exact in FP32), the last two in one unit of tokens each: the
    weights are 1, e^(1/2) and e however the tokens are dealt to waves and pieces."""
    say("scores half apart", rows, hq, hkv, d, page, f8)
    g = np.random.default_rng([94, d])
    step = lambda t: np.where(t // 64 == 2, 0.5, 0) + np.where(t // 64 == 4, 1.0, 0)
    x = filled(g, LENS, rows, hq, hkv, d, page, f8, lambda r, t: {5: np.ones(len(t)), 6: step(t)},
               lambda r, t: 2 * step(t), {5: 2.0 ** 22, 6: 1.0})
    got = x.run(scale=1.0).double().cpu().numpy()
    a = 0
    for n in LENS:
        for i in range(rows):
            t = np.arange(max(n - rows + i + 1, 0))
            w = np.exp(step(t))
            want = (w * 2 * step(t)).sum() / w.sum() if len(t) else 0.0
            # weights: BF16 2^-8, FP32 below 2^-18; the result: BF16 2^-8
            assert (np.abs(got[a + i] - want) <= (2.0 ** -7 + 2.0 ** -14) * want).all(), (n, i)
        a += rows


@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", FORMS)
@pytest.mark.parametrize("power", [24, 25, 31, 36, 60])
def test_attention_largest_score_wins(power, rows, hq, hkv, d, page, f8):
    """Scores of 2^power and one of 1.125 2^power: its token's values come back alone."""
    say("largest score", power, rows, hq, hkv, d, page, f8)
    g = np.random.default_rng([95, d])
    best = 7
    x = filled(g, LENS, rows, hq, hkv, d, page, f8, lambda r, t: {5: np.where(t == best, 1.125, 1.0)},
               lambda r, t: np.where(t == best, 1.75, 1.0 + t % 2), {5: 2.0 ** power})
    got = x.run(scale=1.0).double().cpu().numpy()
    a = 0
    for n in LENS:
        for i in range(rows):
            if n - rows + i >= best:
                assert (got[a + i] == 1.75).all(), (n, i)
        a += rows


@pytest.mark.parametrize("rows,hq,hkv,d,page,f8", FORMS)
def test_attention_equal_large_scores(rows, hq, hkv, d, page, f8):
    """All scores 1.125 2^40, or -1.125 2^40: every weight is 1, the result is the mean."""
    say("equal large scores", rows, hq, hkv, d, page, f8)
    g = np.random.default_rng([96, d])
    for sign in (1.0, -1.0):
        x = filled(g, LENS, rows, hq, hkv, d, page, f8, lambda r, t: {5: np.full(len(t), 1.125)},
                   lambda r, t: t % 2 + 1.0, {5: sign * 2.0 ** 40})
        got = x.run(scale=1.0).double().cpu().numpy()
        a = 0
        for n in LENS:
            for i in range(rows):
                e = max(n - rows + i + 1, 0)
                want = 1 + (e // 2) / e if e else 0.0
                assert (np.abs(got[a + i] - want) <= 2.0 ** -8 * (1 + 2.0 ** -8) * want).all(), (n, i)
            a += rows


@pytest.mark.parametrize("rows,hq,hkv,d,page", [f[:5] for f in FORMS if f[5]])
def test_attention_e4m3_weights(rows, hq, hkv, d, page):
    """Weights over an E4M3 cache keep 11 bits: n tokens of weight 0.502 and value 1 stand against one of
    weight 1 and value -n / 2, so that what is left of their sum is the weight's last bits."""
    say("E4M3 weights", rows, hq, hkv, d, page)
    g = np.random.default_rng([97, d])
    lens, weight = [33, 65, 257], 0.5 * (1 + 0.98 * 2.0 ** -8)
    value = lambda r, t: np.where(t == 0, -(lens[r] // 2.0), 1.0)
    x = filled(g, lens, rows, hq, hkv, d, page, True, lambda r, t: {5: np.where(t == 0, 0.0, -1.0)}, value, {5: 1.0})
    got = x.run(scale=-float(np.log(weight))).double().cpu().numpy()
    a = 0
    for r, n in enumerate(lens):
        for i in range(rows):
            t = np.arange(n - rows + i + 1)
            w, v = np.where(t == 0, 1.0, weight), value(r, t)
            want, size = (w * v).sum() / w.sum(), (w * np.abs(v)).sum() / w.sum()
            # weights: half a step of FP16, 2^-11; exp2, scale and FP32 sums below 2^-18; the result: 2^-8
            tol = 2.0 ** -8 * abs(want) + (2.0 ** -11 + 2.0 ** -18) * (1 + 2.0 ** -7) * size
            assert (np.abs(got[a + i] - want) <= tol).all(), (n, i, got[a + i].ravel()[0], want)
        a += rows


@pytest.mark.parametrize("rows,hq,hkv,d,page", [f[:5] for f in FORMS if f[5]])
@pytest.mark.parametrize("power", [18, 33])
def test_attention_e4m3_small_weights(power, rows, hq, hkv, d, page):
    """One token of weight 1 with value 0 and thousands of weight 2^-power with value 256: none is lost."""
    say("E4M3 small weights", power, rows, hq, hkv, d, page)
    g = np.random.default_rng([98, d])
    x = filled(g, LENS, rows, hq, hkv, d, page, True,
               lambda r, t: {5: np.where(t == 0, 0.0, -float(power // 2)), 6: np.where(t == 0, 0.0, -float(power % 2))},
               lambda r, t: np.where(t == 0, 0.0, 256.0), {5: 2.0, 6: 1.0})
    got = x.run(scale=float(np.log(2))).double().cpu().numpy()
    a, w = 0, 2.0 ** -power
    for n in LENS:
        for i in range(rows):
            e = max(n - rows + i + 1, 0)
            want = 256 * (e - 1) * w / (1 + (e - 1) * w) if e else 0.0
            assert (np.abs(got[a + i] - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * want).all(), (n, i)
        a += rows
