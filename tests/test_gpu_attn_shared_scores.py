"""Attention over shared tokens where scores are far apart, close together at great size, or rise as the
tokens go by: the softmax's running reference on either line, the workgroups' and the waves'.  Tolerances
are those of the same inputs under the attention that shares nothing (test_gpu_attn_scores.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_attn_shared import Group, beams  # noqa: E402
from tests.test_gpu_kv import DEV  # noqa: E402

pytestmark = pytest.mark.gpu

FORMS = [  # requests, rows of each, hq, hkv, d, page, f8
    (9, 5, 10, 2, 64, 16, False),      # 225 query rows a head: each wave rows of its own
    (9, 5, 10, 2, 128, 16, False),
    (7, 5, 12, 4, 256, 64, False),
    (9, 5, 10, 2, 64, 16, True),
    (9, 5, 10, 2, 128, 16, True),
    (60, 2, 5, 1, 128, 32, True),      # 600: three items
    (7, 5, 12, 4, 256, 64, True),
    (3, 4, 5, 1, 128, 16, True),       # 60: waves take tokens too
    (10, 1, 4, 1, 64, 16, True),       # 40
    (3, 2, 3, 1, 256, 16, True),       # 18
    (2, 1, 4, 2, 128, 16, True),       # 4: the waves' line
    (3, 4, 5, 1, 128, 16, False),
]


def filled(g, shared, own, form, keys, values, query):
    """Heads whose queries are `query` {dimension: value}, with keys(t) {dimension: values} and values(t) per
    token, the same in every dimension and for every request."""
    n, rows, hq, hkv, d, page, f8 = form
    x = Group(g, [beams(n, shared, own, rows)], hq, hkv, d, page, f8, scales=(1.0, 1.0))
    x.q.zero_()
    for i, q in query.items():
        x.q[..., i] = q
    k, v = np.zeros((x.n_pages, hkv, page, d), np.float32), np.zeros((x.n_pages, hkv, d, page), np.float32)
    for r, end in enumerate(x.lens):
        t = np.arange(end)
        at = x.table[r, t // page], t % page
        for i, kk in keys(t).items():
            k[at[0], :, at[1], i] = kk[:, None]
        v[at[0], :, :, at[1]] = values(t)[:, None, None]
    x.c.k.copy_(torch.from_numpy(k).to(x.c.k.dtype).to(DEV))
    x.c.v.copy_(torch.from_numpy(v).to(x.c.v.dtype).to(DEV))
    return x


def compare(x, rows, want_of, tol_of, **kw):
    """Every row against want_of(the tokens it sees)."""
    got = x.run(**kw).double().cpu().numpy()
    for r, n in enumerate(x.lens):
        for i in range(rows):
            t = np.arange(n - rows + i + 1)
            want = want_of(t)
            err = np.abs(got[r * rows + i] - want)
            assert (err <= tol_of(t, want)).all(), (r, i, got[r * rows + i].ravel()[:3], want)


@pytest.mark.parametrize("form", [f for f in FORMS if f[6]])
@pytest.mark.parametrize("power", [18, 33])
@pytest.mark.parametrize("shared", [64, 1088, 20032])
def test_small_weights(shared, power, form):
    """One token of weight 1 with value 0 and the others of weight 2^-power with value 256: none is lost, on
    whichever line its rows are."""
    say("shared, small weights", shared, power, form)
    x = filled(np.random.default_rng([101, shared]), shared, 3, form,
               lambda t: {5: np.where(t == 0, 0.0, -float(power // 2)), 6: np.where(t == 0, 0.0, -float(power % 2))},
               lambda t: np.where(t == 0, 0.0, 256.0), {5: 2.0, 6: 1.0})
    mean = lambda t: 256 * (len(t) - 1) * 2.0 ** -power / (1 + (len(t) - 1) * 2.0 ** -power)
    compare(x, form[1], mean, lambda t, want: (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * want, scale=float(np.log(2)))


@pytest.mark.parametrize("form", [f for f in FORMS if f[6]])
def test_bits_of_a_weight(form):
    """Weights over an E4M3 cache keep 11 bits: 256 or more tokens of weight 0.502 and value 1 stand against one of
    weight 1 and value -128, so that what is left of their sum is the weight's last bits."""
    say("shared, weights", form)
    weight = 0.5 * (1 + 0.98 * 2.0 ** -8)
    value = lambda t: np.where(t == 0, -128.0, 1.0)
    x = filled(np.random.default_rng(102), 256, 1, form, lambda t: {5: np.where(t == 0, 0.0, -1.0)}, value, {5: 1.0})

    def sums(t):
        w = np.where(t == 0, 1.0, weight)
        return (w * value(t)).sum() / w.sum(), (w * np.abs(value(t))).sum() / w.sum()
    compare(x, form[1], lambda t: sums(t)[0],
            lambda t, want: 2.0 ** -8 * abs(want) + (2.0 ** -11 + 2.0 ** -18) * (1 + 2.0 ** -7) * sums(t)[1],
            scale=-float(np.log(weight)))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("power", [15, 16, 17, 18, 22])
def test_scores_half_apart(power, form):
    """Scores 2^power, 2^power + 1/2 and 2^power + 1 (exact in FP32), the last two in one unit of tokens
    each: the weights are 1, e^(1/2) and e."""
    say("shared, scores half apart", power, form)
    step = lambda t: np.where(t // 64 == 2, 0.5, 0) + np.where(t // 64 == 4, 1.0, 0)
    for shared in (640, 5056):
        x = filled(np.random.default_rng(103), shared, 9, form, lambda t: {5: np.ones(len(t)), 6: step(t)},
                   lambda t: 2 * step(t), {5: 2.0 ** power, 6: 1.0})
        compare(x, form[1], lambda t: (np.exp(step(t)) * 2 * step(t)).sum() / np.exp(step(t)).sum(),
                lambda t, want: (2.0 ** -7 + 2.0 ** -14) * want, scale=1.0)


@pytest.mark.parametrize("form", FORMS)
def test_largest_score_wins(form):
    """Scores of 2^power and one of 1.125 2^power, in the first unit, in the middle or the last that is shared: its
    token's values come back alone."""
    say("shared, largest score", form)
    for power in (16, 17, 24, 25, 31, 60):
        for best in (7, 1087):
            x = filled(np.random.default_rng(104), 1088, 9, form, lambda t: {5: np.where(t == best, 1.125, 1.0)},
                       lambda t: np.where(t == best, 1.75, 1.0 + t % 2), {5: 2.0 ** power})
            assert (x.run(scale=1.0) == 1.75).all(), (power, best)


@pytest.mark.parametrize("form", FORMS)
def test_equal_scores_of_every_size(form):
    """All scores 1.125 2^power, or -1.125 2^power: every weight is 1, the result is the mean."""
    say("shared, equal scores", form)
    x = filled(np.random.default_rng(105), 640, 9, form, lambda t: {5: np.full(len(t), 1.125)}, lambda t: t % 2 + 1.0, {5: 1.0})
    for power in list(range(10, 50)) + [60, 100]:
        for sign in (1.0, -1.0):
            x.q[..., 5] = sign * 2.0 ** power
            compare(x, form[1], lambda t: 1 + (len(t) // 2) / len(t),
                    lambda t, want: 2.0 ** -8 * (1 + 2.0 ** -8) * want, scale=1.0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("step", [0.0625, 0.25, 0.40625, 0.625, 0.75, 3.0, 6.0, -0.625, -3.0])
def test_scores_that_rise(step, form):
    """Scores that rise (or fall) by `step` every 32 tokens, sixteen times over, far above the smallest and
    not: weights between the reference's steps, and references between the waves' and the pieces'."""
    say("shared, rising scores", step, form)
    n, rows, hq, hkv, d, page, f8 = form
    for far in (0.0, 2.0 ** 16):
        x = filled(np.random.default_rng(106), 1600, 9, form,
                   lambda t: {5: (t // 32 % 16).astype(float), 6: np.ones(len(t))}, lambda t: 1.0 + t % 3, {5: step, 6: far})
        s = lambda t: np.exp(step * (t // 32 % 16) - max(0.0, step * 15))
        # weights: BF16 2^-8, FP16 2^-11 (and E4M3's 2^-9 of rounded exponents far out); the result: BF16 2^-8
        compare(x, rows, lambda t: (s(t) * (1 + t % 3)).sum() / s(t).sum(), lambda t, want: (2.0 ** -7 + 2.0 ** -14) * want, scale=1.0)
