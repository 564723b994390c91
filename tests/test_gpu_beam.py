"""The choice of beams on the GPU against the 64-bit oracle.  Rows and tokens have to be equal unless two
rows' scores are closer than 1e-7 (what a row's log-sum-exp is within: a term exp(t) is off by 2^-23 of
itself and 2^-24 |t| exp(t), in either direction, the FP32 sums of at most 64 terms of a thread by
2^-24 of them per addition, likewise, and all of them are averaged over the row); the inputs here are drawn so that none
are.  Scores are rounded to FP32: 2^-24 of them, and 1e-7 for the log-sum-exp."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from oracle import fork_oracle as fo  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int32)).to(DEV)


def check(x, scores, off, k, **kw):
    """x a CPU tensor [n, vocab] (a view may be strided), scores float32."""
    s = torch.as_tensor(np.asarray(scores, np.float32))
    parent, token, score, close = fo.beam_select(x.double().numpy(), s.double().numpy(), off, k)
    assert close > 1e-7, "inputs whose order is not certain"
    got = w12.beam_select(kw.pop("dev", None) if "dev" in kw else x.to(DEV), s.to(DEV), i32(off), k, **kw)
    p, t, v = (g.cpu().numpy() for g in got)
    assert np.array_equal(p, parent) and np.array_equal(t, token)
    fin = np.isfinite(score)
    assert np.array_equal(np.isnan(v), np.isnan(score)) and np.array_equal(v == -np.inf, score == -np.inf)
    assert (np.abs(v[fin] - score[fin]) <= 2.0 ** -24 * np.abs(score[fin]) + 1e-7).all()
    return got


def logits(g, n, vocab, f32, scale=2.5):
    x = torch.from_numpy(g.standard_normal((n, vocab), dtype=np.float32) * np.float32(scale))
    return x if f32 else x.bfloat16()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,vocab,k", [
    ([1], 1, 1), ([2], 3, 3), ([1], 7, 7), ([4], 64, 64), ([4, 1, 0, 3], 1000, 8), ([2, 2], 4095, 5), ([3], 4097, 16),
    ([3], 4096, 17), ([5, 5], 16383, 64), ([1, 1, 1], 16385, 33), ([4] * 3, 50257, 8), ([16, 2], 32001, 32),
    ([64], 5003, 64), ([64], 20011, 16), ([4], 151936, 8), ([4] * 24, 30011, 8), ([1] * 60, 151, 4), ([2], 700001, 64),
    ([1], 1 << 21, 16), ([2], 300007, 4), ([8] * 10, 60000, 12), ([2], 90001, 16)])
def test_choice(rows, vocab, k, f32):
    print("beam_select", rows, vocab, k, f32, flush=True)
    g = np.random.default_rng([71, vocab, k, f32])
    n = sum(rows)
    check(logits(g, n, vocab, f32), g.standard_normal(n) * 3 - 20, np.concatenate([[0], np.cumsum(rows)]), k)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("vocab,k", [(5, 5), (1000, 64), (16384, 8), (40000, 64)])
def test_equal_logits(vocab, k, f32):
    """All equal: the lowest tokens, and rows with the same scores in order; more equal values than a
    part's candidates have room for."""
    x = torch.full((3, vocab), 1.5, dtype=torch.float32 if f32 else torch.bfloat16)
    check(x, [-1.0, -1.0, -1.0], [0, 2, 3], k)
    x[1] = -0.0
    x[1, ::3] = 0.0
    check(x[:2], [-1.0, -2.0], [0, 2], k)
    # a few values, in turn
    x = torch.arange(3 * vocab).remainder(7).reshape(3, vocab).to(x.dtype)
    check(x, [0.25, 1.0, -0.5], [0, 3], k)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("stride", [256, 1024, 64])
def test_largest_values_of_one_thread(f32, stride):
    """The largest values `stride` tokens apart, so that few threads hold them all."""
    g = np.random.default_rng(72)
    x = logits(g, 2, 33000, f32, 0.5)
    x[:, 5::stride] = (20 + torch.arange(len(x[0, 5::stride])) / 8)[g.permutation(len(x[0, 5::stride]))].to(x.dtype)
    check(x, [0.1, -0.2], [0, 2], 64)


def test_what_is_no_number():
    """-inf and NaN logits, rows without a finite one, +inf, scores of -inf and NaN."""
    g = np.random.default_rng(73)
    for f32 in (False, True):
        x = logits(g, 6, 999, f32)
        x[0, ::2] = -float("inf")
        x[1, 500] = float("nan")
        x[2] = -float("inf")
        x[3, 7] = float("inf")
        x[5] = float("nan")
        check(x, [0, 0, 0, 0, 0, 0], [0, 6], 20)
        check(x, [0, 0, 0, 0, -np.inf, 0], [0, 3, 6], 33)
        check(x[2:4], [0.0, 0.0], [0, 1, 2], 9)
        check(x[:1], [np.nan], [0, 1], 9)
        x[0] = -float("inf")
        x[0, [3, 998]] = 2.0
        check(x[[0, 4]], [0.0, -9.0], [0, 2], 7)
        check(x[:1], [0.0], [0, 1], 7)      # -inf tokens by number behind the two


def test_large_and_small_logits():
    g = np.random.default_rng(74)
    for scale in (1e-30, 1e-3, 300.0, 1e30):
        check(logits(g, 3, 5000, True, scale), [0.0, -0.5, 0.25], [0, 1, 3], 9) if scale < 1e4 else \
            check(logits(g, 1, 5000, True, scale), [0.0], [0, 1], 9)


@pytest.mark.parametrize("f32", [False, True])
def test_rows_anywhere(f32):
    """Rows that begin at every place of a 16-byte vector, columns of a wider buffer with NaN beside them."""
    g = np.random.default_rng(75)
    for skip in range(0, 9):
        wide = torch.full((4, 4120 + skip % 5), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16)
        wide[:, skip:skip + 4099] = logits(g, 4, 4099, f32)
        dev = wide.to(DEV)
        check(wide[:, skip:skip + 4099], g.standard_normal(4), [0, 2, 4], 6, dev=dev[:, skip:skip + 4099])
        check(wide[:, skip:skip + 3], g.standard_normal(4), [0, 4], 3, dev=dev[:, skip:skip + 3])


def test_rows_of_no_group_and_groups_without_rows():
    g = np.random.default_rng(76)
    x = logits(g, 7, 500, True)
    check(x, g.standard_normal(7), [1, 1, 3, 3, 5, 5], 4)
    none = w12.beam_select(torch.empty((0, 500), device=DEV), torch.empty(0, device=DEV), i32([0, 0, 0]), 4)
    assert (none[0] == -1).all() and (none[1] == -1).all() and (none[2] == -float("inf")).all()


@pytest.mark.parametrize("off", [[-1, 2], [0, 3, 2], [0, 5], [3, 2, 4], [0, 2, 1, 4]])
def test_groups_that_are_none(off):
    x = logits(np.random.default_rng(77), 4, 500, True)
    check(x, [0, 0, 0, 0], off, 4)


def test_too_many_rows_in_a_group():
    x = logits(np.random.default_rng(78), 70, 50, True)
    check(x, np.zeros(70), [0, 65, 70], 4)
    check(x, np.arange(70) * 0.37, [0, 64, 70], 4)


def test_same_bits_two_streams_and_graphs():
    g = np.random.default_rng(79)
    xs = [logits(g, 8, 151936, f).to(DEV) for f in (False, True)]
    s, off = torch.from_numpy(g.standard_normal(8).astype(np.float32)).to(DEV), i32([0, 3, 8])
    want = [[t.clone() for t in w12.beam_select(x, s, off, 12)] for x in xs]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    streams, graphs = [torch.cuda.Stream() for _ in xs], []
    torch.cuda.synchronize()
    same = lambda: all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
    for _ in range(10):
        for x, st, o in zip(xs, streams, outs):
            with torch.cuda.stream(st):
                w12.beam_select(x, s, off, 12, *o)
        torch.cuda.synchronize()
        assert same()
    for x, o in zip(xs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w12.beam_select(x, s, off, 12, *o)
    for _ in range(3):
        for o in outs:
            o[0].zero_(), o[2].zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        w12.beam_select(xs[0], s, off, 12)
        torch.cuda.synchronize()
        assert same()


def test_refusals():
    x, s, off = torch.zeros((4, 100), device=DEV), torch.zeros(4, device=DEV), i32([0, 4])
    for bad in (lambda: w12.beam_select(x.half(), s, off, 4), lambda: w12.beam_select(x.T, s, off, 4),
                lambda: w12.beam_select(x, s[:3], off, 4), lambda: w12.beam_select(x, s.double(), off, 4),
                lambda: w12.beam_select(x, s, off.long(), 4), lambda: w12.beam_select(x, s, off, 4, score_out=s.view(1, 4)),
                lambda: w12.beam_select(x.expand(4, 100)[:1].expand(4, 100), s, off, 4),
                lambda: w12.beam_select(x, s, off, 4, ws=torch.zeros(100000, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for k in (0, 65, 101):
        with pytest.raises(w12.W12Error):
            w12.beam_select(x, s, off, k)
    with pytest.raises(w12.W12Error):
        w12.beam_select(x, s, off, 4, ws=torch.zeros(16384, dtype=torch.uint8, device=DEV))
