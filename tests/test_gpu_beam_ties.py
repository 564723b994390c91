"""Rows with the same logits have the same log-sum-exp, bit for bit, wherever they begin in memory: equal
scores of different rows come in the order of the rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from tests.test_gpu_beam import DEV, check, i32, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("vocab", [1001, 32001, 50257, 128259])   # packed rows begin inside a 16-byte vector
@pytest.mark.parametrize("rows,k", [(4, 2), (4, 8), (3, 32), (16, 8)])   # ties across the choice's end among them
def test_rows_with_the_same_logits(rows, k, vocab, f32):
    print("beam_select, equal rows", rows, k, vocab, f32, flush=True)
    g = np.random.default_rng([81, vocab, k])
    x = logits(g, 1, vocab, f32).expand(rows, vocab).contiguous()
    check(x, np.full(rows, -1.0), [0, rows], k)
    # two of them among others
    x = torch.cat([logits(g, 1, vocab, f32), x[:1], logits(g, 2, vocab, f32), x[:1]])
    check(x, [0.5, 0.0, 0.25, -0.25, 0.0], [0, 5], k)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,vocab,k", [(3, 4099, 6), (48, 151931, 8), (96, 30011, 40), (1, 600001, 5)])
def test_scores_wherever_rows_begin(n, vocab, k, f32):
    """The same rows at every place of a vector, at the strides that follow: the same bits."""
    g = np.random.default_rng([82, vocab])
    x, s = logits(g, n, vocab, f32).to(DEV), torch.from_numpy(g.standard_normal(n).astype(np.float32)).to(DEV)
    off = i32(list(range(0, n + 1, 3)) if n % 3 == 0 else [0, n])
    want = w12.beam_select(x, s, off, k)
    for skip in range(1, 9):
        wide = torch.full((n, vocab + skip), float("nan"), dtype=x.dtype, device=DEV)
        wide[:, skip:] = x
        assert all(torch.equal(a, b) for a, b in zip(w12.beam_select(wide[:, skip:], s, off, k), want)), skip
