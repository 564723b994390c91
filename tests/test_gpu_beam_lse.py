"""How far a row's log-sum-exp is from exact, where nothing averages out: one logit that stands out and all
others equal, or a random rest behind it, and rows of two values.  The prior score takes the logit's own
log-probability away, so that what comes back is the difference, and FP32 holds it to 2^-24 of
itself.  A term is off by 9.8e-8 of itself at most (8.5e-8 of the hardware's exp2, and 1.3e-8 for the second order
of its argument's rest), the sums are FP64: the log-sum-exp is within 1e-7."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from tests.test_gpu_beam import DEV, i32  # noqa: E402

pytestmark = pytest.mark.gpu
BOUND = 1e-7
# rows whose threads take 16, 32 and 64 values of this vocabulary
SHARES = [24, 48, 96]
VOCAB = 151936


def off_by(x, at):
    """Rows x, each a group: the error of the log-sum-exp, from the score of token `at` or its equal, the
    best."""
    n, top = len(x), x[:, at].double()
    lse = torch.logsumexp(x.double(), -1)
    prior = (lse - top).float()
    parent, token, score = w12.beam_select(x, prior, i32(range(n + 1)), 1)
    assert (parent[:, 0] == torch.arange(n, device=DEV)).all()
    assert (x.gather(1, token.long())[:, 0] == x[:, at]).all()
    want = prior.double() - (lse - top)
    return (score[:, 0].double() - want).abs() - 2.0 ** -24 * want.abs()


def ahead(n):
    """How far the largest logit is ahead: values that the sum's roundings all push one way, and others."""
    return torch.tensor([5.4296875, 2.66796875] + [(37 * i % 4000 + 1) / 256 for i in range(n - 2)], device=DEV)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", SHARES)
@pytest.mark.parametrize("top", [0.0, 8.0, -13.5, 31.0, 33.0, 63.5, 64.5, 300.0, -23.5, -24.5, -70.0])
def test_all_others_equal(top, n, f32):
    x = (top - ahead(n))[:, None].repeat(1, VOCAB)
    x[:, 77] = top
    err = off_by(x if f32 else x.bfloat16(), 77)
    assert (err <= BOUND).all(), err.max().item()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", SHARES)
def test_one_ahead_of_a_random_rest(n, f32):
    g = torch.Generator(device=DEV)
    g.manual_seed(83)
    for at in (77, VOCAB - 1):
        x = torch.randn((n, VOCAB), generator=g, device=DEV) * 2.5
        x[:, at] = 14 + torch.arange(n, device=DEV) / 8
        err = off_by(x if f32 else x.bfloat16(), at)
        assert (err <= BOUND).all(), err.max().item()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", SHARES)
def test_rows_of_two_values(n, f32):
    x = (3.0 - ahead(n))[:, None].repeat(1, VOCAB)
    x[:, 1::2] -= 0.37109375
    x[:, 5::64] = 2.984375
    x[:, 40000] = 3.0
    err = off_by(x if f32 else x.bfloat16(), 40000)
    assert (err <= BOUND).all(), err.max().item()


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 19, 2.0 ** 20, 2.0 ** 21, 2.0 ** 40, 1e38])
def test_logits_of_any_size(scale):
    """Where they are large only those near the largest count: whole numbers from 0 down, the largest of
    each row 0, `scale` or -`scale` (2^21: where the reference changes from 0 to the maximum)."""
    near = -(torch.arange(5003, device=DEV) % 97).float()
    near[1234] = 0.5
    x = torch.stack([near, near + scale, near - scale])
    x[:, 7] = -float("inf")
    x[:, 8:10] = -3.4028234663852886e38
    x[0, 1000:2000] = -scale
    best = x.max(1).values
    at = [int((row == b).nonzero()[0]) for row, b in zip(x, best)]
    for row, j in zip(x, at):
        v = row.double()
        lse = torch.logsumexp(v, -1)
        parent, token, score = w12.beam_select(row[None], torch.zeros(1, device=DEV), i32([0, 1]), 1)
        assert token.item() == j
        assert abs(score.item() - (v[j] - lse).item()) <= BOUND + 2.0 ** -24 * abs((v[j] - lse).item())


@pytest.mark.parametrize("step", [0.5, 40.0, 200.0])
def test_parts_far_apart(step):
    """Rows that rise by `step` from one 4096 logits to the next, up or down, part by part."""
    part = (torch.arange(40 * 4096, device=DEV) // 4096).float()
    for sign in (1.0, -1.0):
        x = (sign * step * part).repeat(2, 1)
        x[:, 50000] = x.max() + 1.0
        assert (off_by(x, 50000) <= BOUND).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("top", [31.5, 32.0, 48.0, 63.0, 64.0, 90.0, -24.0, -25.0])
def test_rests_of_every_distance(top, f32):
    """2^18 logits, alike but for the one that stands out, 10 to 30 below it: where together they weigh as much
    as it does, or nothing, and their distance has more bits than they."""
    g = np.random.default_rng(86)
    n, vocab = 41, 1 << 18
    x = torch.from_numpy(np.repeat((top - np.linspace(10, 30, n) - g.random(n) / 64).astype(np.float32)[:, None], vocab, 1)).to(DEV)
    x = x if f32 else x.bfloat16()
    x[:, 5000] = top
    assert (off_by(x, 5000) <= BOUND).all()
