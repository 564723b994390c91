"""One workspace, made for the largest of several calls, serves all of them, larger and smaller in turn."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_beam import DEV, check, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
def test_one_workspace_as_beams_finish(f32):
    say("beam_select, one workspace", f32)
    g, vocab = np.random.default_rng(84), 50257
    ws = w12.beam_workspace(96, vocab, 32)
    for rows, k in ((96, 32), (78, 16), (79, 16), (95, 8), (4, 32), (4, 16), (1, 1), (96, 17)):
        groups = np.concatenate([np.arange(0, rows, 4), [rows]])
        check(logits(g, rows, vocab, f32), g.standard_normal(rows) * 3 - 20, groups, k, ws=ws)
        assert not ws[:16384].any()
