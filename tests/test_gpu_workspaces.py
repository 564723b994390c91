"""One workspace, made for the largest of several calls, serves all of them, larger and smaller in turn."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_attn_shared import Group, beams  # noqa: E402
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


def test_one_workspace_for_layers_with_heads_of_their_own():
    """As a stack has it whose layers' heads differ: made for the widest."""
    say("attn_shared, one workspace")
    ws = w12.attn_shared_workspace(20, 8, 256, DEV)
    for d, f8 in ((256, False), (128, False), (64, True), (128, True), (256, True), (64, False)):
        x = Group(np.random.default_rng([85, d]), [beams(20, 640, 20, 1)], 8, 1, d, 16, f8)
        x.check(x.run(ws=ws))
