"""Around the border between the two lines with heads of 256 values, which lies at 16 query rows, and the tiles of
32 behind it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_attn_shared import Group  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2, 15, 16, 17, 18, 31, 32, 33])
@pytest.mark.parametrize("d,f8", [(256, False), (256, True), (64, True), (128, True)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2)])
def test_numbers_of_query_rows(rows, d, f8, hq, hkv):
    say("attn_shared, query rows", rows, d, f8, hq, hkv)
    n = 2
    each = [rows // n + (i < rows % n) for i in range(n)]
    for shared in (64, 832):
        groups = [(shared, [shared + max(each) + 3 * i for i in range(n)], each)]
        Group(np.random.default_rng([67, rows, shared]), groups, hq, hkv, d, 16, f8).check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("heads", [15, 16, 17, 31, 32])
def test_rows_of_a_head_by_its_queries(heads, f8):
    """The same numbers from the query heads of one token each, beside a group of more rows."""
    say("attn_shared, query heads", heads, f8)
    groups = [(832, [840, 835], [1, 0]), (832, [836, 901], [1, 1]), (320, [330, 331, 332, 333], [1, 2, 1, 3])]
    Group(np.random.default_rng([68, heads]), groups, heads, 1, 256, 64, f8).check()
