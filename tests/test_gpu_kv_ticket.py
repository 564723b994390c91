"""kv_plan on a state whose ticket is not zero."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import say  # noqa: E402
from tests.test_gpu_kv import Pool, i32, offsets  # noqa: E402
import lossless_bit_weight_w12_amd as w12  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ticket", [1, 2, 7, 255, 256, -1, -2147483648, 123456789])
@pytest.mark.parametrize("n,max_pages,per", [(1, 4, 3), (24, 2000, 3), (24, 4000, 600), (300, 60, 3)])
def test_plan_refuses_a_ticket_that_is_not_zero(n, max_pages, per, ticket):
    """One workgroup or several: every request is refused and no table changes; with the ticket at zero
    again the same call is served."""
    say("plan, ticket", ticket, n, max_pages, per)
    p = Pool(2000, 16, n, max_pages, head=1990)
    p.step(np.full(n, 20), offsets([1] * n), n)
    p.pt.state[2] = ticket
    before = [t.clone() for t in (p.pt.table, p.pt.held, p.pt.ring, p.pt.state)]
    m = n * per
    got = w12.kv_plan(p.pt, i32(np.full(n, 33)), i32(offsets([per] * n)), m)
    for t in got:
        assert (t == -1).all()
    for a, b in zip(before, (p.pt.table, p.pt.held, p.pt.ring, p.pt.state)):
        assert torch.equal(a, b)
    p.pt.state[2] = 0
    p.step(np.full(n, 33), offsets([per] * n), m)
