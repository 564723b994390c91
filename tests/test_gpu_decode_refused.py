"""The decode step with attention when the pool runs dry: a refused request keeps its length, its
pages and its cache, and is served as if nothing had happened once pages are free."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from lossless_bit_weight_w12_amd.decode_step import DecodeAttention, DecodeStack  # noqa: E402
from oracle import kv_oracle as ko  # noqa: E402
import w12_inputs as wi  # noqa: E402
from tests.gpu_util import say, to_dev  # noqa: E402
from tests.test_gpu_decode_attention import D, HID, HKV, HQ, NL, PAGE, VOCAB, build, i32  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROWS = [3, 1, 5, 2]


def stack_of(g, fused, m, n_pages):
    """A stack as in the decode step's tests, its pool cut to n_pages."""
    stack, at, *rest = build(g, fused, False, m)
    at = DecodeAttention(**{**at.__dict__, "pages": w12.page_table(n_pages, PAGE, len(ROWS), 12, DEV)})
    return DecodeStack(stack.layers, stack.head, m, fused_rms=fused, attention=at), at


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("drafts", [True, False])
def test_refused_request_keeps_its_length(fused, drafts):
    """Request 2 crosses a page border while the pool is empty.  The step is run again after
    request 0 has ended: request 2's rows attend over exactly its own tokens."""
    say("refused request, fused", fused, "drafts", drafts)
    g = np.random.default_rng([71, fused, drafts])
    m = sum(ROWS)
    stack, at = stack_of(g, fused, m, 4)
    off = np.concatenate([[0], np.cumsum(ROWS)])
    nd = i32([r - 1 if drafts else 0 for r in ROWS])
    draft = i32(g.integers(0, VOCAB, m))

    def step(length):
        at.length.copy_(i32(length))
        x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
        _, am, acc, caps = stack.step(x0, draft, capture=range(NL), req_ndraft=nd)
        torch.cuda.synchronize()
        before = at.length.cpu().numpy().copy()
        at.length += acc + 1        # the rule of DecodeAttention
        return before, am.cpu().numpy(), acc.cpu().numpy(), caps

    _, _, acc, _ = step([0, 0, 0, 0])                 # a page each: the pool is empty
    assert (acc >= 0).all() and int(at.pages.state[1]) == 0
    before, _, acc, _ = step([1, 1, 10, 1])           # request 2 holds 10 tokens (5 of them rejected ones)
    assert (acc >= 0).all()
    kept = [[at.caches[li].k.clone(), at.caches[li].v.clone()] for li in range(NL)]
    before, am, acc, _ = step([2, 2, 12, 2])          # 12 + 5 tokens need a second page
    assert stack.kv_len.cpu().tolist() == [5, 3, -1, 4]
    assert acc[2] == -1 and (acc[[0, 1, 3]] >= 0).all()
    assert at.length.cpu().tolist() == [2 + acc[0] + 1, 2 + acc[1] + 1, 12, 2 + acc[3] + 1]
    assert (am[off[2]:off[3]] == -1).all()
    page = int(at.pages.table[2, 0])
    for li in range(NL):
        assert torch.equal(at.caches[li].k[page], kept[li][0][page]) and torch.equal(at.caches[li].v[page], kept[li][1][page])
    # request 0 ends and gives its page back; its entry of the batch has no rows any more
    rows = [0] + ROWS[1:]
    off2 = np.concatenate([[ROWS[0]], ROWS[0] + np.cumsum(rows)])
    at.req_off.copy_(i32(off2))
    nd[0] = 0
    before, am, acc, caps = step([0] + at.length.cpu().tolist()[1:])
    assert before[2] == 12 and stack.kv_len.cpu().tolist()[2] == 17 and acc[2] >= 0 and at.length[2] == 12 + acc[2] + 1
    real = np.arange(off2[0], off2[-1])
    for li in range(NL):
        c = at.caches[li]
        turned = caps[li]["turned"].double().cpu().numpy().reshape(m, HQ, D)
        want, tol = ko.attention(turned, c.k.double().cpu().numpy(), c.v.double().cpu().numpy(),
                                 at.pages.table.cpu().numpy(), stack.kv_len.cpu().numpy(), off2, D ** -0.5)
        got = caps[li]["in"]["o"][0].double().cpu().numpy().reshape(m, HQ, D)
        assert (np.abs(got[real] - want[real]) <= tol[real]).all(), li
    assert HKV == c.k.shape[1] and (am[real] >= 0).all()


def test_refused_request_in_a_graph():
    """The captured step gives the same -1, replay after replay, and 0 and more once it is served."""
    say("refused request in a graph")
    g = np.random.default_rng(72)
    m = sum(ROWS)
    stack, at = stack_of(g, True, m, 4)
    nd, draft = i32([r - 1 for r in ROWS]), i32(g.integers(0, VOCAB, m))
    x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        stack.prepare(draft, nd)
        stack.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            stack.run()
        for length, refused in (([0, 0, 0, 0], []), ([2, 2, 12, 2], [2]), ([2, 2, 11, 2], []), ([2, 16, 12, 2], [1, 2]),
                                ([16, 2, 3, -1], [0, 3])):
            at.length.copy_(i32(length))
            stack.h.copy_(x0)
            graph.replay()
            torch.cuda.synchronize()
            got = stack.accepted.cpu().numpy()
            assert [r for r in range(4) if got[r] < 0] == refused and (got[refused] == -1).all(), length
            stack.h.copy_(x0)
            stack.run()
            torch.cuda.synchronize()
            assert stack.accepted.cpu().numpy().tolist() == got.tolist()


def test_lengths_never_pass_what_was_appended():
    """length += min(accepted + 1, rows) with a request without rows, one without drafts, and one whose
    last row has a draft too, when every draft is right and when none is."""
    say("lengths after a step")
    g = np.random.default_rng(75)
    m = sum(ROWS)
    stack, at = stack_of(g, True, m, 40)
    rows = np.array([3, 0, 5, 2])
    nd = i32([2, 0, 5, 0])
    off = np.concatenate([[0], np.cumsum(rows)])
    at.req_off.copy_(i32(off))
    start = [20, 7, 33, 0]
    x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
    at.length.copy_(i32(start))
    am = stack.step(x0, i32(np.zeros(m)), req_ndraft=nd)[1].clone()
    for draft, want in ((am, [2, 0, 5, 0]), ((am + 1) % VOCAB, [0, 0, 0, 0])):
        at.length.copy_(i32(start))
        acc = stack.step(x0, draft, req_ndraft=nd)[2]      # (the same tokens to the same places)
        assert acc.cpu().tolist() == want
        at.length += torch.minimum(acc + 1, i32(rows))
        got = at.length.cpu().numpy()
        assert got.tolist() == [s + min(a + 1, r) for s, a, r in zip(start, want, rows)]
        assert (got <= stack.kv_len.cpu().numpy()).all()
    # a pool that holds nothing for request 3: refused and idle requests keep their lengths
    at.length.copy_(i32([20, 7, 33, 12 * PAGE]))
    acc = stack.step(x0, am, req_ndraft=nd)[2]
    at.length += torch.minimum(acc + 1, i32(rows))
    assert at.length.cpu().tolist() == [23, 7, 38, 12 * PAGE] and acc.cpu().tolist() == [2, 0, 5, -1]


def test_lengths_as_a_column():
    """Lengths of shape [n, 1] are taken as those of shape [n]."""
    g = np.random.default_rng(77)
    m = sum(ROWS)
    stack, at = stack_of(g, True, m, 4)
    nd, draft = i32([r - 1 for r in ROWS]), i32(g.integers(0, VOCAB, m))
    x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
    at.length.copy_(i32([2, 2, 12, 2]))
    want = stack.step(x0, draft, req_ndraft=nd)[2].cpu().tolist()
    column = DecodeAttention(**{**at.__dict__, "length": at.length.view(-1, 1)})
    other = DecodeStack(stack.layers, stack.head, m, attention=column)
    assert other.step(x0, draft, req_ndraft=nd)[2].cpu().tolist() == want
