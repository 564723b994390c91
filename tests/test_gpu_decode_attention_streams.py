"""A stack with attention built on one stream and run on another; and its byte count."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import w12_inputs as wi  # noqa: E402
from lossless_bit_weight_w12_amd.decode_step import DecodeStack  # noqa: E402
from tests.gpu_util import say, to_dev  # noqa: E402
from tests.test_gpu_decode_attention import D, HID, HQ, NL, ROWS, VOCAB, build, i32  # noqa: E402

pytestmark = pytest.mark.gpu


def test_stack_built_on_a_busy_stream():
    """The stream that the stack is built on is busy (a bounded spin): its zeroed workspace and buffers
    are in place all the same when the step runs on the default stream, with no wait by the caller."""
    say("stack built on a busy stream")
    g = np.random.default_rng(74)
    m = sum(ROWS)
    plain, at, *_ = build(g, True, False, m)
    nd, draft = i32([r - 1 for r in ROWS]), i32(g.integers(0, VOCAB, m))
    x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
    at.length.copy_(i32([150, 3, 97, 0]))
    torch.cuda.synchronize()
    want = [t.clone() for t in plain.step(x0, draft, req_ndraft=nd)[:3]] + [plain.a.clone()]
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            stack = DecodeStack(plain.layers, plain.head, m, attention=at)
        # (the tables already fit: the step writes the same tokens to the same places)
        got = [t.clone() for t in stack.step(x0, draft, req_ndraft=nd)[:3]] + [stack.a.clone()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_bytes_of_a_step_with_attention():
    """Without fused rescales a step with attention has one rescale less per layer, that of q: the
    attention reads its heads."""
    m = sum(ROWS)
    plain, at, *_ = build(np.random.default_rng(76), False, False, m)
    chain = DecodeStack(plain.layers, plain.head, m, fused_rms=False)
    assert chain.io_bytes() - plain.io_bytes() == NL * 2 * 2 * m * HQ * D
    fused = DecodeStack(plain.layers, plain.head, m)
    assert DecodeStack(plain.layers, plain.head, m, attention=at).io_bytes() == fused.io_bytes()


def test_run_from_another_stream():
    """A step prepared on one stream, which is busy (a bounded spin), and run while another is current:
    all of it, the accepted lengths of refused requests too, happens on the first."""
    say("run from another stream")
    g = np.random.default_rng(78)
    m = sum(ROWS)
    stack, at, *_ = build(g, True, False, m)
    nd, draft = i32([r - 1 for r in ROWS]), i32(g.integers(0, VOCAB, m))
    x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
    at.length.copy_(i32([20, -1, 7, 300]))      # no length, and one past the table
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        stack.prepare(draft, nd)
    for _ in range(3):
        stack.accepted.fill_(100)
        stack.h.copy_(x0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        stack.run()
        torch.cuda.synchronize()
        got = stack.accepted.cpu().tolist()
        assert got[1] == got[3] == -1 and 0 <= got[0] <= 2 and 0 <= got[2] <= 4
