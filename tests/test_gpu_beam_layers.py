"""A decode step over counted pages whose layers' caches differ, in type and in pages behind the pool's:
the pages that beams may not share are copied in every layer."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from lossless_bit_weight_w12_amd.decode_step import DecodeAttention, DecodeStack  # noqa: E402
import w12_inputs as wi  # noqa: E402
from tests.gpu_util import say, to_dev  # noqa: E402
from tests.test_gpu_beam_steps import beams, same_counts  # noqa: E402
from tests.test_gpu_decode_attention import D, HID, HKV, NL, PAGE, i32  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("kinds", [[(F8, 0), (torch.bfloat16, 0)], [(torch.bfloat16, 0), (torch.bfloat16, 7)],
                                   [(torch.bfloat16, 3), (F8, 1)]])
def test_layers_whose_caches_differ(kinds):
    say("beams, caches that differ", kinds)
    assert NL >= 2
    g, n, m, pool = np.random.default_rng(94), 4, 40, 40
    stack, at = beams(g, True, False, [37], n, pool, m)
    bits = {F8: torch.uint8, torch.bfloat16: torch.int16}
    caches = []
    for li in range(NL):
        dt, more = kinds[li % 2]
        c = w12.kv_cache(pool + more, PAGE, HKV, D, dt, *((0.0625, 0.0625) if dt == F8 else ()), device=DEV)
        caches.append(c)
    at = DecodeAttention(**{**at.__dict__, "caches": caches})
    stack = DecodeStack(stack.layers, stack.head, m, attention=at)
    x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
    at.req_off.copy_(i32([0] + [37] * n))          # the prompt, as the first request's rows
    stack.step(x0, i32(np.zeros(m)), req_ndraft=i32(np.zeros(n)))
    assert stack.kv_len.tolist() == [37, 0, 0, 0]
    at.length.fill_(37)                            # all four continue it
    at.parent.zero_()
    at.req_off.copy_(i32(np.arange(n + 1)))
    stack.step(x0, i32(np.zeros(m)), req_ndraft=i32(np.zeros(n)))
    torch.cuda.synchronize()
    same_counts(at)
    copies, part = stack.copies.cpu().numpy(), 37 % PAGE
    assert copies[0].tolist() == [copies[0, 0]] * 2 + [0, 0] and (copies[1:, 2] == part).all()
    for c in at.caches:
        k, v = c.k.view(bits[c.k.dtype]), c.v.view(bits[c.v.dtype])
        for page, new in copies[1:, :2].tolist():
            assert page != new and k[page, :, :part].any()
            assert torch.equal(k[new, :, :part], k[page, :, :part]) and torch.equal(v[new, :, :, :part], v[page, :, :, :part])
