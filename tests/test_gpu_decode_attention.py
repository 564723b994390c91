"""The decode step with attention (DecodeStack with a DecodeAttention): every operator of every
layer against its oracle on captured inputs, over steps with accepted and rejected drafts, and
the whole step captured into a graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from lossless_bit_weight_w12_amd.decode_step import DecodeAttention, DecodeStack, MATS  # noqa: E402
from oracle import kv_oracle as ko  # noqa: E402
from oracle import w12_oracle as o  # noqa: E402
import w12_inputs as wi  # noqa: E402
from tests.gpu_util import rms_reference, say, to_dev, to_host  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
HID, MLP, VOCAB, HQ, HKV, D, PAGE, NL = 256, 512, 1024, 4, 2, 64, 16, 2
ROWS = [3, 1, 5, 2]


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int32)).to(DEV)


def build(g, fused, f8, m):
    shapes = {"q": (HQ * D, HID), "k": (HKV * D, HID), "v": (HKV * D, HID), "o": (HID, HQ * D),
              "gate": (MLP, HID), "up": (MLP, HID), "down": (HID, MLP)}
    host = [{n: wi.gaussian_bf16(shapes[n], 0.06, g) for n in MATS} for _ in range(NL)]
    layers = [{n: w12.encode(to_dev(L[n], torch)) for n in MATS} for L in host]
    head = wi.gaussian_bf16((VOCAB, HID), 0.06, g)
    freq = 1e4 ** (-np.arange(D // 2) / (D // 2))
    norms = [[to_dev(wi.gaussian_bf16((1, D), 1.0, g)[0], torch).view(torch.bfloat16) for _ in range(2)]
             for _ in range(NL)]
    n = len(ROWS)
    at = DecodeAttention(
        n_heads=HQ, pages=w12.page_table(64, PAGE, n, 12, DEV),
        caches=[w12.kv_cache(64, PAGE, HKV, D, F8 if f8 else torch.bfloat16, *((0.0625, 0.0625) if f8 else ()),
                             device=DEV) for _ in range(NL)],
        ropes=[w12.Rope(torch.from_numpy(freq).to(DEV), *norms[li]) for li in range(NL)],
        length=i32(np.zeros(n)), req_off=i32(np.concatenate([[0], np.cumsum(ROWS)])))
    stack = DecodeStack(layers, w12.encode(to_dev(head, torch)), m, fused_rms=fused, attention=at)
    return stack, at, host, head, freq, norms


@pytest.mark.parametrize("fused,f8", [(True, False), (False, False), (True, True)])
def test_steps_with_attention(fused, f8):
    """Five steps of four requests (one padded row); every request's drafts are partly rejected."""
    say("decode step with attention, fused", fused, "f8", f8)
    g = np.random.default_rng([61, fused, f8])
    rows = sum(ROWS)
    m = rows + 1
    stack, at, host, head, freq, norms = build(g, fused, f8, m)
    nd = i32([r - 1 for r in ROWS])
    off = at.req_off.cpu().numpy()
    real = np.arange(rows)
    for step in range(5):
        x0 = wi.gaussian_bf16((m, HID), 1.0, g)
        draft = i32(g.integers(0, VOCAB, m))
        before = at.length.cpu().numpy().copy()
        h, am, acc, caps = stack.step(to_dev(x0, torch).view(torch.bfloat16), draft, capture=range(NL), req_ndraft=nd)
        torch.cuda.synchronize()
        kv_len = stack.kv_len.cpu().numpy()
        assert kv_len.tolist() == (before + ROWS).tolist()
        pos, slot = stack.pos.cpu().numpy(), stack.slot.cpu().numpy()
        assert pos[rows] == -1 and slot[rows] == -1
        for li in range(NL):
            cap = caps[li]
            for name in MATS:
                x_in, rms = cap["in"][name]
                assert rms == (fused and name in ("gate", "up", "down") or fused and li > 0 and name in "qkv")
                xh = to_host(x_in)[real]
                z, s = rms_reference(xh, host[li][name]) if rms else o.gemm_reference(xh, host[li][name])
                assert o.gemm_accept(to_host(cap[name])[real], z, s).all(), (step, li, name)
            heads = lambda t: t.double().cpu().numpy().reshape(m, -1, D)[real]
            y, mag = ko.rotated_heads(heads(cap["q"]), norms[li][0].double().cpu().numpy(), 1e-6, freq, pos[real], False)
            turned = heads(cap["turned"])
            assert (np.abs(turned - y) <= 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(y) + 2.0 ** -18 * mag).all(), (step, li)
            c = at.caches[li]
            kc, vc = c.k.double().cpu().numpy() * c.k_scale, c.v.double().cpu().numpy() * c.v_scale
            yk, mk = ko.rotated_heads(heads(cap["k"]), norms[li][1].double().cpu().numpy(), 1e-6, freq, pos[real], False)
            v = heads(cap["v"])
            rel, small = (2.0 ** -4, 2.0 ** -10 * 0.0625) if f8 else (2.0 ** -8, 0.0)
            for i in real:
                p, q = divmod(int(slot[i]), PAGE)
                assert (np.abs(kc[p, :, q] - yk[i]) <= rel * (1 + rel) * np.abs(yk[i]) + small + 2.0 ** -17 * mk[i]).all()
                assert (np.abs(vc[p, :, :, q] - v[i]) <= (rel if f8 else 0) * np.abs(v[i]) + small).all()
            want, tol = ko.attention(turned, kc, vc, at.pages.table.cpu().numpy(), kv_len, off, D ** -0.5)
            got = cap["in"]["o"][0].double().cpu().numpy().reshape(m, HQ, D)
            assert (np.abs(got[real] - want) <= tol).all(), (step, li)
            assert (got[rows] == 0).all()
        am_ref, _ = o.argmax_exact(to_host(h)[real], head)
        assert am.cpu().numpy()[real].tolist() == am_ref.tolist()
        acc_ref = [o.accepted_length(am_ref[off[r]:off[r + 1]], draft.cpu().numpy()[off[r]:off[r + 1] - 1])
                   for r in range(len(ROWS))]
        assert acc.cpu().numpy().tolist() == acc_ref
        # (drafts are random: half of what a real drafter would have right is kept by hand)
        at.length.copy_(i32(before + 1 + g.integers(0, 6, len(ROWS)) % ROWS))
    assert int(at.pages.held.sum()) + int(at.pages.state[1]) == at.pages.n_pages


def test_step_with_attention_in_a_graph():
    """The prepared step captured and replayed with new inputs and lengths, eager steps between:
    the replays give what the eager step gives."""
    g = np.random.default_rng(62)
    m = sum(ROWS)
    stack, at, *_ = build(g, True, False, m)
    nd, draft = i32([r - 1 for r in ROWS]), i32(g.integers(0, VOCAB, m))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        stack.prepare(draft, nd)
        stack.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            stack.run()
        for i in range(5):
            at.length.copy_(i32(g.integers(0, 150, len(ROWS))))
            x0 = to_dev(wi.gaussian_bf16((m, HID), 1.0, g), torch).view(torch.bfloat16)
            stack.h.copy_(x0)
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (stack.h, stack.argmax, stack.accepted, stack.kv_len, stack.slot, stack.a)]
            stack.h.copy_(x0)
            stack.run()      # the tables already fit
            torch.cuda.synchronize()
            for a, b in zip(got, (stack.h, stack.argmax, stack.accepted, stack.kv_len, stack.slot, stack.a)):
                assert torch.equal(a, b), i


def test_decode_attention_refusals():
    g = np.random.default_rng(63)
    stack, at, *_ = build(g, True, False, sum(ROWS))
    with pytest.raises(ValueError, match="req_ndraft"):
        stack.prepare(i32(np.zeros(sum(ROWS))))
    other = w12.kv_cache(64, 32, HKV, D, device=DEV)
    for change in (dict(caches=at.caches[:1]), dict(ropes=[]), dict(n_heads=8), dict(caches=[other] * NL),
                   dict(caches=[w12.kv_cache(63, PAGE, HKV, D, device=DEV)] * NL)):
        bad = DecodeAttention(**{**at.__dict__, **change})
        with pytest.raises(ValueError):
            DecodeStack(stack.layers, stack.head, sum(ROWS), attention=bad)
