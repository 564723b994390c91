"""Beam search over the decode step: pages forked and copied, the shared tokens read once, the beams
that go on chosen and their states reordered.  Every beam's tokens are kept apart on the host as
well, and each attention is held against 64 bits over those."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from lossless_bit_weight_w12_amd.decode_step import DecodeAttention, DecodeStack  # noqa: E402
from oracle import fork_oracle as fo  # noqa: E402
from oracle import kv_oracle as ko  # noqa: E402
import w12_inputs as wi  # noqa: E402
from tests.gpu_util import say, to_dev  # noqa: E402
from tests.test_gpu_decode_attention import D, HID, HKV, HQ, NL, PAGE, VOCAB, build, i32  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def beams(g, fused, f8, prompts, per, n_pages, m, shared=True):
    """A stack of len(prompts) * per requests on a pool whose pages they may share."""
    stack, at, *_ = build(g, fused, f8, m)
    n = len(prompts) * per
    caches = [w12.kv_cache(n_pages, PAGE, HKV, D, F8 if f8 else torch.bfloat16,
                           *((0.0625, 0.0625) if f8 else ()), device=DEV) for _ in range(NL)]
    groups = (i32(np.arange(len(prompts) + 1) * per), i32(prompts)) if shared else None
    at = DecodeAttention(**{**at.__dict__, "pages": w12.page_table(n_pages, PAGE, n, 20, DEV, shared=True),
                            "caches": caches, "length": i32(np.zeros(n)), "req_off": i32(np.zeros(n + 1)),
                            "parent": i32(-np.ones(n)), "groups": groups})
    return DecodeStack(stack.layers, stack.head, m, fused_rms=fused, attention=at), at


def same_counts(at):
    table, held, refs = (t.cpu().numpy() for t in (at.pages.table, at.pages.held, at.pages.refs))
    n_pages = at.pages.n_pages
    used = np.concatenate([table[r, :h] for r, h in enumerate(held)])
    count = np.bincount(used, minlength=n_pages)
    assert np.array_equal(refs[:n_pages], count) and not refs[n_pages:3 * n_pages].any()
    assert int(at.pages.state[1]) == (count == 0).sum()


@pytest.mark.parametrize("fused,f8,shared", [(True, False, True), (False, True, True), (True, False, False)])
def test_beam_search_steps(fused, f8, shared):
    say("beam search, fused", fused, "f8", f8, "shared", shared)
    g = np.random.default_rng([91, fused, f8, shared])
    prompts, per, m = [75, 30], 3, 110          # (the second one's 64 shared tokens: none)
    n = len(prompts) * per
    stack, at = beams(g, fused, f8, prompts, per, 60, m, shared)
    embed = to_dev(wi.gaussian_bf16((VOCAB, HID), 1.0, g), torch).view(torch.bfloat16)
    grp_off, ends = i32(np.arange(len(prompts) + 1) * per), np.cumsum(prompts)
    hist = [[[np.zeros((0, HKV, D))] * 2 for _ in range(NL)] for _ in range(n)]   # [request][layer] k, v
    tokens = [[] for _ in range(n)]
    for step in range(9):
        first = step == 0
        if first:      # the prompts, as the rows of their first beams
            rows = [prompts[r // per] if r % per == 0 else 0 for r in range(n)]
            x0 = embed[torch.from_numpy(g.integers(0, VOCAB, m)).to(DEV)]
        else:
            rows = [1] * n
            x0 = embed[torch.cat([token.view(-1), token.new_zeros(m - n)]).long()]
        parent, length = at.parent.cpu().numpy(), at.length.cpu().numpy()
        off = np.concatenate([[0], np.cumsum(rows)])
        at.req_off.copy_(i32(off))
        _, _, acc, caps = stack.step(x0, i32(np.zeros(m)), capture=range(NL), req_ndraft=i32(np.zeros(n)))
        torch.cuda.synchronize()
        kv_len, slot = stack.kv_len.cpu().numpy(), stack.slot.cpu().numpy()
        assert kv_len.tolist() == [max(0, int(a)) + b for a, b in zip(length, rows)] and (acc == 0).all()
        hist = [[list(hist[p][li]) if p >= 0 else [np.zeros((0, HKV, D))] * 2 for li in range(NL)] for p in parent]
        for li in range(NL):
            c = at.caches[li]
            kc, vc = c.k.double().cpu().numpy() * c.k_scale, c.v.double().cpu().numpy() * c.v_scale
            pad = 20 * PAGE
            kk, vv = np.zeros((n, HKV, pad, D)), np.zeros((n, HKV, D, pad))   # one long page a request
            for r in range(n):
                have = [h[:length[r]] for h in hist[r][li]]
                at_rows = [divmod(int(s), PAGE) for s in slot[off[r]:off[r + 1]]]
                new = (np.array([kc[p, :, q] for p, q in at_rows]).reshape(-1, HKV, D),
                       np.array([vc[p, :, :, q] for p, q in at_rows]).reshape(-1, HKV, D))
                hist[r][li] = [np.concatenate(x) for x in zip(have, new)]
                kk[r, :, :kv_len[r]] = hist[r][li][0].transpose(1, 0, 2)
                vv[r, :, :, :kv_len[r]] = hist[r][li][1].transpose(1, 2, 0)
            turned = caps[li]["turned"].double().cpu().numpy().reshape(m, HQ, D)
            want, tol = ko.attention(turned, kk, vv, np.arange(n)[:, None], kv_len, off, D ** -0.5)
            got = caps[li]["in"]["o"][0].double().cpu().numpy().reshape(m, HQ, D)
            assert (np.abs(got - want)[:off[-1]] <= tol[:off[-1]]).all(), (step, li)
        # the beams that go on
        z, _ = w12.logits_f32(stack.h, stack.head)
        if first:
            z, scores, offs = z[torch.from_numpy(ends - 1).to(DEV)], torch.zeros(len(prompts), device=DEV), i32([0, 1, 2])
        else:
            z, offs = z[:n], grp_off
        par, token, new_scores = w12.beam_select(z, scores.view(-1), offs, per)
        want = fo.beam_select(z.double().cpu().numpy(), scores.double().cpu().numpy().reshape(-1), offs.cpu().numpy(), per)
        assert want[3] > 1e-6      # (no two scores closer than that decide)
        assert np.array_equal(par.cpu().numpy(), want[0]) and np.array_equal(token.cpu().numpy(), want[1])
        scores = new_scores
        par = par.view(-1) * per if first else par.view(-1)
        at.parent.copy_(par)
        at.length.copy_(stack.kv_len[par.long()])
        tokens = [tokens[p] + [t] for p, t in zip(par.tolist(), token.view(-1).tolist())]
        same_counts(at)
    assert len({tuple(t) for t in tokens}) == n
    assert any(tokens[r][0] == tokens[r + 1][0] for r in range(n - 1))     # some beam was continued twice
    # the end: everything is released
    at.length.zero_()
    at.parent.fill_(-1)
    at.req_off.zero_()
    stack.step(x0, i32(np.zeros(m)), req_ndraft=i32(np.zeros(n)))
    torch.cuda.synchronize()
    assert int(at.pages.state[1]) == at.pages.n_pages and not at.pages.refs[:at.pages.n_pages].any()


def test_beam_search_in_a_graph():
    """One whole step, the choice and the next step's tables with it, captured and replayed: the
    same bits as the eager steps of an equal stack."""
    say("beam search in a graph")
    prompts, per, m = [140, 70], 4, 8
    n, vocab = len(prompts) * per, VOCAB
    runs = []
    for _ in range(2):
        g = np.random.default_rng(92)
        stack, at = beams(g, True, False, prompts, per, 120, m)
        embed = to_dev(wi.gaussian_bf16((vocab, HID), 1.0, g), torch).view(torch.bfloat16)
        # prompts in hand: random keys and values in pages that every beam of a group holds
        for c in at.caches:
            c.k.copy_(to_dev(wi.gaussian_bf16((c.k.numel() // D, D), 1.0, g), torch).view(torch.bfloat16).view(c.k.shape))
            c.v.copy_(to_dev(wi.gaussian_bf16((c.v.numel() // D, D), 0.5, g), torch).view(torch.bfloat16).view(c.v.shape))
        rows = [prompts[r // per] if r % per == 0 else 0 for r in range(n)]
        w12.kv_fork(at.pages, at.parent, at.length, i32(np.concatenate([[0], np.cumsum(rows)])), sum(rows))
        at.length.copy_(i32([prompts[r // per] for r in range(n)]))
        at.parent.copy_(i32([r - r % per for r in range(n)]))
        at.req_off.copy_(i32(np.arange(n + 1)))
        scores = -torch.arange(n, dtype=torch.float32, device=DEV) / 8
        token = i32(g.integers(0, vocab, n)).view(-1, per)
        par, new_scores = torch.empty_like(token), torch.empty((len(prompts), per), device=DEV)
        draft, nd = i32(np.zeros(m)), i32(np.zeros(n))
        off = i32(np.arange(len(prompts) + 1) * per)

        def step(stack=stack, at=at, embed=embed, scores=scores, token=token, par=par, new_scores=new_scores, off=off):
            torch.index_select(embed, 0, token.view(-1), out=stack.h)
            stack.run()
            z, _ = w12.logits_f32(stack.h, stack.head)
            w12.beam_select(z, scores, off, per, par, token, new_scores)
            scores.copy_(new_scores.view(-1))
            at.parent.copy_(par.view(-1))
            torch.index_select(stack.kv_len, 0, par.view(-1), out=at.length)

        runs.append((stack, at, step, (scores, token, par), (draft, nd)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for stack, at, step, out, args in runs:
            stack.prepare(*args)
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            runs[0][2]()
        for i in range(20):
            graph.replay()
            torch.cuda.synchronize()
            runs[1][2]()
            torch.cuda.synchronize()
            (s0, a0, _, o0, _), (s1, a1, _, o1, _) = runs
            for x, y in zip((s0.h, s0.a, s0.kv_len, s0.slot, a0.pages.table, a0.pages.held, a0.pages.refs, a0.caches[1].k, *o0),
                            (s1.h, s1.a, s1.kv_len, s1.slot, a1.pages.table, a1.pages.held, a1.pages.refs, a1.caches[1].k, *o1)):
                assert torch.equal(x, y), i
            same_counts(a0)
        assert s0.kv_len.tolist() == [prompts[r // per] + 21 for r in range(n)]


def test_what_needs_counts():
    g = np.random.default_rng(93)
    stack, at, *_ = build(g, True, False, 11)
    with pytest.raises(ValueError, match="counts"):
        DecodeStack(stack.layers, stack.head, 11, attention=DecodeAttention(**{**at.__dict__, "parent": at.length}))
