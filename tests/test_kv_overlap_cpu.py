"""Overlapping arguments of the cache calls are refused by the binding, before any HIP call: a
launch would read what it writes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from lossless_bit_weight_w12_amd import w12 as B  # noqa: E402


class Device(torch.Tensor):
    """A host tensor that passes for a device one in the binding's checks."""

    @property
    def is_cuda(self):
        return True


def tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Device)


def bits(t):
    """The bytes a tensor holds, as a set of addresses."""
    at = np.zeros((), np.int64)
    for n, st in zip(t.shape, t.stride()):
        at = at[..., None] + np.arange(n) * st
    es = t.element_size()
    return set((t.data_ptr() + (at.reshape(-1)[:, None] * es + np.arange(es)).reshape(-1)).tolist())


def test_meet_against_every_byte():
    """Random row sets in one buffer: the answer of the arithmetic and that of the byte sets."""
    g = np.random.default_rng(81)
    buf = torch.zeros(400, dtype=torch.int16)
    seen = set()
    for _ in range(4000):
        ts = []
        for _ in range(2):
            m, heads, d = int(g.integers(1, 6)), int(g.integers(1, 3)), int(g.integers(1, 6))
            stride = int(g.integers(heads * d, 30)) if g.random() < 0.5 else 30
            span = (m - 1) * stride + heads * d
            ts.append(buf.as_strided((m, heads, d), (stride, d, 1), int(g.integers(0, min(400 - span, 60)))))
        meet = bool(bits(ts[0]) & bits(ts[1]))
        same = ts[0].stride(0) == ts[1].stride(0)
        seen.add((meet, same))
        assert B._meet(B._rows(ts[0]), B._rows(ts[1])) == meet and B._meet(B._rows(ts[1]), B._rows(ts[0])) == meet
    assert len(seen) == 4
    empty = B._rows(buf[:0])
    assert not B._meet(empty, B._rows(buf)) and not B._meet(B._rows(buf), empty)


@pytest.fixture
def no_stream(monkeypatch):
    monkeypatch.setattr(B, "_stream", lambda dev: None)


M, HQ, HKV, D, PAGE, PAGES = 6, 4, 2, 64, 16, 8
WIDE = (HQ + 2 * HKV) * D + 16


def attn(**kw):
    buf = tensor(2 * M * WIDE)
    ints = tensor(64, dtype=torch.int32)
    cache = w12.KvCache(tensor(PAGES, HKV, PAGE, D), tensor(PAGES, HKV, D, PAGE))
    a = dict(q=buf[:M * HQ * D].view(M, HQ, D), cache=cache, table=ints[:8].view(2, 4), kv_len=ints[8:10],
             req_off=ints[10:13], out=buf[M * HQ * D:2 * M * HQ * D].view(M, HQ, D), scale=None,
             ws=tensor(4096 + 64, dtype=torch.uint8))
    for k, v in kw.items():
        a[k] = v(a, buf) if callable(v) else v
    return B._attn_args(**a)


def heads(t, n=HQ):
    return t.unflatten(1, (n, D))


def test_attention_output_apart(no_stream):
    attn()
    wide = tensor(M + 1, WIDE)
    # columns of one buffer, and rows in turn, are apart
    attn(q=heads(wide[:M, :HQ * D]), out=heads(wide[:M, HQ * D:2 * HQ * D]))
    attn(q=heads(wide[0:6:2, :HQ * D]), out=heads(wide[1:6:2, :HQ * D]), req_off=tensor(3, dtype=torch.int32))
    q = heads(wide[:M, :HQ * D])
    for out in (q, heads(wide[1:, :HQ * D]),                        # itself, a row on
                heads(wide[:M, D:D + HQ * D]),                      # a head on
                heads(wide[:M, 8:8 + HQ * D]),                      # a few values on
                heads(wide[:M, WIDE - HQ * D:])):                   # its columns, past q's end: apart
        if out.data_ptr() == wide.data_ptr() + 2 * (WIDE - HQ * D):
            attn(q=q, out=out)
            continue
        with pytest.raises(ValueError, match="overlap"):
            attn(q=q, out=out)
    flat = tensor(3 * M * HQ * D)
    with pytest.raises(ValueError, match="overlap"):                # rows of another stride, interleaved
        attn(q=flat[:M * HQ * D].view(M, HQ, D), out=flat.as_strided((M, HQ, D), (2 * HQ * D, D, 1), HQ * D))
    last = lambda a, buf: a["cache"].k.view(-1)[-M * HQ * D:].view(M, HQ, D)
    with pytest.raises(ValueError, match="cache's k"):
        attn(out=last)
    with pytest.raises(ValueError, match="cache's v"):
        attn(out=lambda a, buf: a["cache"].v.view(-1)[:M * HQ * D].view(M, HQ, D))


def test_attention_workspace_apart(no_stream):
    for name, of in (("q", lambda a, buf: buf.view(torch.uint8)[64:]),
                     ("cache's v", lambda a, buf: a["cache"].v.view(-1).view(torch.uint8)),
                     ("kv_len", lambda a, buf: a["kv_len"].view(torch.uint8))):
        with pytest.raises(ValueError, match="overlap"):
            attn(ws=of)


def rope(q_out=None, cache=None, **kw):
    wide = tensor(M + 1, WIDE)
    ints = tensor(2 * M, dtype=torch.int32)
    a = dict(q=heads(wide[:M, :HQ * D]), k=heads(wide[:M, HQ * D:(HQ + HKV) * D], HKV),
             v=heads(wide[:M, (HQ + HKV) * D:(HQ + 2 * HKV) * D], HKV),
             cache=cache or w12.KvCache(tensor(PAGES, HKV, PAGE, D), tensor(PAGES, HKV, D, PAGE)),
             rope=w12.Rope(), pos=ints[:M], slot=ints[M:])
    a.update(kw)
    return B._rope_args(**a, q_out=q_out(a, wide) if q_out else tensor(M, HQ, D))


def test_rope_outputs_apart(no_stream):
    rope()
    rope(lambda a, wide: a["q"])                                    # in place
    for out in (lambda a, wide: heads(wide[1:, :HQ * D]),           # q a row on
                lambda a, wide: heads(wide[:M, D:D + HQ * D]),      # q a head on (and into k)
                lambda a, wide: heads(wide[:M, HQ * D:2 * HQ * D]),  # over k and v
                lambda a, wide: heads(wide[:M, HQ * D + 8:2 * HQ * D + 8]),
                lambda a, wide: a["cache"].k.view(-1)[:M * HQ * D].view(M, HQ, D)):
        with pytest.raises(ValueError, match="overlap"):
            rope(out)
    c = w12.KvCache(tensor(PAGES, HKV, 64, 64), tensor(PAGES, HKV, 64, 64))
    rope(cache=c)
    with pytest.raises(ValueError, match="overlap"):                # one buffer for k and v
        rope(cache=w12.KvCache(c.k, c.k))
    v = c.v.view(-1)[:M * HKV * D].view(M, HKV, D)
    with pytest.raises(ValueError, match="overlap"):                # rows that lie in the cache
        rope(cache=c, v=v)


def test_plan_arrays_apart(no_stream):
    """Results apart from each other, and the tables that a call updates apart from what it reads."""
    i = lambda n: tensor(n, dtype=torch.int32)
    pt = w12.PageTable(16, i(8).view(2, 4), i(2), i(8), i(4))
    a = dict(pt=pt, length=i(2), req_off=i(3), kv_len=i(2), pos=i(5), slot=i(5))
    call = lambda **kw: B._plan_args(**{**a, **kw})
    call()
    both = i(9)
    for kw in (dict(kv_len=a["length"]), dict(pos=both[:5], slot=both[4:]), dict(length=pt.held), dict(length=pt.state[:2]),
               dict(req_off=pt.ring[5:]), dict(length=pt.table[1, :2]), dict(slot=pt.ring[:5]),
               dict(pt=w12.PageTable(16, pt.table, pt.ring[6:], pt.ring, pt.state))):
        with pytest.raises(ValueError, match="overlaps"):
            call(**kw)
