"""Arguments of the calls for shared pages, shared attention and beams that overlap or do not fit are
refused by the binding, before any HIP call."""
import pytest

torch = pytest.importorskip("torch")
import lossless_bit_weight_w12_amd as w12  # noqa: E402
from lossless_bit_weight_w12_amd import w12 as B  # noqa: E402
from tests.test_kv_overlap_cpu import no_stream, tensor  # noqa: E402, F401

pytestmark = pytest.mark.usefixtures("no_stream")
M, HQ, HKV, D, PAGE, PAGES, REQ = 6, 4, 2, 64, 16, 8, 3


def ints(n):
    return tensor(n, dtype=torch.int32)


def pool(**kw):
    a = dict(page_size=PAGE, table=ints(4 * 4).view(4, 4), held=ints(4), ring=ints(PAGES), state=ints(4),
             refs=ints(5 * PAGES + 1024))
    return w12.PageTable(**{**a, **kw})


def fork(pt=None, **kw):
    a = dict(parent=ints(REQ), length=ints(REQ), req_off=ints(REQ + 1), kv_len=ints(REQ), pos=ints(M), slot=ints(M),
             copies=ints(4 * REQ).view(REQ, 4))
    return B._fork_args(pt or pool(), **{**a, **kw})


def test_fork_arguments():
    fork()
    fork(parent=None)
    x = ints(64)
    for kw in (dict(kv_len=x[:3], parent=x[2:5]), dict(pos=x[:6], slot=x[5:11]), dict(copies=x[:12].view(3, 4), length=x[11:14]),
               dict(kv_len=x[:3], req_off=x[2:6])):
        with pytest.raises(ValueError, match="overlap"):
            fork(**kw)
    with pytest.raises(ValueError, match="overlap"):                # the parents inside the table
        pt = pool()
        fork(pt, parent=pt.table.view(-1)[4:7])
    with pytest.raises(ValueError, match="overlap"):
        pt = pool()
        fork(pt, slot=pt.refs[100:106])
    with pytest.raises(ValueError, match="counts"):
        fork(pool(refs=None))
    for kw in (dict(parent=ints(2)), dict(kv_len=ints(4)), dict(copies=ints(12)), dict(copies=ints(12).view(4, 3)),
               dict(copies=ints(8).view(2, 4)), dict(req_off=ints(3)), dict(parent=torch.zeros(3, dtype=torch.int64)),
               dict(slot=ints(5)), dict(pos=ints(2 * M)[::2])):
        with pytest.raises(ValueError):
            fork(**kw)
    with pytest.raises(ValueError):
        fork(pool(refs=ints(5 * PAGES)))


def test_plan_leaves_shared_pages_alone():
    with pytest.raises(ValueError, match="share"):
        B._plan_args(pool(), ints(REQ), ints(REQ + 1), ints(REQ), ints(M), ints(M))


def cache(n=PAGES, page=PAGE, d=D):
    return w12.KvCache(tensor(n, HKV, page, d), tensor(n, HKV, d, page))


def test_copy_arguments():
    quads = ints(8).view(2, 4)
    c = cache()
    B._copy_args([c, cache()], quads)
    B._copy_args([c], quads[:0])
    for caches in ([c, c], [w12.KvCache(c.k, c.k.view(PAGES, HKV, D, PAGE))], []):
        with pytest.raises(ValueError):
            B._copy_args(caches, quads)
    inside = c.k.view(-1).view(torch.int32)[:8].view(2, 4)
    with pytest.raises(ValueError, match="overlap"):
        B._copy_args([c], inside)
    for bad in (ints(8), ints(6).view(2, 3), tensor(2, 4), ints(16).view(2, 8)[:, :4]):
        with pytest.raises(ValueError):
            B._copy_args([c], bad)


def test_compact_arguments():
    quads, moved = ints(16).view(4, 4), ints(1)
    B._compact_args(pool(), 4, quads, moved)
    for first in (-1, 5, PAGES):
        with pytest.raises(ValueError, match="leaves"):
            B._compact_args(pool(), first, quads, moved)
    with pytest.raises(ValueError, match="counts"):
        B._compact_args(pool(refs=None), 4, quads, moved)
    with pytest.raises(ValueError, match="overlap"):
        B._compact_args(pool(), 4, quads, quads.view(-1)[3:4])
    pt = pool()
    with pytest.raises(ValueError, match="overlap"):
        B._compact_args(pt, 4, quads, pt.held[:1])


def shared(**kw):
    a = dict(q=tensor(M, HQ, D), cache=cache(), table=ints(16).view(4, 4), kv_len=ints(REQ), req_off=ints(REQ + 1),
             grp_off=ints(3), grp_len=ints(2), out=tensor(M, HQ, D), scale=None,
             ws=tensor(w12.attn_shared_workspace(M, HQ, D, "cpu").numel(), dtype=torch.uint8))
    return B._shared_args(**{**a, **kw})


def test_shared_attention_arguments():
    shared()
    q, x, c = tensor(M, HQ, D), ints(64), cache()
    for kw in (dict(q=q, out=q), dict(cache=c, out=c.v.view(-1)[:M * HQ * D].view(M, HQ, D)),
               dict(cache=c, ws=c.k.view(-1).view(torch.uint8)), dict(q=q, ws=q.view(-1).view(torch.uint8)),
               dict(grp_len=x[:2], ws=x.view(torch.uint8)), dict(kv_len=x[3:6], ws=x.view(torch.uint8))):
        with pytest.raises(ValueError, match="overlap"):
            shared(**kw)
    for kw in (dict(grp_off=ints(2)), dict(grp_len=ints(3)), dict(table=ints(8).view(2, 4)), dict(table=ints(16)),
               dict(q=tensor(M, HQ, 2 * D)), dict(out=tensor(M, HQ + 1, D)), dict(q=tensor(M, HQ, D, dtype=torch.float32)),
               dict(ws=tensor(64)), dict(grp_len=torch.zeros(2, dtype=torch.int64)),
               dict(q=tensor((1 << 17) // HQ + 1, HQ, D), out=tensor((1 << 17) // HQ + 1, HQ, D))):
        with pytest.raises(ValueError):
            shared(**kw)


def beam(**kw):
    a = dict(logits=tensor(6, 40, dtype=torch.float32), scores=tensor(6, dtype=torch.float32), grp_off=ints(3),
             parent=ints(8).view(2, 4), token=ints(8).view(2, 4), score_out=tensor(2, 4, dtype=torch.float32),
             ws=tensor(1 << 20, dtype=torch.uint8))
    return B._beam_args(**{**a, **kw})


def test_beam_arguments():
    beam()
    wide, x, f = tensor(6, 64), ints(64), tensor(64, dtype=torch.float32)
    beam(logits=wide[:, 3:43])
    for kw in (dict(scores=f[:6], score_out=f[5:13].view(2, 4)), dict(parent=x[:8].view(2, 4), token=x[7:15].view(2, 4)),
               dict(grp_off=x[:3], token=x[2:10].view(2, 4)), dict(logits=f[:60].view(6, 10), ws=f.view(torch.uint8)),
               dict(logits=f.view(4, 16)[:, :10], scores=f[10:14], score_out=f[:8].view(2, 4))):
        with pytest.raises(ValueError, match="overlap"):
            beam(**kw)
    for kw in (dict(logits=wide.to(torch.float16)), dict(logits=wide.t()), dict(logits=tensor(6, 1).expand(6, 40)),
               dict(logits=tensor(1, 40).expand(6, 40)), dict(scores=tensor(6)), dict(scores=f[:5]), dict(token=x[:6]),
               dict(parent=x[:8]), dict(grp_off=x[:4]), dict(score_out=f[:7]), dict(ws=f)):
        with pytest.raises(ValueError):
            beam(**kw)
    with pytest.raises(ValueError, match="HIP"):
        beam(logits=torch.zeros(6, 40))
