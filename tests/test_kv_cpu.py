"""The attention side of a decode step without a GPU: pins of its oracle, and the refusals of
the C calls and of the binding, which come before any HIP call."""
import ctypes

import numpy as np
import pytest

import lossless_bit_weight_w12_amd as w12
from lossless_bit_weight_w12_amd import w12 as B
from oracle import kv_oracle as ko

FAKE = 0x10000          # non-null, aligned, never dereferenced (validation fails first)
NULL, SHAPE, RANGE, FORMAT, WS, ALIGN = -1, -2, -3, -4, -5, -7


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(w12.lib_path()):
        from lossless_bit_weight_w12_amd import build
        build.build(verbose=False)
    return w12.lib()


# ------------------------------------------------------------------------------ the oracle
def test_plan_oracle_worked_example():
    """Two requests, pages of 16: request 0 holds pages 4, 2 for 20 tokens and adds 13 (33
    tokens: a third page), request 1 shrinks from 3 pages (7, 0, 5) to 10 tokens."""
    table = np.array([[4, 2, -1, -1], [7, 0, 5, -1]], np.int32)
    held = np.array([2, 3], np.int32)
    ring = np.array([6, 9, 9, 9, 9, 9, 9, 1], np.int32)      # free: 1, then 6
    state = np.array([7, 2, 0, 0], np.int32)
    kv_len, pos, slot = ko.kv_plan(16, table, held, ring, state, [20, 10], [0, 13, 13], 14)
    assert kv_len.tolist() == [33, 10]
    assert pos.tolist() == list(range(20, 33)) + [-1]
    assert slot.tolist() == [2 * 16 + i for i in range(4, 16)] + [1 * 16] + [-1]
    assert table.tolist() == [[4, 2, 1, -1], [7, 0, 5, -1]] and held.tolist() == [3, 1]
    assert ring.tolist() == [6, 0, 5, 9, 9, 9, 9, 1] and state.tolist() == [0, 3, 0, 0]


def test_plan_oracle_refuses_in_order():
    """Three free pages: request 0 takes two, request 1 needs two and stops the rest, request
    2 needs none and is served, request 3 needs one and is not."""
    table = np.full((4, 4), -1, np.int32)
    table[2, 0] = 3
    held = np.array([0, 0, 1, 0], np.int32)
    ring = np.array([0, 1, 2, -1], np.int32)
    state = np.array([0, 3, 0, 0], np.int32)
    kv_len, pos, slot = ko.kv_plan(16, table, held, ring, state, [0, 0, 3, 0], [0, 17, 34, 35, 36], 36)
    assert kv_len.tolist() == [17, -1, 4, -1] and held.tolist() == [2, 0, 1, 0]
    assert state.tolist() == [2, 1, 0, 0]
    assert (pos[17:34] == -1).all() and slot[34] == 3 * 16 + 3 and slot[35] == -1


def test_plan_oracle_conserves_pages():
    g = np.random.default_rng(3)
    n, page, max_pages, n_pages = 9, 16, 12, 60
    table, held = np.full((n, max_pages), -1, np.int32), np.zeros(n, np.int32)
    ring, state = np.arange(n_pages, dtype=np.int32), np.array([5, n_pages, 0, 0], np.int32)
    for _ in range(60):
        rows = g.integers(0, 40, n)
        off = np.concatenate([[0], np.cumsum(rows)])
        ko.kv_plan(page, table, held, ring, state, g.integers(0, 180, n), off, int(off[-1]))
        free = [int(ring[(state[0] + i) % n_pages]) for i in range(state[1])]
        used = [int(table[r, i]) for r in range(n) for i in range(held[r])]
        assert sorted(free + used) == list(range(n_pages))


def test_rotation_oracle_is_a_rotation():
    """Lengths of pairs are kept, position 0 changes nothing, and scores depend on the
    distance of positions alone."""
    g = np.random.default_rng(1)
    freq = 1e4 ** (-np.arange(16) / 16)
    for inter in (False, True):
        x = g.standard_normal((2, 3, 40))
        y, _ = ko.rotated_heads(x, None, 0.0, freq, [0, 77], inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
        a, _ = ko.rotated_heads(x, None, 0.0, freq, [1000, 1013], inter)
        b, _ = ko.rotated_heads(x, None, 0.0, freq, [5, 18], inter)
        assert np.allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1), atol=1e-10)


def test_attention_oracle_against_torch():
    import torch
    g = np.random.default_rng(2)
    n_pages, hkv, page, d, hq = 9, 2, 16, 64, 6
    k, v = g.standard_normal((n_pages, hkv, page, d)), g.standard_normal((n_pages, hkv, d, page))
    table = np.array([[3, 1, 8, 0], [2, 7, -1, -1], [5, -1, -1, -1]], np.int32)
    kv_len, off = [50, 18, 0], [1, 4, 6, 7]
    q = g.standard_normal((8, hq, d))
    out, tol = ko.attention(q, k, v, table, kv_len, off, 0.125)
    assert np.isnan(out[[0, 7]]).all() and (out[6] == 0).all() and (tol[1:6] > 0).all()
    for r, (a, b) in enumerate([(1, 4), (4, 6)]):
        ids = table[r, :-(-kv_len[r] // page)]
        kk = k[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :kv_len[r]].repeat(hq // hkv, 0)
        vv = v[ids].transpose(1, 0, 3, 2).reshape(hkv, -1, d)[:, :kv_len[r]].repeat(hq // hkv, 0)
        mask = np.arange(kv_len[r])[None, :] <= kv_len[r] - (b - a) + np.arange(b - a)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[a:b].transpose(1, 0, 2)), torch.from_numpy(kk), torch.from_numpy(vv),
            attn_mask=torch.from_numpy(mask), scale=0.125).numpy().transpose(1, 0, 2)
        assert np.allclose(out[a:b], ref, atol=1e-12)


# ------------------------------------------------------------------------------- C refusals
def pages(**kw):
    p = B.W12Pages()
    p.n_pages, p.page_size, p.max_req, p.max_pages = 100, 16, 8, 20
    p.table = p.held = p.ring = p.state = FAKE
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def plan(L, p=None, length=FAKE, off=FAKE, n_req=4, m=3, kv_len=FAKE, pos=FAKE, slot=FAKE):
    return L.w12_kv_plan(ctypes.byref(p or pages()), length, off, n_req, m, kv_len, pos, slot, None)


def test_plan_refusals(L):
    assert L.w12_kv_plan(None, FAKE, FAKE, 1, 1, FAKE, FAKE, FAKE, None) == NULL
    for kw in (dict(length=None), dict(off=None), dict(kv_len=None), dict(pos=None), dict(slot=None)):
        assert plan(L, **kw) == NULL, kw
    for name in ("table", "held", "ring", "state"):
        assert plan(L, pages(**{name: None})) == NULL, name
        assert plan(L, pages(**{name: FAKE + 2})) == ALIGN, name
    for kw in (dict(page_size=0), dict(page_size=8), dict(page_size=48), dict(page_size=512),
               dict(n_pages=0), dict(n_pages=1 << 27), dict(max_pages=0), dict(max_pages=(1 << 26) + 1),
               dict(max_req=0), dict(max_req=4097)):
        assert plan(L, pages(**kw)) == SHAPE, kw
    assert plan(L, n_req=0) == RANGE and plan(L, n_req=9) == RANGE
    assert plan(L, m=(1 << 20) + 1) == RANGE
    for kw in (dict(length=FAKE + 1), dict(off=FAKE + 2), dict(kv_len=FAKE + 2), dict(pos=FAKE + 2),
               dict(slot=FAKE + 3)):
        assert plan(L, **kw) == ALIGN, kw


def kv(**kw):
    c = B.W12Kv()
    c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.dtype = 100, 16, 2, 128, B.KV_BF16
    c.k_scale = c.v_scale = 1.0
    c.k = c.v = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rope(**kw):
    r = B.W12Rope()
    r.q_norm = r.k_norm = r.inv_freq = FAKE
    r.rot_dim, r.interleaved, r.eps = 128, 0, 1e-6
    for k, v in kw.items():
        setattr(r, k, v)
    return r


BAD_CACHE = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(page_size=24), SHAPE), (dict(page_size=8), SHAPE),
             (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 27), SHAPE), (dict(head_dim=96), SHAPE),
             (dict(head_dim=512), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=3), SHAPE),
             (dict(dtype=2), FORMAT), (dict(k_scale=0.0, dtype=1), FORMAT),
             (dict(k_scale=float("nan"), dtype=1), FORMAT), (dict(v_scale=float("inf"), dtype=1), FORMAT),
             (dict(v_scale=-1.0, dtype=1), FORMAT), (dict(k_scale=2.0), FORMAT), (dict(k=FAKE + 8), ALIGN),
             (dict(v=FAKE + 4), ALIGN)]


def qk(L, c=None, r=None, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, m=3, heads=8, pos=FAKE,
       slot=FAKE, out=FAKE, os_=1024):
    return L.w12_qk_rope(q, qs, k, ks, v, vs, m, heads, ctypes.byref(c or kv()), ctypes.byref(r or rope()),
                         pos, slot, out, os_, None)


def test_qk_rope_refusals(L):
    assert L.w12_qk_rope(FAKE, 1024, FAKE, 256, FAKE, 256, 1, 8, None, ctypes.byref(rope()), FAKE, FAKE,
                         FAKE, 1024, None) == NULL
    assert L.w12_qk_rope(FAKE, 1024, FAKE, 256, FAKE, 256, 1, 8, ctypes.byref(kv()), None, FAKE, FAKE,
                         FAKE, 1024, None) == NULL
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(slot=None), dict(out=None)):
        assert qk(L, **kw) == NULL, kw
    for kw, st in BAD_CACHE:
        assert qk(L, kv(**kw)) == st, kw
    assert qk(L, r=rope(inv_freq=None)) == NULL
    for kw in (dict(rot_dim=8), dict(rot_dim=130), dict(rot_dim=144)):
        assert qk(L, r=rope(**kw)) == SHAPE, kw
    for kw in (dict(qs=1016), dict(qs=1028), dict(ks=248), dict(ks=260), dict(vs=0), dict(os_=1023),
               dict(os_=1 << 40), dict(heads=0), dict(heads=7), dict(heads=1026)):
        assert qk(L, **kw) == SHAPE, kw
    assert qk(L, m=(1 << 20) + 1) == RANGE
    assert qk(L, kv(n_kv_heads=64), heads=64, qs=8192, ks=8192, vs=8192, os_=8192, m=1 << 20) == RANGE
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(interleaved=2)):
        assert qk(L, r=rope(**kw)) == FORMAT, kw
    for kw in (dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(out=FAKE + 8), dict(pos=FAKE + 2),
               dict(slot=FAKE + 1)):
        assert qk(L, **kw) == ALIGN, kw
    for kw in (dict(q_norm=FAKE + 8), dict(k_norm=FAKE + 2), dict(inv_freq=FAKE + 4)):
        assert qk(L, r=rope(**kw)) == ALIGN, kw
    assert qk(L, m=0, q=None, k=None, v=None, pos=None, slot=None, out=None) == 0   # nothing to do


def attn(L, c=None, q=FAKE, qs=1024, m=3, heads=8, table=FAKE, max_pages=20, kv_len=FAKE, off=FAKE, n_req=2,
         scale=0.1, out=FAKE, os_=1024, ws=FAKE, wsb=w12.ATTN_WS_BYTES):
    return L.w12_attn_paged(q, qs, m, heads, ctypes.byref(c or kv()), table, max_pages, kv_len, off, n_req,
                            scale, out, os_, ws, wsb, None)


def test_attn_refusals(L):
    assert L.w12_attn_paged(FAKE, 1024, 1, 8, None, FAKE, 20, FAKE, FAKE, 1, 0.1, FAKE, 1024, FAKE,
                            w12.ATTN_WS_BYTES, None) == NULL
    for kw in (dict(q=None), dict(table=None), dict(kv_len=None), dict(off=None), dict(out=None), dict(ws=None)):
        assert attn(L, **kw) == NULL, kw
    for kw, st in BAD_CACHE:
        assert attn(L, kv(**kw)) == st, kw
    for kw in (dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(qs=1016), dict(qs=1030), dict(os_=0),
               dict(heads=0), dict(heads=9), dict(heads=1026)):
        assert attn(L, **kw) == SHAPE, kw
    for kw in (dict(n_req=0), dict(n_req=4097), dict(m=(1 << 20) + 1), dict(max_pages=1 << 26, m=128),
               dict(m=1 << 20, max_pages=8192)):
        assert attn(L, **kw) == RANGE, kw
    for s in (float("nan"), float("inf"), 3e38):
        assert attn(L, scale=s) == FORMAT, s
    assert attn(L, kv(dtype=1, k_scale=3e38), scale=2.0) == FORMAT   # the product overflows
    assert attn(L, wsb=w12.ATTN_WS_BYTES - 1) == WS
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 2), dict(ws=FAKE + 128), dict(table=FAKE + 2),
               dict(kv_len=FAKE + 2), dict(off=FAKE + 1)):
        assert attn(L, **kw) == ALIGN, kw
    assert attn(L, m=0, q=None, out=None) == 0


def test_constants_match_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w12.h")).read()

    def define(name):
        m = re.search(r"#define\s+%s\s+\(?(\d+)u?(?:\s*<<\s*(\d+))?\)?" % name, text)
        assert m, name
        return int(m.group(1)) << int(m.group(2) or 0)

    for name in ("KV_BF16", "KV_E4M3", "MAX_REQ", "MAX_KV_ROWS", "MAX_HEADS", "ATTN_WS_BYTES"):
        assert define("W12_" + name) == getattr(w12, name), name


# ------------------------------------------------------------------------- binding refusals
def test_binding_refuses_host_tensors():
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pt = w12.page_table(8, 16, 2, 4, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        w12.kv_plan(pt, i(2), i(3), 1)
    cache = w12.kv_cache(8, 16, 2, 64, device="cpu")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        w12.qk_rope(q, q[:, :2], q[:, :2], cache, w12.Rope(), i(1), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        w12.attn_paged(q, cache, i(2, 4), i(2), i(3))


def test_empty_cache_and_table():
    import torch
    c = w12.kv_cache(3, 32, 2, 64, dtype=torch.float8_e4m3fn, k_scale=0.5, device="cpu")
    assert tuple(c.k.shape) == (3, 2, 32, 64) and tuple(c.v.shape) == (3, 2, 64, 32)
    assert c.k.dtype == c.v.dtype == torch.float8_e4m3fn and c.k.view(torch.uint8).sum() == 0
    pt = w12.page_table(5, 16, 2, 3, device="cpu")
    assert pt.n_pages == 5 and pt.state.tolist() == [0, 5, 0, 0] and pt.ring.tolist() == list(range(5))
    assert tuple(pt.table.shape) == (2, 3) and pt.held.tolist() == [0, 0]
