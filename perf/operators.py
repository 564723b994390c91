"""The attention side of a decode step, case by case: bringing the block tables of a paged
key-value cache in line with the requests' lengths (kv_plan), the norm and rotation of the
query and key heads with the append to the cache (qk_rope), and the attention of the new
rows over the cache (attn_paged).

Every case exists in a plain form (elementary torch operations) and as the library's calls;
`own` chooses between them.
"""
import math

import torch

own = False

GOLD = 0.6180339887498949


# ---------------------------------------------------------------------------------- cases
def listed():
    """40 query and 8 key heads of 128 values is the decode step's q[5120, 5120] and
    k, v[1024, 5120]; 24 requests of 5 rows (4 drafted tokens and the bonus row) is the
    batched verification."""
    h = {"hq": 40, "hkv": 8, "d": 128}
    return [
        # one user, one new token, a page that still has room: the call's own latency
        {"name": "plan_one", "op": "plan", "n": 1, "lo": 300, "hi": 300, "rows": 1, "ragged": False, "page": 16, "spare": 64},
        # a verification step of 24 requests: every draft block may open a page, and a
        # rejected block gives it back
        {"name": "plan_verify", "op": "plan", "n": 24, "lo": 1, "hi": 8191, "rows": 5, "ragged": True, "page": 16, "spare": 512},
        # 64 prompts admitted at once and released: whole tables are filled and emptied
        {"name": "plan_admit", "op": "plan", "n": 64, "lo": 0, "hi": 0, "rows": 4095, "ragged": True, "page": 16, "spare": 17000},
        # one user, one new token
        {"name": "rope_one", "op": "rope", "m": 1, "per": 1, "rot": 128, "inter": False, "norm": True, "f8": False, "page": 16, "pad": 0, **h},
        # the batched verification into an 8-bit cache
        {"name": "rope_verify_f8", "op": "rope", "m": 120, "per": 5, "rot": 128, "inter": False, "norm": True, "f8": True, "page": 16, "pad": 0, **h},
        # four prompts' chunks of 2048 tokens
        {"name": "rope_prompt", "op": "rope", "m": 8192, "per": 2048, "rot": 128, "inter": False, "norm": True, "f8": False, "page": 16, "pad": 0, **h},
        # a small drafter's heads: half rotated, pairs side by side, no norms, a padded batch
        {"name": "rope_half", "op": "rope", "m": 77, "per": 3, "hq": 12, "hkv": 4, "d": 64, "rot": 32, "inter": True, "norm": False, "f8": False, "page": 32, "pad": 5},
        # one user, a short chat: latency
        {"name": "attn_one", "op": "attn", "n": 1, "lo": 17, "hi": 17, "rows": 1, "ragged": False, "f8": False, "page": 16, **h},
        # 24 requests, one new token each, contexts of 1 to 8191 tokens
        {"name": "attn_batch", "op": "attn", "n": 24, "lo": 1, "hi": 8191, "rows": 1, "ragged": False, "f8": False, "page": 16, **h},
        # the batched verification over an 8-bit cache
        {"name": "attn_verify_f8", "op": "attn", "n": 24, "lo": 100, "hi": 8000, "rows": 5, "ragged": False, "f8": True, "page": 16, **h},
        # one user with a long context
        {"name": "attn_long", "op": "attn", "n": 1, "lo": 131001, "hi": 131001, "rows": 1, "ragged": False, "f8": False, "page": 16, **h},
        # a drafter with one wide key head, ragged draft blocks, larger pages
        {"name": "attn_wide", "op": "attn", "n": 7, "lo": 1, "hi": 3001, "rows": 4, "ragged": True, "f8": False, "page": 64, "hq": 8, "hkv": 1, "d": 256},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        n = _log(rng, 1, 256)
        hi = _log(rng, 1, 8000)
        if rng.random() < 0.3:      # prompts admitted and released
            return {"op": op, "n": n, "lo": 0, "hi": 0, "rows": max(1, min(_log(rng, 16, 4000), 120000 // n)), "ragged": True,
                    "page": page, "spare": 120000 // page + n}
        return {"op": op, "n": n, "lo": rng.randint(0, hi), "hi": hi, "rows": _log(rng, 1, 16), "ragged": rng.random() < 0.5,
                "page": page, "spare": rng.choice([1 + n // 8, 4 * n])}
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    f8 = rng.random() < 0.4
    if op == "rope":
        m = _log(rng, 1, max(1, min(8192, 8192 * 40 * 128 // (hq * d))))
        return {"op": op, "m": m, "per": _log(rng, max(1, m // 128), min(m, 2048)), "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2]),
                "inter": rng.random() < 0.3, "norm": rng.random() < 0.7, "f8": f8, "page": page, "pad": rng.choice([0, 0, m // 10])}
    n = _log(rng, 1, 64)
    hi = _log(rng, 1, min(131000, 100000 * 8 * 128 // (n * hkv * d)))
    return {"op": op, "n": n, "lo": rng.randint(1, hi), "hi": hi, "rows": _log(rng, 1, 16), "ragged": rng.random() < 0.5,
            "f8": f8, "page": page, "hq": hq, "hkv": hkv, "d": d}


def _spread(case):
    """Per request its length, from lo to hi (the last one hi), and its number of new rows."""
    n, lo, hi, rows = case["n"], case["lo"], case["hi"], case["rows"]
    at = [((r + 1) * GOLD) % 1.0 for r in range(n - 1)] + [1.0]
    back = [((r + 1) * GOLD * GOLD) % 1.0 for r in range(n)]
    lens = [lo + int(round((hi - lo) * a)) for a in at]
    return lens, [1 + int((rows - 1) * b + 0.5) if case["ragged"] else rows for b in back]


def _offsets(rows):
    off = [0]
    for v in rows:
        off.append(off[-1] + v)
    return off


# --------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    st = {"case": case}
    {"plan": _prepare_plan, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](case, st, g, dev)
    return st


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _normal(shape, g, dev, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)


def _prepare_plan(case, st, g, dev):
    """The pool in the state that earlier steps left: each request holds the pages of its
    length, in no order, and the free ring starts anywhere."""
    lens, rows = _spread(case)
    n, page = case["n"], case["page"]
    held = [-(-v // page) for v in lens]
    cols = max(-(-(a + b) // page) for a, b in zip(lens, rows)) + 3
    used = sum(held)
    pages = used + case["spare"]
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    st["held"] = _ints(held, dev)
    col = torch.arange(cols, device=dev)
    first = torch.tensor(_offsets(held)[:-1], device=dev)
    mine = col[None, :] < st["held"][:, None]
    at = torch.where(mine, first[:, None] + col[None, :], 0)
    st["table"] = torch.where(mine, perm[at], -1).to(torch.int32).contiguous()
    head = int(torch.randint(0, pages, (1,), generator=g, device=dev).item())
    st["ring"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
    place = (head + torch.arange(case["spare"], device=dev)) % pages
    st["ring"][place] = perm[used:]
    st["state"] = _ints([head, case["spare"], 0, 0], dev)
    st["len"], st["off"] = _ints(lens, dev), _ints(_offsets(rows), dev)
    st["none"] = torch.zeros_like(st["off"])
    m = sum(rows)
    st["kv_len"], st["back"] = (torch.zeros(n, dtype=torch.int32, device=dev) for _ in range(2))
    st["pos"], st["slot"] = (torch.zeros(m, dtype=torch.int32, device=dev) for _ in range(2))
    st["empty"] = torch.zeros(0, dtype=torch.int32, device=dev)
    if own:
        import lossless_bit_weight_w12_amd as w12
        pt = w12.PageTable(page_size=page, table=st["table"], held=st["held"], ring=st["ring"], state=st["state"])
        st["calls"] = [w12.prepare_kv_plan(pt, st["len"], st["off"], st["kv_len"], st["pos"], st["slot"]),
                       w12.prepare_kv_plan(pt, st["len"], st["none"], st["back"], st["empty"], st["empty"])]


def _cache(pages, case, g, dev):
    dt = torch.float8_e4m3fn if case["f8"] else torch.bfloat16
    shape = (pages, case["hkv"], case["page"], case["d"])
    return _normal(shape, g, dev, dt), _normal((shape[0], shape[1], shape[3], shape[2]), g, dev, dt)


def _prepare_rope(case, st, g, dev):
    """Rows of requests at any positions; each request's tokens lie in consecutive places of
    its pages.  The last `pad` rows belong to no request."""
    m, per, page, d = case["m"], case["per"], case["page"], case["d"]
    n = -(-m // per)
    each = (page + per - 2) // page + 1
    st["q"], st["k"], st["v"] = (_normal((m, h, d), g, dev) for h in (case["hq"], case["hkv"], case["hkv"]))
    st["k"] *= 3.0
    st["kc"], st["vc"] = _cache(n * each, case, g, dev)
    row = torch.arange(m, device=dev)
    r, i = row // per, row % per
    start = torch.randint(0, 131072 - per, (n,), generator=g, device=dev)
    perm = torch.randperm(n * each, generator=g, device=dev)
    at = start % page
    slot = perm[r * each + (at[r] + i) // page] * page + (at[r] + i) % page
    real = row < m - case["pad"]
    st["pos"] = torch.where(real, start[r] + i, -1).to(torch.int32)
    st["slot"] = torch.where(real, slot, -1).to(torch.int32)
    st["freq"] = 1e6 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
    st["qn"], st["kn"] = ((_normal((d,), g, dev, scale=0.3) + 1.0) if case["norm"] else None for _ in range(2))
    st["scales"] = (0.03125, 0.0078125) if case["f8"] else (1.0, 1.0)
    st["qo"] = torch.zeros_like(st["q"])
    if own:
        import lossless_bit_weight_w12_amd as w12
        cache = w12.KvCache(st["kc"], st["vc"], *st["scales"])
        rope = w12.Rope(st["freq"], q_norm=st["qn"], k_norm=st["kn"], eps=1e-6, interleaved=case["inter"])
        st["calls"] = [w12.prepare_qk_rope(st["q"], st["k"], st["v"], cache, rope, st["pos"], st["slot"], st["qo"])]


def _prepare_attn(case, st, g, dev):
    """A pool somewhat larger than the requests need, their pages in no order, what earlier
    requests left in the free places; queries that make some tokens matter more."""
    lens, rows = _spread(case)
    page, d = case["page"], case["d"]
    need = [-(-v // page) for v in lens]
    cols = max(need) + 1
    pages = sum(need) + 5
    st["kc"], st["vc"] = _cache(pages, case, g, dev)
    st["scales"] = (0.5, 0.25) if case["f8"] else (1.0, 1.0)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    col = torch.arange(cols, device=dev)
    mine = col[None, :] < torch.tensor(need, device=dev)[:, None]
    at = torch.where(mine, torch.tensor(_offsets(need)[:-1], device=dev)[:, None] + col[None, :], 0)
    st["table"] = torch.where(mine, perm[at], -1).to(torch.int32).contiguous()
    st["kv_len"], st["off"] = _ints(lens, dev), _ints(_offsets(rows), dev)
    m = sum(rows)
    st["q"] = _normal((m, case["hq"], d), g, dev, scale=3.0)
    st["out"] = torch.zeros_like(st["q"])
    st["r"] = torch.tensor([r for r, c in enumerate(rows) for _ in range(c)], device=dev)
    st["i"] = torch.tensor([i for c in rows for i in range(c)], device=dev)
    st["most"], st["lens"], st["rows"] = max(rows), lens, rows
    if own:
        import lossless_bit_weight_w12_amd as w12
        cache = w12.KvCache(st["kc"], st["vc"], *st["scales"])
        st["calls"] = [w12.prepare_attn_paged(st["q"], cache, st["table"], st["kv_len"], st["off"], st["out"])]


# ------------------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        for call in st["calls"]:
            call()
    elif op == "plan":
        _plan(st, st["off"], st["kv_len"], st["pos"], st["slot"])
        _plan(st, st["none"], st["back"], st["empty"], st["empty"])
    elif op == "rope":
        _rope(st)
    else:
        _attn(st)
    if op == "plan":
        return {k: st[k] for k in ("kv_len", "back", "pos", "slot", "table", "held", "ring", "state")}
    if op == "rope":
        return {"q": st["qo"], "k_cache": st["kc"], "v_cache": st["vc"]}
    return {"out": st["out"]}


def _plan(st, off, kv_len, pos, slot):
    """The tables brought in line with len + new rows: pages past the need go to the end of
    the free ring, in request order, and pages that are missing come from its start; a
    request that finds too few, and every later one that needs any, stays as it is."""
    page, table, held, ring = st["case"]["page"], st["table"], st["held"].long(), st["ring"]
    size = ring.numel()
    head, count = st["state"][0].long(), st["state"][1].long()
    length, off = st["len"].long(), off.long()
    target = length + off[1:] - off[:-1]
    want = (target + page - 1) // page
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    gone = (col >= want[:, None]) & (col < held[:, None])
    order = gone.reshape(-1).cumsum(0).reshape(gone.shape) - 1
    ext = torch.cat([ring, ring[:1]])
    ext.scatter_(0, torch.where(gone, (head + count + order) % size, size).reshape(-1), table.reshape(-1))
    have = count + gone.sum()
    need = (want - held).clamp(min=0)
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= have)
    taken = torch.where(served & (need > 0), upto, 0).max()
    new = (col >= held[:, None]) & (col < want[:, None]) & served[:, None]
    rank = (upto - need)[:, None] + col - held[:, None]
    table.copy_(torch.where(new, ext[(head + rank) % size], table))
    ring.copy_(ext[:size])
    st["held"].copy_(torch.where(served, want, held))
    kv_len.copy_(torch.where(served, target, -1))
    st["state"][0].copy_((head + taken) % size)
    st["state"][1].copy_(have - taken)
    if pos.numel():
        row = torch.arange(pos.numel(), device=pos.device)
        r = torch.searchsorted(off[1:].contiguous(), row, right=True)
        p = length[r] + row - off[r]
        s = table[r, p // page].long() * page + p % page
        pos.copy_(torch.where(served[r], p, -1))
        slot.copy_(torch.where(served[r], s, -1))


def _rotated(x, weight, angle, case):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = case["rot"]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if case["inter"] else torch.cat([u, v], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rope(st):
    """Norm of each head, rotation by the position, and the append to the cache at the
    row's slot: keys as [page, head, place, value], values as [page, head, value, place]."""
    case = st["case"]
    real = case["m"] - case["pad"]
    angle = st["pos"][:real].double()[:, None] * st["freq"][None, :]
    st["qo"][:real] = _rotated(st["q"][:real], st["qn"], angle, case).bfloat16()
    k, v = _rotated(st["k"][:real], st["kn"], angle, case), st["v"][:real].float()
    kc, vc = st["kc"], st["vc"]
    if case["f8"]:
        k, v = ((x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8) for x, s in zip((k, v), st["scales"]))
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    slot = st["slot"][:real].long()
    kc[slot // case["page"], :, slot % case["page"]] = k
    vc[slot // case["page"], :, :, slot % case["page"]] = v


def _attn(st):
    """softmax(scale q K^T) V for every row over its request's tokens up to the row's own."""
    case = st["case"]
    n, most, d, hkv, page = case["n"], st["most"], case["d"], case["hkv"], case["page"]
    per = case["hq"] // hkv
    table = st["table"].long().clamp(min=0)
    size = table.shape[1] * page
    kv_len, off = st["kv_len"].long(), st["off"].long()
    rows = off[1:] - off[:-1]
    at = (off[:-1, None] + torch.arange(most, device=off.device)).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[at].reshape(n, most, hkv, per, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, most * per, d)
    k = st["kc"][table] if not case["f8"] else st["kc"].view(torch.uint8)[table].view(torch.float8_e4m3fn)
    k = k.float().permute(0, 2, 1, 3, 4).reshape(n, hkv, size, d)
    s = torch.matmul(q, k.transpose(-1, -2)) * (st["scales"][0] / math.sqrt(d))
    del k
    limit = (kv_len - rows)[:, None] + torch.arange(most, device=off.device) + 1
    seen = torch.arange(size, device=off.device)[None, None, :] < limit[:, :, None]
    seen = seen[:, None, :, None, :].expand(n, 1, most, per, size).reshape(n, 1, most * per, size)
    top = s.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top)).masked_fill(~seen, 0.0)
    del s, seen
    v = st["vc"][table] if not case["f8"] else st["vc"].view(torch.uint8)[table].view(torch.float8_e4m3fn)
    v = v.float().permute(0, 2, 1, 4, 3).reshape(n, hkv, size, d)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) * st["scales"][1] / torch.where(total == 0, 1.0, total)
    o = o.reshape(n, hkv, most, per, d).permute(0, 2, 1, 3, 4).reshape(n, most, case["hq"], d)
    st["out"].copy_(o[st["r"], st["i"]].bfloat16())


# ----------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        lens, rows = _spread(case)
        page, left = case["page"], case["spare"]
        new = 0
        for a, b in zip(lens, rows):
            need = -(-(a + b) // page) - -(-a // page)
            if need > left:
                break
            new, left = new + need, left - need
        # lengths, offsets, counts read and written twice; positions and slots written;
        # every page that changes hands read and written on each of its two ways
        return {"bytes": 2 * 4 * 5 * case["n"] + 8 * sum(rows) + 2 * 8 * new, "flops": 0}
    es = 1 if case["f8"] else 2
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        m = case["m"] - case["pad"]
        return {"bytes": m * d * (4 * hq + 2 * hkv * (2 + es)) + 8 * case["m"], "flops": m * d * (hq + hkv) * 7}
    lens, rows = _spread(case)
    m, pages = sum(rows), sum(-(-v // case["page"]) for v in lens)
    pairs = sum(max(0, a - b + i + 1) for a, b in zip(lens, rows) for i in range(b))
    return {"bytes": 2 * sum(lens) * hkv * d * es + 4 * m * hq * d + 4 * pages, "flops": 4 * pairs * hq * d}


# -------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return None
    return _exact_rope(case, st) if case["op"] == "rope" else _exact_attn(case, st)


def _exact_rope(case, st):
    rot, half, page = case["rot"], case["rot"] // 2, case["page"]
    live = st["pos"] >= 0
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=live.device),
                       st["pos"][live].double().outer(st["freq"]))[:, None, :]
    first = torch.arange(half, device=live.device) * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else half)

    def heads(x, w):
        x = x[live].double()
        if w is not None:
            x = w.double() * x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q = st["qo"].double()
    q[live] = heads(st["q"], st["qn"])
    k, v = st["kc"].double(), st["vc"].double()
    slot = st["slot"][live].long()
    kk, vv = heads(st["k"], st["kn"]) / st["scales"][0], st["v"][live].double() / st["scales"][1]
    if case["f8"]:
        kk, vv = kk.clamp(-448, 448), vv.clamp(-448, 448)
    k.transpose(1, 2)[slot // page, slot % page] = kk
    v.permute(0, 3, 1, 2)[slot // page, slot % page] = vv
    return {"q": q, "k_cache": k, "v_cache": v}


def _exact_attn(case, st):
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    q = st["q"].double()
    out = torch.zeros_like(q)
    a = 0
    for r, (length, rows) in enumerate(zip(st["lens"], st["rows"])):
        ids = st["table"][r, :-(-length // page)].long()
        for h in range(hkv):
            k = st["kc"][ids, h].double().reshape(-1, d)[:length] * st["scales"][0]
            v = st["vc"][ids, h].double().transpose(1, 2).reshape(-1, d)[:length] * st["scales"][1]
            for i in range(rows):
                end = length - rows + i + 1
                if end > 0:
                    mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                    w = torch.softmax(q[a + i, mine] @ k[:end].T / math.sqrt(d), -1)
                    out[a + i, mine] = w @ v[:end]
        a += rows
    return {"out": out}
