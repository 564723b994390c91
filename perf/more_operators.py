"""Several continuations of one prompt, case by case: block tables whose pages requests share
(kv_fork), the copies that this asks of the caches (kv_copy), a range of the pool cleared of
pages (kv_compact), the attention of requests that share their first tokens (attn_shared), and
the choice of the beams that go on (beam_select).

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
    k, v[1024, 5120]; 64 layers and a head of 151936 tokens are its others; 24 prompts are the
    batched verification's 24 requests."""
    h = {"hq": 40, "hkv": 8, "d": 128}
    return [
        # one prompt continued in four ways, and its beams released: latency
        {"name": "fork_one", "op": "fork", "grp": 1, "per": 4, "lo": 300, "hi": 300, "tail": 1, "rows": 1, "admit": True, "page": 16},
        # a step of beam search: half of the beams go on, the others become copies of them
        {"name": "fork_beams", "op": "fork", "grp": 24, "per": 4, "lo": 100, "hi": 8000, "tail": 200, "rows": 1, "admit": False, "page": 16},
        # the copied ends of 24 of 32 beams, all layers at once
        {"name": "copy_beams", "op": "copy", "n": 32, "skip": 4, "layers": 64, "f8": False, "page": 16, **h},
        # one copy in an 8-bit cache with large pages, few layers
        {"name": "copy_small_f8", "op": "copy", "n": 1, "skip": 0, "layers": 5, "f8": True, "page": 64, "hq": 12, "hkv": 3, "d": 64},
        # a small pool, half of it given up
        {"name": "compact_small", "op": "compact", "n": 5, "lo": 1, "hi": 700, "share": 1, "page": 16, "pages": 401, "clear": 200},
        # the pool of 256 requests of up to 8191 tokens, four to a prompt, a third given up
        {"name": "compact_pool", "op": "compact", "n": 256, "lo": 500, "hi": 8191, "share": 4, "page": 16, "pages": 120000, "clear": 40000},
        # one prompt, four beams: latency
        {"name": "attn_one", "op": "attn", "grp": 1, "per": 4, "lo": 300, "hi": 300, "tail": 40, "rows": 1, "f8": False, "page": 16, **h},
        # 24 prompts of up to 8000 tokens, four beams each
        {"name": "attn_beams", "op": "attn", "grp": 24, "per": 4, "lo": 100, "hi": 8000, "tail": 500, "rows": 1, "f8": False, "page": 16, **h},
        # 64 requests verify 5 rows each behind one long instruction, in an 8-bit cache
        {"name": "attn_verify_f8", "op": "attn", "grp": 1, "per": 64, "lo": 8000, "hi": 8000, "tail": 1000, "rows": 5, "f8": True, "page": 16, **h},
        # 16 questions to one long document
        {"name": "attn_long", "op": "attn", "grp": 1, "per": 16, "lo": 131001, "hi": 131001, "tail": 300, "rows": 1, "f8": False, "page": 16, **h},
        # four beams of one request
        {"name": "beam_one", "op": "beam", "grp": 1, "per": 4, "vocab": 151936, "k": 8, "f32": True},
        # four beams of 24 requests, logits in BF16
        {"name": "beam_batch", "op": "beam", "grp": 24, "per": 4, "vocab": 151936, "k": 8, "f32": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["fork", "copy", "compact", "attn", "attn", "beam"])
    page = rng.choice([16, 32, 64, 128, 256])
    d, hkv, f8 = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8]), rng.random() < 0.4
    if op == "fork":
        per, hi = _log(rng, 1, 16), _log(rng, 1, 8000)
        return {"op": op, "grp": _log(rng, 1, 256 // per), "per": per, "lo": rng.randint(1, hi), "hi": hi,
                "tail": _log(rng, 1, 300), "rows": _log(rng, 1, 16), "admit": rng.random() < 0.5, "page": page}
    if op == "copy":
        layers = rng.randint(1, 64)
        most = max(1, 64 * 16 * 8 * 128 * 24 * 2 // (layers * page * hkv * d * (1 if f8 else 2)))
        return {"op": op, "n": _log(rng, 1, min(256, most)), "skip": rng.choice([0, 2, 3]), "layers": layers,
                "f8": f8, "page": page, "hq": hkv, "hkv": hkv, "d": d}
    if op == "compact":
        pages = _log(rng, 64, 110000)
        share, hi = rng.choice([1, 1, 2, 4, 8]), _log(rng, 1, 8000)
        n = _log(rng, 1, max(1, min(256, pages // (2 * (hi // page + 1)) * share)))
        return {"op": op, "n": n, "lo": rng.randint(1, hi), "hi": hi, "share": share, "page": page,
                "pages": pages + 2 * (hi // page + 1), "clear": rng.randint(1, pages // 4)}
    if op == "beam":
        per, vocab = _log(rng, 1, 16), _log(rng, 1000, 160000)
        return {"op": op, "grp": _log(rng, 1, max(1, 96 // per)), "per": per, "vocab": vocab, "k": _log(rng, 1, 64),
                "f32": rng.random() < 0.5}
    per = _log(rng, 2, 64)
    grp = _log(rng, 1, max(1, 64 // per))
    rows = _log(rng, 1, 8)
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    hi = _log(rng, 1, min(100000, 1000000 * 8 * 128 // (grp * per * max(hkv, hq * rows / 40) * d)))
    return {"op": op, "grp": grp, "per": per, "lo": rng.randint(1, hi), "hi": hi, "tail": _log(rng, rows, max(rows, min(2000, hi))),
            "rows": rows, "f8": f8, "page": page, "hq": hq, "hkv": hkv, "d": d}


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, unevenly, the last one hi."""
    return [lo + int(round((hi - lo) * (((r + 1) * GOLD) % 1.0 if r + 1 < n else 1.0))) for r in range(n)]


def _offsets(rows):
    off = [0]
    for v in rows:
        off.append(off[-1] + v)
    return off


# --------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 29)
    st = {"case": case}
    {"fork": _prepare_fork, "copy": _prepare_copy, "compact": _prepare_compact, "attn": _prepare_attn,
     "beam": _prepare_beam}[case["op"]](case, st, g, dev)
    return st


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _normal(shape, g, dev, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)


def _tables(st, rows, n_pages, cols, g, dev):
    """Tables over a pool whose pages are held in no order: rows is a list of lists of page
    numbers, which are dealt out at random; the free ring starts anywhere."""
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    used = max((p for r in rows for p in r), default=-1) + 1
    flat = torch.full((len(rows), cols), -1, dtype=torch.int64)
    for r, pages in enumerate(rows):
        flat[r, :len(pages)] = torch.tensor(pages, dtype=torch.int64)
    flat = flat.to(dev)
    st["table"] = torch.where(flat >= 0, perm[flat.clamp(min=0)], -1).to(torch.int32).contiguous()
    st["held"] = _ints([len(r) for r in rows], dev)
    head = int(torch.randint(0, n_pages, (1,), generator=g, device=dev).item())
    st["ring"] = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
    st["ring"][(head + torch.arange(n_pages - used, device=dev)) % n_pages] = perm[used:]
    st["state"] = _ints([head, n_pages - used, 0, 0], dev)
    count = torch.bincount(st["table"][flat >= 0].long(), minlength=n_pages).to(torch.int32)
    if own:
        import lossless_bit_weight_w12_amd as w12
        st["refs"] = w12.page_refs(n_pages, dev)
        st["refs"][:n_pages] = count
        return w12.PageTable(page_size=st["case"]["page"], table=st["table"], held=st["held"], ring=st["ring"],
                             state=st["state"], refs=st["refs"])
    st["refs"] = count


def _prepare_fork(case, st, g, dev):
    """admit: rows behind those of the call hold the prompts; every request takes its prompt's
    pages and adds rows, then all are released.  Else a step: the requests of a prompt hold its full
    pages together and the rest each by itself, some go on and the others become copies of them."""
    grp, per, page, rows = case["grp"], case["per"], case["page"], case["rows"]
    n = grp * per
    prompt = _spread(grp, case["lo"], case["hi"])
    pick = torch.Generator()
    pick.manual_seed(int(torch.randint(0, 1 << 30, (1,), generator=g, device=dev).item()))
    held, nxt = [], 0

    def new(k):
        nonlocal nxt
        nxt += k
        return list(range(nxt - k, nxt))

    if case["admit"]:
        templates = [new(-(-p // page)) for p in prompt]
        held = [[] for _ in range(n)] + templates
        length = [prompt[i // per] for i in range(n)]
        parent = [n + i // per for i in range(n)]
    else:
        length, parent = [], []
        for p, more in zip(prompt, _spread(grp, 0, case["tail"] - 1)):
            both = new(p // page)
            alive = sorted(torch.randperm(per, generator=pick)[:(per + 1) // 2].tolist())
            for b in range(per):
                held.append(both + new(-(-(p + more) // page) - p // page))
                length.append(p + more)
                parent.append(len(held) - 1 - b + (b if b in alive else alive[b % len(alive)]))
    cols = max(-(-(a + rows) // page) for a in length) + 2
    spare = 2 * n * (-(-(max(1, rows) + page) // page) + 1) + 5
    pt = _tables(st, held, nxt + spare, cols, g, dev)
    st["length"], st["parent"] = _ints(length, dev), _ints(parent, dev)
    st["off"] = _ints([rows * i for i in range(n + 1)], dev)
    st["zero"], st["none"], st["no_rows"] = _ints([0] * n, dev), _ints([-1] * n, dev), _ints([0] * (n + 1), dev)
    st["kv_len"], st["back"] = _ints([0] * n, dev), _ints([0] * n, dev)
    st["pos"], st["slot"] = _ints([0] * (n * rows), dev), _ints([0] * (n * rows), dev)
    st["copies"], st["no_copies"] = (torch.zeros((n, 4), dtype=torch.int32, device=dev) for _ in range(2))
    st["empty"] = torch.zeros(0, dtype=torch.int32, device=dev)
    st["length_list"], st["parent_list"], st["held_list"] = length, parent, [len(h) for h in held]
    if own:
        import lossless_bit_weight_w12_amd as w12
        st["calls"] = [w12.prepare_kv_fork(pt, st["parent"], st["length"], st["off"], st["kv_len"], st["pos"], st["slot"], st["copies"])]
        if case["admit"]:
            st["calls"].append(w12.prepare_kv_fork(pt, st["none"], st["zero"], st["no_rows"], st["back"], st["empty"], st["empty"],
                                                   st["no_copies"]))


def _prepare_copy(case, st, g, dev):
    """Every `skip`-th entry (0: none) copies nothing (a beam that goes on); three of four that copy have a
    page of their own to read."""
    n, page, layers = case["n"], case["page"], case["layers"]
    pages = 2 * n + 3
    dt = torch.float8_e4m3fn if case["f8"] else torch.bfloat16
    shape = (layers, pages, case["hkv"], page, case["d"])
    st["k"], st["v"] = _normal(shape, g, dev, dt), _normal((*shape[:3], shape[4], shape[3]), g, dev, dt)
    perm = torch.randperm(pages, generator=g, device=dev)
    tokens = torch.randint(1, page, (n,), generator=g, device=dev)
    i = torch.arange(n, device=dev)
    on = (i % case["skip"] != case["skip"] - 1) if case["skip"] else torch.ones_like(i, dtype=torch.bool)
    src, dst = perm[i // 4 * 4 + (i % 4).clamp(max=2)], perm[n + i]
    copies = torch.stack([src, dst, tokens, torch.zeros_like(src)], 1)
    st["copies"] = torch.where(on[:, None], copies, torch.tensor([-1, -1, 0, 0], device=dev)).to(torch.int32).contiguous()
    if own:
        import lossless_bit_weight_w12_amd as w12
        s = (0.5, 0.25) if case["f8"] else (1.0, 1.0)
        st["calls"] = [w12.prepare_kv_copy([w12.KvCache(a, b, *s) for a, b in zip(st["k"], st["v"])], st["copies"])]


def _prepare_compact(case, st, g, dev):
    """`share` requests to a prompt, whose first half they hold together."""
    page, n = case["page"], case["n"]
    lens = _spread(n, case["lo"], case["hi"])
    rows, nxt, both = [], 0, []
    for r, v in enumerate(lens):
        need = -(-v // page)
        if r % case["share"] == 0:
            both = list(range(nxt, nxt + need // 2))
            nxt += len(both)
        mine = both[:need]
        rows.append(mine + list(range(nxt, nxt + need - len(mine))))
        nxt += need - len(mine)
    room = max(case["pages"] - case["clear"], nxt)
    pages = room + case["clear"]
    pt = _tables(st, rows, pages, max(len(r) for r in rows) + 3, g, dev)
    st["pages"], st["live"], st["rows_held"] = pages, nxt, sum(len(r) for r in rows)
    st["moves"], st["moves_back"] = (torch.zeros((case["clear"], 4), dtype=torch.int32, device=dev) for _ in range(2))
    st["moved"], st["moved_back"] = _ints([0], dev), _ints([0], dev)
    if own:
        import lossless_bit_weight_w12_amd as w12
        st["calls"] = [w12.prepare_kv_compact(pt, pages - case["clear"], st["moves"], st["moved"]),
                       w12.prepare_kv_compact(pt, 0, st["moves_back"], st["moved_back"])]


def _prepare_attn(case, st, g, dev):
    """Each prompt's full pages once, behind them pages of each request's own; queries that make
    some tokens matter more."""
    grp, per, page, d, rows = case["grp"], case["per"], case["page"], case["d"], case["rows"]
    n = grp * per
    prompt = _spread(grp, case["lo"], case["hi"])
    tail = _spread(n, rows, case["tail"])
    lens = [prompt[r // per] + tail[r] for r in range(n)]
    held, nxt, both = [], 0, []
    for r, v in enumerate(lens):
        if r % per == 0:
            both = list(range(nxt, nxt + prompt[r // per] // page))
            nxt += len(both)
        mine = -(-v // page) - len(both)
        held.append(both + list(range(nxt, nxt + mine)))
        nxt += mine
    _tables(st, held, nxt + 5, max(len(h) for h in held) + 1, g, dev)
    dt = torch.float8_e4m3fn if case["f8"] else torch.bfloat16
    shape = (nxt + 5, case["hkv"], page, d)
    st["kc"], st["vc"] = _normal(shape, g, dev, dt), _normal((shape[0], shape[1], d, page), g, dev, dt)
    st["scales"] = (0.5, 0.25) if case["f8"] else (1.0, 1.0)
    st["kv_len"], st["off"] = _ints(lens, dev), _ints([rows * i for i in range(n + 1)], dev)
    st["grp_off"] = _ints([per * i for i in range(grp + 1)], dev)
    st["grp_len"] = _ints([p // page * page for p in prompt], dev)
    st["q"] = _normal((n * rows, case["hq"], d), g, dev, scale=3.0)
    st["out"] = torch.zeros_like(st["q"])
    st["lens"] = lens
    if own:
        import lossless_bit_weight_w12_amd as w12
        cache = w12.KvCache(st["kc"], st["vc"], *st["scales"])
        st["calls"] = [w12.prepare_attn_shared(st["q"], cache, st["table"], st["kv_len"], st["off"], st["grp_off"],
                                               st["grp_len"], st["out"])]


def _prepare_beam(case, st, g, dev):
    """Logits of which a few stand out, and the sums of the log-probabilities so far."""
    n, vocab, k = case["grp"] * case["per"], case["vocab"], case["k"]
    x = torch.randn((n, vocab), generator=g, device=dev) * 2.5
    st["logits"] = (x if case["f32"] else x.bfloat16()).contiguous()
    st["scores"] = torch.randn((n,), generator=g, device=dev) * 2.0 - 30.0
    st["grp_off"] = _ints([case["per"] * i for i in range(case["grp"] + 1)], dev)
    st["parent"], st["token"] = (torch.zeros((case["grp"], k), dtype=torch.int32, device=dev) for _ in range(2))
    st["out"] = torch.zeros((case["grp"], k), dtype=torch.float32, device=dev)
    if own:
        import lossless_bit_weight_w12_amd as w12
        st["calls"] = [w12.prepare_beam_select(st["logits"], st["scores"], st["grp_off"], st["parent"], st["token"], st["out"])]


# ------------------------------------------------------------------------------ one pass
def run(st):
    op, case = st["case"]["op"], st["case"]
    if own:
        for call in st["calls"]:
            call()
    elif op == "fork":
        _fork(st, st["parent"], st["length"], st["off"], st["kv_len"], st["pos"], st["slot"], st["copies"])
        if case["admit"]:
            _fork(st, st["none"], st["zero"], st["no_rows"], st["back"], st["empty"], st["empty"], st["no_copies"])
    elif op == "copy":
        _copy(st)
    elif op == "compact":
        _compact(st, st["pages"] - case["clear"], st["moves"], st["moved"])
        _compact(st, 0, st["moves_back"], st["moved_back"])
    elif op == "attn":
        _attn(st)
    else:
        _beam(st)
    if op == "fork":
        out = {k: st[k] for k in ("kv_len", "back", "pos", "slot", "copies", "no_copies", "table", "held", "ring", "state")}
        return {**out, "refs": st["refs"][:st["ring"].numel()]}
    if op == "copy":
        return {"k": st["k"], "v": st["v"]}
    if op == "compact":
        out = {k: st[k] for k in ("moves", "moved", "moves_back", "moved_back", "table", "ring", "state")}
        return {**out, "refs": st["refs"][:st["pages"]]}
    if op == "attn":
        return {"out": st["out"]}
    return {"parent": st["parent"], "token": st["token"], "score": st["out"]}


def _fork(st, parent, length, off, kv_len, pos, slot, copies):
    """Request r becomes the first length[r] tokens of request parent[r] as it was (-1: none) and
    new rows.  Pages are shared; a request that will write into its last page takes a copy of it
    if another holds it too (of several that will write, the first keeps it).  Pages that nobody
    holds any longer go to the end of the free ring by column, then request; new ones come from
    what its start held before the call.  If they do not suffice nothing changes."""
    page, table, ring = st["case"]["page"], st["table"], st["ring"]
    dev, size, n = table.device, ring.numel(), parent.numel()
    head, count = st["state"][0].long(), st["state"][1].long()
    length, off, held, refs = length.long(), off.long(), st["held"].long(), st["refs"][:size].long()
    row, col = torch.arange(n, device=dev), torch.arange(table.shape[1], device=dev)[None, :]
    rows = off[1:] - off[:-1]
    keep, want = (length + page - 1) // page, (length + rows + page - 1) // page
    writes = (length % page > 0) & (rows > 0)
    old = table.long().clone()
    mine = old[parent.long().clamp(min=0)]
    had = col < held[:n, None]
    last = (keep - 1).clamp(min=0)
    tail = mine[row, last].clamp(min=0)
    claimed = (col < keep[:, None]) & ~(writes[:, None] & (col == last[:, None]))
    ext = torch.cat([refs, refs.new_zeros(1)])
    ext.scatter_add_(0, torch.where(had, old[:n], size).reshape(-1), ext.new_full((had.numel(),), -1))
    ext.scatter_add_(0, torch.where(claimed, mine, size).reshape(-1), ext.new_full((had.numel(),), 1))
    first = torch.full((size + 1,), n, dtype=torch.int64, device=dev)
    first.scatter_reduce_(0, torch.where(writes, tail, size), row, "amin")
    keeps = writes & (ext[tail] == 0) & (first[tail] == row)
    ext.scatter_add_(0, torch.where(keeps, tail, size), torch.ones_like(row))
    copied = writes & ~keeps
    need = want - keep + copied
    upto = need.cumsum(0)
    enough = upto[-1] <= count
    # given back: pages that nobody holds, at the first of those that held them
    place = (col * n + row[:, None])
    lowest = torch.full((size + 1,), col.numel() * n, dtype=torch.int64, device=dev)
    lowest.scatter_reduce_(0, torch.where(had, old[:n], size).reshape(-1), place.reshape(-1), "amin")
    gone = had & (ext[old[:n].clamp(min=0)] == 0) & (lowest[old[:n].clamp(min=0)] == place)
    order = gone.T.reshape(-1).cumsum(0).reshape(col.numel(), n).T - 1
    more = torch.cat([ring.long(), ring[:1].long()])
    more.scatter_(0, torch.where(gone, (head + count + order) % size, size).reshape(-1), old[:n].reshape(-1))
    # taken
    is_copy = copied[:, None] & (col == last[:, None])
    fresh = is_copy | ((col >= keep[:, None]) & (col < want[:, None]))
    rank = (upto - need)[:, None] + torch.where(is_copy, 0, col - keep[:, None] + copied[:, None])
    taken = ring.long()[(head + rank) % size]
    new = torch.where(fresh, taken, torch.where(col < keep[:, None], mine, old[:n]))
    ext.scatter_add_(0, torch.where(fresh, taken, size).reshape(-1), ext.new_full((had.numel(),), 1))
    table[:n] = torch.where(enough, new, old[:n]).to(torch.int32)
    ring.copy_(torch.where(enough, more[:size], ring.long()))
    st["held"][:n] = torch.where(enough, want, held[:n]).to(torch.int32)
    st["refs"][:size] = torch.where(enough, ext[:size], refs).to(torch.int32)
    st["state"][0] = torch.where(enough, (head + upto[-1]) % size, head).to(torch.int32)
    st["state"][1] = torch.where(enough, count - upto[-1] + gone.sum(), count).to(torch.int32)
    kv_len.copy_(torch.where(enough, length + rows, -1))
    one = torch.stack([torch.where(writes, tail, -1), torch.where(writes, new[row, last], -1),
                       torch.where(copied, length % page, 0), torch.zeros_like(row)], 1)
    none = torch.tensor([-1, -1, 0, 0], device=dev)
    copies.copy_(torch.where(enough, one, none))
    if pos.numel():
        i = torch.arange(pos.numel(), device=dev)
        r = torch.searchsorted(off[1:].contiguous(), i, right=True)
        p = length[r] + i - off[r]
        pos.copy_(torch.where(enough, p, -1))
        slot.copy_(torch.where(enough, new[r, p // page] * page + p % page, -1))


def _copy(st):
    """The first tokens places of a page, rounded up to 16, in every layer."""
    c = st["copies"].long()
    c = c[c[:, 2] > 0]
    k, v = (x.view(torch.uint8) if st["case"]["f8"] else x for x in (st["k"], st["v"]))
    here = torch.arange(st["case"]["page"], device=c.device)[None, :] < (c[:, 2:3] + 15) // 16 * 16
    for kl, vl in zip(k, v):
        kl[c[:, 1]] = torch.where(here[:, None, :, None], kl[c[:, 0]], kl[c[:, 1]])
        vl[c[:, 1]] = torch.where(here[:, None, None, :], vl[c[:, 0]], vl[c[:, 1]])


def _compact(st, start, moves, moved):
    """The i-th page in use of start .. start + len(moves) - 1 moves to the i-th free page
    outside, both in ascending order; the ring then holds the free pages outside, ascending, then
    the whole range."""
    size, dev, clear = st["pages"], st["table"].device, moves.shape[0]
    refs, state = st["refs"][:size].long(), st["state"]
    ids = torch.arange(size, device=dev)
    inside = (ids >= start) & (ids < start + clear)
    src, dst = inside & (refs > 0), ~inside & (refs == 0)
    enough = src.sum() <= dst.sum()
    to = torch.zeros(size + 1, dtype=torch.int64, device=dev)
    to.scatter_(0, torch.where(dst, dst.cumsum(0) - 1, size), ids)
    where = torch.where(src, to[(src.cumsum(0) - 1).clamp(min=0)], ids)
    col = torch.arange(st["table"].shape[1], device=dev)[None, :]
    t = st["table"].long()
    named = torch.where(col < st["held"].long()[:, None], where[t.clamp(min=0)], t)
    st["table"].copy_(torch.where(enough, named, t))
    after = torch.zeros(size + 1, dtype=torch.int64, device=dev).scatter_(0, torch.where(refs > 0, where, size), refs)[:size]
    free_out, free_in = (after == 0) & ~inside, (after == 0) & inside
    n_out = free_out.sum()
    ring = torch.cat([st["ring"].long(), st["ring"][:1].long()])
    ring.scatter_(0, torch.where(free_out, free_out.cumsum(0) - 1, size), ids)
    ring.scatter_(0, torch.where(free_in, n_out + free_in.cumsum(0) - 1, size), ids)
    st["ring"].copy_(torch.where(enough, ring[:size], st["ring"].long()))
    st["refs"][:size] = torch.where(enough, after, refs).to(torch.int32)
    state[0] = torch.where(enough, 0, state[0])
    state[1] = torch.where(enough, (after == 0).sum(), state[1]).to(torch.int32)
    go = (src & enough)[start:start + clear]
    one = torch.stack([ids, where, torch.full_like(ids, st["case"]["page"]), torch.zeros_like(ids)], 1)[start:start + clear]
    moves.copy_(torch.where(go[:, None], one, torch.tensor([-1, -1, 0, 0], device=dev)))
    moved.copy_(torch.where(enough, src.sum(), -1))


def _attn(st):
    """softmax(scale q K^T) V for every row over its request's tokens up to the row's own."""
    case = st["case"]
    n, rows, d, hkv, page = case["grp"] * case["per"], case["rows"], case["d"], case["hkv"], case["page"]
    group = case["hq"] // hkv
    kv_len, table = st["kv_len"].long(), st["table"].long().clamp(min=0)
    size = table.shape[1] * page
    byte = (lambda x: x.view(torch.uint8)) if case["f8"] else (lambda x: x)
    back = (lambda x: x.view(torch.float8_e4m3fn)) if case["f8"] else (lambda x: x)
    step = max(1, (1 << 31) // (size * hkv * d * 4))
    for a in range(0, n, step):
        b = min(n, a + step)
        q = st["q"][a * rows:b * rows].float().reshape(b - a, rows, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(b - a, hkv, rows * group, d)
        k = back(byte(st["kc"])[table[a:b]]).float().permute(0, 2, 1, 3, 4).reshape(b - a, hkv, size, d)
        s = torch.matmul(q, k.transpose(-1, -2)) * (st["scales"][0] / math.sqrt(d))
        del k
        limit = (kv_len[a:b] - rows)[:, None] + torch.arange(rows, device=q.device) + 1
        seen = torch.arange(size, device=q.device)[None, None, :] < limit[:, :, None]
        seen = seen[:, None, :, None, :].expand(b - a, 1, rows, group, size).reshape(b - a, 1, rows * group, size)
        s = s.masked_fill(~seen, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        del s, seen
        v = back(byte(st["vc"])[table[a:b]]).float().permute(0, 2, 1, 4, 3).reshape(b - a, hkv, size, d)
        o = torch.matmul(p, v) * st["scales"][1] / p.sum(-1, keepdim=True)
        st["out"][a * rows:b * rows] = o.reshape(b - a, hkv, rows, group, d).permute(0, 2, 1, 3, 4).reshape((b - a) * rows, case["hq"], d).bfloat16()


def _beam(st):
    """The k best of a group's rows and tokens by score + log softmax(logits), in 64 bits, lower
    rows and tokens first where equal."""
    case = st["case"]
    grp, per, k = case["grp"], case["per"], case["k"]
    x = st["logits"].double()
    top = x.amax(-1, keepdim=True)
    norm = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    val, tok = torch.sort(st["logits"], dim=-1, descending=True, stable=True)
    score = st["scores"].double()[:, None] + (val[:, :k].double() - norm)
    val, at = torch.sort(score.reshape(grp, per * k), dim=-1, descending=True, stable=True)
    at, first = at[:, :k], st["grp_off"][:-1].long()[:, None]
    st["parent"].copy_(first + at // k)
    st["token"].copy_(tok[:, :k].reshape(grp, per * k).gather(1, at))
    st["out"].copy_(val[:, :k])


# ----------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "fork":
        n = case["grp"] * case["per"]
        pages = [v // case["page"] for v in _spread(case["grp"], case["lo"], case["hi"])]
        # per request its parent, length, offset, held pages, new length and copy, per row its place; a
        # table row read and written for a request that becomes another's copy, page by page once
        moving = sum(pages) * case["per"]
        if not case["admit"]:
            moving = moving * (case["per"] // 2) // case["per"]
        return {"bytes": (44 * n + 8 * n * case["rows"] + 8 * moving) * (2 if case["admit"] else 1), "flops": 0}
    if case["op"] == "copy":
        n = case["n"] - (case["n"] // case["skip"] if case["skip"] else 0)
        places = (case["page"] + 16) // 2 if case["page"] > 16 else 16   # on the mean
        return {"bytes": 2 * 2 * n * case["layers"] * case["hkv"] * case["d"] * places * (1 if case["f8"] else 2) + 16 * case["n"], "flops": 0}
    if case["op"] == "compact":
        held = sum(-(-v // case["page"]) for v in _spread(case["n"], case["lo"], case["hi"]))
        # every count read and every table entry, the free ring and the list of moves written, twice
        return {"bytes": 2 * (4 * case["pages"] + 4 * held + 4 * case["pages"] + 16 * case["clear"]), "flops": 0}
    if case["op"] == "beam":
        n = case["grp"] * case["per"]
        return {"bytes": n * case["vocab"] * (4 if case["f32"] else 2) + 4 * n + 12 * case["grp"] * case["k"], "flops": 4 * n * case["vocab"]}
    es = 1 if case["f8"] else 2
    grp, per, rows, page = case["grp"], case["per"], case["rows"], case["page"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    prompt, tail = _spread(grp, case["lo"], case["hi"]), _spread(grp * per, rows, case["tail"])
    both = [p // page * page for p in prompt]
    tokens = sum(both) + sum(prompt[r // per] - both[r // per] + t for r, t in enumerate(tail))
    pairs = sum(rows * (prompt[r // per] + t) for r, t in enumerate(tail))
    return {"bytes": 2 * tokens * hkv * d * es + 4 * grp * per * rows * hq * d + 4 * tokens // page, "flops": 4 * pairs * hq * d}


# -------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    if case["op"] not in ("attn", "beam"):
        return None
    st = prepare(case, seed)
    return _exact_attn(case, st) if case["op"] == "attn" else _exact_beam(case, st)


def _exact_attn(case, st):
    hq, hkv, d, rows = case["hq"], case["hkv"], case["d"], case["rows"]
    per = hq // hkv
    q = st["q"].double()
    out = torch.zeros_like(q)
    for r, length in enumerate(st["lens"]):
        ids = st["table"][r, :-(-length // case["page"])].long()
        for h in range(hkv):
            k = st["kc"][ids, h].double().reshape(-1, d)[:length] * st["scales"][0]
            v = st["vc"][ids, h].double().transpose(1, 2).reshape(-1, d)[:length] * st["scales"][1]
            mine = slice(h * per, (h + 1) * per)
            for i in range(rows):
                end = length - rows + i + 1
                out[r * rows + i, mine] = torch.softmax(q[r * rows + i, mine] @ k[:end].T / math.sqrt(d), -1) @ v[:end]
    return {"out": out}


def _exact_beam(case, st):
    """The scores alone: which rows and tokens they are is whole numbers."""
    p = torch.log_softmax(st["logits"].double(), -1) + st["scores"].double()[:, None]
    each = p.reshape(case["grp"], -1)
    return {"parent": None, "token": None, "score": torch.topk(each, case["k"], dim=-1).values}
