"""One weight-streaming decode step over a stack of W12 layers, built from the library's
entry points only (every GEMM, rescale and the verification run in its HIP kernels).

Dataflow per layer (no nonlinearity; rms(v) = v / sqrt(mean(v^2)) per row):  q, k, v =
h W_q^T, h W_k^T, h W_v^T;  o = rms(q) W_o^T;  gate, up = rms(o) W_gate^T, rms(o)
W_up^T;  down = rms(up) W_down^T;  h <- rms(down).  k, v and gate are computed and not
fed forward.  By default every rms(v) W^T runs as one RMS GEMM (w12_gemm_rms /
w12_gemm_group_rms: (v W^T) / rms(v), the division on the FP32 accumulators), so the
next layer's q, k, v read the previous down directly and only the final h is rescaled
on its own (w12_rms_rescale, rounded to BF16); with fused_rms=False every rescale is its
own launch and the GEMMs read the rounded rescaled rows.  After the last layer the LM
head verifies a draft block greedily on the final h (exact-logit argmax per row,
accepted-prefix length), which is the verification step of greedy speculative decoding
in "StargazerX0/SpecPilot" (hotrepo.ai digest), section "Results and verification"; W12
weights are read inside the GEMMs as in "SpecPilot: an agent doubled speculative
decoding speed, and the 10.87x needs context", section "The mechanisms it found".

With a DecodeAttention the step is a decoder's own: q and k are normed and turned per head and
appended with v to the layer's paged cache (w12_qk_rope), the rows of every request attend over
its cache (w12_attn_paged), and o reads that (o = attention W_o^T) in place of rms(q); the block
tables are brought in line with the requests' lengths once per step (w12_kv_plan).  The accepted
lengths of requests that the pool refused become -1 in an elementwise minimum of torch's.
"""
from __future__ import annotations

from dataclasses import dataclass

from . import w12

MATS = ("q", "k", "v", "o", "gate", "up", "down")


@dataclass
class DecodeAttention:
    """The attention of a DecodeStack: request r keeps length[r] tokens in the cache and its
    new rows are req_off[r] .. req_off[r+1]-1 of the batch (int32 device tensors, read anew by
    every step).  After a verification length += min(accepted + 1, the request's rows): its first
    row's token and the accepted ones stay, the rejected ones are overwritten by the next step,
    a request without rows stays as it is, and of a request whose last row had a draft too, that
    one is no row yet.  A request that the pool had too few pages for, or whose length is none,
    has accepted -1: it keeps its length and comes again, with the same rows, once pages are
    free."""
    n_heads: int
    pages: object      # w12.PageTable, shared by the layers
    caches: list       # w12.KvCache per layer
    ropes: list        # w12.Rope per layer
    length: object     # int32 [n_req]
    req_off: object    # int32 [n_req + 1]
    scale: float = None    # default head_dim ** -0.5


class DecodeStack:
    """Layers: a list of dicts name -> W12Tensor (names as in MATS); head: W12Tensor of
    the LM head.  All activation buffers are allocated once for m rows.  attention: a
    DecodeAttention, or None for the chain without it."""

    def __init__(self, layers, head, m: int, fused_rms: bool = True, attention=None):
        import torch
        if not layers:
            raise ValueError("empty layer stack")
        self.layers, self.head, self.m, self.fused_rms = layers, head, m, fused_rms
        self.attention = attention
        hid = layers[0]["q"].k
        dev = head.device
        bf = dict(dtype=torch.bfloat16, device=dev)
        out = {name: torch.empty((m, layers[0][name].n), **bf) for name in MATS}
        self.out = out
        self.a = torch.empty((m, layers[0]["o"].k), **bf)       # rms(q): input of o
        self.b = torch.empty((m, layers[0]["gate"].k), **bf)    # rms(o): input of gate/up
        self.c = torch.empty((m, layers[0]["down"].k), **bf)    # rms(up): input of down
        self.h = torch.empty((m, hid), **bf)
        self.argmax = torch.empty(m, dtype=torch.int32, device=dev)
        self.accepted = torch.empty(1, dtype=torch.int32, device=dev)
        if attention is not None:
            self._attention_buffers(attention, dev)

    def _attention_buffers(self, at, dev):
        import torch
        if len(at.caches) != len(self.layers) or len(at.ropes) != len(self.layers):
            raise ValueError("DecodeAttention: one cache and one rope per layer")
        for L, c in zip(self.layers, at.caches):
            n_pages, kv_heads, page_size, d = c.k.shape
            if page_size != at.pages.page_size or n_pages < at.pages.n_pages:
                raise ValueError("DecodeAttention: a cache does not hold the pool's pages")
            if (L["q"].n, L["k"].n, L["v"].n, L["o"].k) != (at.n_heads * d, kv_heads * d, kv_heads * d, at.n_heads * d):
                raise ValueError("DecodeAttention: the heads do not fit q, k, v and o")
        i32 = dict(dtype=torch.int32, device=dev)
        self.kv_len = torch.empty_like(at.length)
        self.pos, self.slot = torch.empty(self.m, **i32), torch.empty(self.m, **i32)
        # Rows of no request are left as they are by the attention: zeros here (so o is 0 and, with
        # rms(0) = 0 / 0, the rest of the row NaN), later what they held when they were a
        # request's.  What a step gives for them means nothing; no other row depends on it.
        self.turned, self.a = torch.zeros_like(self.out["q"]), torch.zeros_like(self.a)
        self.accepted = torch.empty(at.length.numel(), **i32)
        self.attn_ws = w12.attn_workspace(dev)
        # The fills above are through before the stack is handed out: its steps may run on any
        # stream, and a ticket that is cleared while a join is under way would end it early.
        torch.cuda.current_stream(dev).synchronize()

    def _attention_calls(self, li: int):
        """Norm, rotation and append of the layer's heads, then the attention into self.a."""
        at, o, c = self.attention, self.out, self.attention.caches[li]
        heads = lambda t: t.view(self.m, -1, c.k.shape[3])
        q = heads(self.turned)
        return [w12.prepare_qk_rope(heads(o["q"]), heads(o["k"]), heads(o["v"]), c, at.ropes[li], self.pos,
                                    self.slot, q),
                w12.prepare_attn_paged(q, c, at.pages.table, self.kv_len, at.req_off, heads(self.a), at.scale,
                                       self.attn_ws)]

    def _layer_calls(self, L, first: bool, li: int):
        calls = self._chain_calls(L, first)
        if self.attention is None:
            return calls
        # o reads the attention's output as it is, where the chain reads rms(q)
        after_o = 2 if self.fused_rms else 3
        return (calls[:1] + self._attention_calls(li) + [w12.prepare_gemm(self.a, L["o"], self.out["o"])] +
                calls[after_o:])

    def _chain_calls(self, L, first: bool):
        o = self.out
        if self.fused_rms:
            # q, k, v read h (first layer) or the previous down through its RMS; o, gate/up
            # and down read q, o and up through theirs
            qkv_in = self.h if first else o["down"]
            return [w12.prepare_gemm_group(qkv_in, [L["q"], L["k"], L["v"]],
                                           [o["q"], o["k"], o["v"]], rms=not first),
                    w12.prepare_gemm(o["q"], L["o"], o["o"], rms=True),
                    w12.prepare_gemm_group(o["o"], [L["gate"], L["up"]], [o["gate"], o["up"]],
                                           rms=True),
                    w12.prepare_gemm(o["up"], L["down"], o["down"], rms=True)]
        # q, k, v read h and gate, up read rms(o): one grouped launch each
        return [w12.prepare_gemm_group(self.h, [L["q"], L["k"], L["v"]], [o["q"], o["k"], o["v"]]),
                w12.prepare_rms(o["q"], self.a),
                w12.prepare_gemm(self.a, L["o"], o["o"]),
                w12.prepare_rms(o["o"], self.b),
                w12.prepare_gemm_group(self.b, [L["gate"], L["up"]], [o["gate"], o["up"]]),
                w12.prepare_rms(o["up"], self.c),
                w12.prepare_gemm(self.c, L["down"], o["down"]),
                w12.prepare_rms(o["down"], self.h)]

    def prepare(self, draft, req_ndraft=None):
        """Marshal every call of the step once (on the current stream): the layers read
        and write the stack's own buffers; the step starts from self.h.  With attention the
        verification is of its requests: draft int32 [m], req_ndraft int32 [n_req] (see
        w12.lmhead_verify_batched), accepted [n_req], -1 also for a request without pages."""
        self.calls = [self._layer_calls(L, li == 0, li) for li, L in enumerate(self.layers)]
        if self.fused_rms:   # the final h, rescaled on its own for the LM head
            self.calls[-1].append(w12.prepare_rms(self.out["down"], self.h))
        self.draft = draft
        at = self.attention
        if at is None:
            self.verify_call = w12.prepare_verify(self.h, self.head, draft, self.argmax, self.accepted)
            return
        if req_ndraft is None:
            raise ValueError("a step with attention verifies its requests: req_ndraft is missing")
        import torch
        self.stream = torch.cuda.current_stream(self.head.device)
        self.plan_call = w12.prepare_kv_plan(at.pages, at.length, at.req_off, self.kv_len, self.pos, self.slot)
        self.verify_call = w12.prepare_verify_batched(self.h, self.head, at.req_off, req_ndraft, draft,
                                                      self.argmax, self.accepted)

    def _verify(self):
        import torch
        self.verify_call()
        if self.attention is not None:
            # The verification knows nothing of the cache: a refused request's rows are NaN and
            # mismatch at once, accepted 0.  Its kv_len is -1, a served one's at least its rows
            # and so at least what it accepts: the smaller of the two says both.
            with torch.cuda.stream(self.stream):   # that of the prepared calls
                torch.minimum(self.accepted, self.kv_len.view(-1), out=self.accepted)

    def run(self):
        """One step from the current contents of self.h (after prepare)."""
        if self.attention is not None:
            self.plan_call()
        for calls in self.calls:
            for c in calls:
                c()
        self._verify()

    def step(self, h0, draft, capture=(), req_ndraft=None):
        """Run every layer from h0 [m, hidden] and verify `draft` on the final h.
        capture: layer indices whose GEMM inputs and outputs are cloned and returned as
        {layer: {"in": {name: (input, rms applied)}, name: output for name in MATS}}; with
        attention also "turned", q after norm and rotation.
        Returns (h, argmax, accepted, captured)."""
        self.prepare(draft, req_ndraft)
        caps = {}
        self.h.copy_(h0)
        o = self.out
        if self.attention is not None:
            self.plan_call()
        for li, calls in enumerate(self.calls):
            if li in capture:
                x_qkv = (self.h if li == 0 or not self.fused_rms else o["down"]).clone()
            for c in calls:
                c()
            if li in capture:
                if self.fused_rms:
                    rq = li > 0
                    ins = {"q": (x_qkv, rq), "k": (x_qkv, rq), "v": (x_qkv, rq),
                           "o": (o["q"].clone(), True), "gate": (o["o"].clone(), True),
                           "up": (o["o"].clone(), True), "down": (o["up"].clone(), True)}
                else:
                    ins = {"q": (x_qkv, False), "k": (x_qkv, False), "v": (x_qkv, False),
                           "o": (self.a.clone(), False), "gate": (self.b.clone(), False),
                           "up": (self.b.clone(), False), "down": (self.c.clone(), False)}
                if self.attention is not None:
                    ins["o"] = (self.a.clone(), False)
                caps[li] = {"in": ins, **{k: v.clone() for k, v in o.items()}}
                if self.attention is not None:
                    caps[li]["turned"] = self.turned.clone()
        self._verify()
        return self.h, self.argmax, self.accepted, caps

    def weight_bytes(self) -> int:
        return sum(t.nbytes() for L in self.layers for t in L.values()) + self.head.nbytes()

    def io_bytes(self) -> int:
        """Activation bytes the GEMMs, rescales and the verification read and write."""
        m = self.m
        total = 0      # (without the attention's: what it reads depends on the lengths)
        for L in self.layers:
            for name in MATS:
                t = L[name]
                total += 2 * m * (t.k + t.n)
            if not self.fused_rms:
                # rescales: read + write (with attention q has none)
                for name in ("q", "o", "up", "down")[self.attention is not None:]:
                    total += 2 * 2 * m * L[name].n
        if self.fused_rms:                                # the final h: read + write
            total += 2 * 2 * m * self.layers[-1]["down"].n
        t = self.head
        total += 2 * m * t.k + 2 * 16 * m * (t.n // 16) + 4 * m   # x, block records, argmax
        return total
