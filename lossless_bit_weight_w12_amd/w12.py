"""Thin Python binding of libw12.so (ctypes).

Argument marshalling only: torch supplies device memory and the current HIP stream;
every step of encode, decode, GEMM and verification runs in the library's HIP kernels.
There is no CPU fallback: without the built library (or without a GPU) the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_float, c_int, c_int32, c_size_t, c_uint8, c_uint32, c_uint64, c_void_p
from dataclasses import dataclass

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libw12.so")
_LIB = None

OP_ENCODE, OP_DECODE, OP_GEMM, OP_GEMM_BF16, OP_VERIFY, OP_GEMM_GROUP, OP_VERIFY2, OP_GEMM_F8 = \
    0, 1, 2, 3, 4, 5, 6, 7
MAX_M = 128
MAX_GROUP = 4
KV_BF16, KV_E4M3 = 0, 1
MAX_REQ = 4096                 # W12_MAX_REQ: requests of one cache call
MAX_KV_ROWS = 1 << 20          # W12_MAX_KV_ROWS: rows of one cache call
MAX_HEADS = 1024               # W12_MAX_HEADS
MAX_LAYERS = 1024              # W12_MAX_LAYERS: caches of one kv_copy
MAX_COPIES = 1 << 22           # W12_MAX_COPIES
MAX_VOCAB = 1 << 21            # W12_MAX_VOCAB
MAX_BEAMS, MAX_BEAM_K = 64, 64  # W12_MAX_BEAMS: rows of a group, W12_MAX_BEAM_K: pairs chosen
LOGITS_BF16, LOGITS_F32 = 0, 1
MAX_SHARED_ROWS = 1 << 17      # W12_MAX_SHARED_ROWS: query rows (m * n_heads) of one attn_shared
ATTN_WS_BYTES = 36 << 20       # W12_ATTN_WS_BYTES
STATUS = {0: "W12_OK", -1: "W12_ERR_NULL", -2: "W12_ERR_SHAPE", -3: "W12_ERR_RANGE",
          -4: "W12_ERR_FORMAT", -5: "W12_ERR_WORKSPACE", -6: "W12_ERR_HIP", -7: "W12_ERR_ALIGN"}
EXPORTS = ("w12_tiles_bytes", "w12_workspace_bytes", "w12_workspace_init", "w12_encode_count",
           "w12_encode", "w12_decode", "w12_gemm", "w12_gemm_group", "w12_gemm_rms",
           "w12_gemm_group_rms", "w12_gemm_bf16", "w12_bf16_tile",
           "w12_gemm_bf16_tiled", "w12_lmhead_verify", "w12_lmhead_verify_batched",
           "w12_logits_f32",
           "w12_rms_rescale", "w12_status_str", "w12_version", "w12_gemm_noalloc", "w12_stream_read",
           "w12_screen_bytes", "w12_screen_encode", "w12_lmhead_verify2", "w12_lmhead_verify2_batched",
           "w12_screen_logits_f32", "w12_f8_tile", "w12_gemm_f8", "w12_gemm_f8_group",
           "w12_gemm_f8_rms", "w12_gemm_f8_group_rms", "w12_kv_plan", "w12_qk_rope",
           "w12_attn_paged", "w12_kv_fork", "w12_kv_copy", "w12_kv_compact",
           "w12_attn_shared_ws_bytes", "w12_attn_shared", "w12_beam_ws_bytes", "w12_beam_select")
NOALLOC_SCRATCH_BYTES = 32 << 20   # W12_NOALLOC_SCRATCH_BYTES
ENCODE_TOTAL_OFFSET = 2112   # W12_ENCODE_TOTAL_OFFSET: true escape count in an encode workspace


class W12Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({status_str(status)})")


class W12Desc(ctypes.Structure):
    _fields_ = [("n", c_uint64), ("k", c_uint64), ("n_esc", c_uint64),
                ("codebook", c_uint8 * 16), ("e_max", c_uint8), ("reserved", c_uint8 * 7),
                ("tiles", c_void_p), ("esc_off", c_void_p), ("esc", c_void_p)]


class W12Pages(ctypes.Structure):
    _fields_ = [("n_pages", c_uint32), ("page_size", c_uint32), ("max_req", c_uint32),
                ("max_pages", c_uint32), ("table", c_void_p), ("held", c_void_p),
                ("ring", c_void_p), ("state", c_void_p)]


class W12Kv(ctypes.Structure):
    _fields_ = [("n_pages", c_uint32), ("page_size", c_uint32), ("n_kv_heads", c_uint32),
                ("head_dim", c_uint32), ("dtype", c_uint32), ("k_scale", c_float),
                ("v_scale", c_float), ("k", c_void_p), ("v", c_void_p)]


class W12Rope(ctypes.Structure):
    _fields_ = [("q_norm", c_void_p), ("k_norm", c_void_p), ("inv_freq", c_void_p),
                ("rot_dim", c_uint32), ("interleaved", c_uint32), ("eps", c_float)]


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load libw12.so; raises if it has not been built (no silent fallback)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run "
                               "`python -m lossless_bit_weight_w12_amd.build` first")
        # torch ships its own HIP runtime (soname libamdhip64.so.7, the one libw12.so needs).
        # Loaded first, it is the runtime the library binds to; the other way round the
        # process would hold two HIP runtimes, and the library's launches on torch's
        # streams and memory would fail.
        import torch  # noqa: F401
        L = ctypes.CDLL(_LIB_PATH)
        L.w12_tiles_bytes.restype = c_size_t
        L.w12_tiles_bytes.argtypes = [c_uint64, c_uint64]
        L.w12_workspace_bytes.restype = c_size_t
        L.w12_workspace_bytes.argtypes = [c_int, c_uint32, c_uint64, c_uint64]
        L.w12_workspace_init.restype = c_int32
        L.w12_workspace_init.argtypes = [c_void_p, c_size_t, c_void_p]
        L.w12_encode_count.restype = c_int32
        L.w12_encode_count.argtypes = [c_void_p, c_uint64, c_uint64, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_size_t, c_void_p]
        L.w12_encode.restype = c_int32
        L.w12_encode.argtypes = [c_void_p, ctypes.POINTER(W12Desc), c_void_p, c_size_t, c_void_p]
        L.w12_decode.restype = c_int32
        L.w12_decode.argtypes = [ctypes.POINTER(W12Desc), c_void_p, c_void_p]
        L.w12_gemm.restype = c_int32
        L.w12_gemm.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p, c_void_p,
                               c_size_t, c_void_p]
        L.w12_gemm_group.restype = c_int32
        L.w12_gemm_group.argtypes = [c_void_p, c_uint32, c_void_p, c_uint32, c_void_p, c_void_p,
                                     c_size_t, c_void_p]
        L.w12_gemm_noalloc.restype = c_int32
        L.w12_gemm_noalloc.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p, c_void_p]
        L.w12_stream_read.restype = c_int32
        L.w12_stream_read.argtypes = [c_void_p, c_uint64, c_uint32, c_void_p, c_void_p]
        L.w12_gemm_rms.restype = c_int32
        L.w12_gemm_rms.argtypes = L.w12_gemm.argtypes
        L.w12_gemm_group_rms.restype = c_int32
        L.w12_gemm_group_rms.argtypes = L.w12_gemm_group.argtypes
        L.w12_gemm_bf16.restype = c_int32
        L.w12_gemm_bf16.argtypes = [c_void_p, c_uint32, c_void_p, c_uint64, c_uint64, c_void_p,
                                    c_void_p, c_size_t, c_void_p]
        L.w12_bf16_tile.restype = c_int32
        L.w12_bf16_tile.argtypes = [c_void_p, c_uint64, c_uint64, c_void_p, c_void_p]
        L.w12_gemm_bf16_tiled.restype = c_int32
        L.w12_gemm_bf16_tiled.argtypes = [c_void_p, c_uint32, c_void_p, c_uint64, c_uint64,
                                          c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_f8_tile.restype = c_int32
        L.w12_f8_tile.argtypes = [c_void_p, c_uint64, c_uint64, c_void_p, c_void_p]
        L.w12_gemm_f8.restype = c_int32
        L.w12_gemm_f8.argtypes = [c_void_p, c_uint32, c_void_p, c_void_p, c_uint64, c_uint64,
                                  c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_gemm_f8_group.restype = c_int32
        L.w12_gemm_f8_group.argtypes = [c_void_p, c_uint32, c_void_p, c_void_p, c_void_p, c_uint32,
                                        c_uint64, c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_gemm_f8_rms.restype = c_int32
        L.w12_gemm_f8_rms.argtypes = L.w12_gemm_f8.argtypes
        L.w12_gemm_f8_group_rms.restype = c_int32
        L.w12_gemm_f8_group_rms.argtypes = L.w12_gemm_f8_group.argtypes
        L.w12_lmhead_verify.restype = c_int32
        L.w12_lmhead_verify.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p,
                                        c_uint32, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_lmhead_verify_batched.restype = c_int32
        L.w12_lmhead_verify_batched.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p,
                                                c_void_p, c_uint32, c_void_p, c_void_p, c_void_p,
                                                c_void_p, c_size_t, c_void_p]
        L.w12_logits_f32.restype = c_int32
        L.w12_logits_f32.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p,
                                     c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_screen_bytes.restype = c_size_t
        L.w12_screen_bytes.argtypes = [c_uint64, c_uint64]
        L.w12_screen_encode.restype = c_int32
        L.w12_screen_encode.argtypes = [c_void_p, c_uint64, c_uint64, c_void_p, c_size_t, c_void_p]
        L.w12_lmhead_verify2.restype = c_int32
        L.w12_lmhead_verify2.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p,
                                         c_void_p, c_uint32, c_void_p, c_void_p, c_void_p,
                                         c_size_t, c_void_p]
        L.w12_lmhead_verify2_batched.restype = c_int32
        L.w12_lmhead_verify2_batched.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc),
                                                 c_void_p, c_void_p, c_void_p, c_uint32, c_void_p,
                                                 c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_screen_logits_f32.restype = c_int32
        L.w12_screen_logits_f32.argtypes = [c_void_p, c_uint32, ctypes.POINTER(W12Desc), c_void_p,
                                            c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.w12_rms_rescale.restype = c_int32
        L.w12_rms_rescale.argtypes = [c_void_p, c_uint32, c_uint64, c_void_p, c_void_p]
        L.w12_kv_plan.restype = c_int32
        L.w12_kv_plan.argtypes = [ctypes.POINTER(W12Pages), c_void_p, c_void_p, c_uint32, c_uint32,
                                  c_void_p, c_void_p, c_void_p, c_void_p]
        L.w12_qk_rope.restype = c_int32
        L.w12_qk_rope.argtypes = [c_void_p, c_uint64, c_void_p, c_uint64, c_void_p, c_uint64,
                                  c_uint32, c_uint32, ctypes.POINTER(W12Kv), ctypes.POINTER(W12Rope),
                                  c_void_p, c_void_p, c_void_p, c_uint64, c_void_p]
        L.w12_attn_paged.restype = c_int32
        L.w12_attn_paged.argtypes = [c_void_p, c_uint64, c_uint32, c_uint32, ctypes.POINTER(W12Kv),
                                     c_void_p, c_uint32, c_void_p, c_void_p, c_uint32, c_float,
                                     c_void_p, c_uint64, c_void_p, c_size_t, c_void_p]
        L.w12_kv_fork.restype = c_int32
        L.w12_kv_fork.argtypes = [ctypes.POINTER(W12Pages), c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_uint32, c_uint32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
        L.w12_kv_copy.restype = c_int32
        L.w12_kv_copy.argtypes = [ctypes.POINTER(W12Kv), c_uint32, c_void_p, c_uint32, c_void_p]
        L.w12_kv_compact.restype = c_int32
        L.w12_kv_compact.argtypes = [ctypes.POINTER(W12Pages), c_void_p, c_uint32, c_uint32, c_void_p,
                                     c_void_p, c_void_p]
        L.w12_attn_shared_ws_bytes.restype = c_size_t
        L.w12_attn_shared_ws_bytes.argtypes = [c_uint32, c_uint32, c_uint32]
        L.w12_attn_shared.restype = c_int32
        L.w12_attn_shared.argtypes = [c_void_p, c_uint64, c_uint32, c_uint32, ctypes.POINTER(W12Kv),
                                      c_void_p, c_uint32, c_void_p, c_void_p, c_uint32, c_void_p,
                                      c_void_p, c_uint32, c_float, c_void_p, c_uint64, c_void_p,
                                      c_size_t, c_void_p]
        L.w12_beam_ws_bytes.restype = c_size_t
        L.w12_beam_ws_bytes.argtypes = [c_uint32, c_uint32, c_uint32]
        L.w12_beam_select.restype = c_int32
        L.w12_beam_select.argtypes = [c_void_p, c_uint32, c_uint64, c_uint32, c_uint32, c_void_p,
                                      c_void_p, c_uint32, c_uint32, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_size_t, c_void_p]
        L.w12_status_str.restype = ctypes.c_char_p
        L.w12_status_str.argtypes = [c_int32]
        L.w12_version.restype = c_uint32
        L.w12_version.argtypes = []
        _LIB = L
    return _LIB


def status_str(s: int) -> str:
    return lib().w12_status_str(int(s)).decode()


def _check(fn: str, st: int):
    if st != 0:
        raise W12Error(fn, st)


def tiles_bytes(n: int, k: int) -> int:
    return int(lib().w12_tiles_bytes(n, k))


def workspace_bytes(op: int, m: int, n: int, k: int) -> int:
    return int(lib().w12_workspace_bytes(op, m, n, k))


# ----------------------------------------------------------------------------- torch glue
def _torch():
    import torch
    return torch


def _stream(dev):
    return c_void_p(_torch().cuda.current_stream(dev).cuda_stream)


def _ptr(t) -> c_void_p:
    return c_void_p(t.data_ptr())


def _as_bits(t):
    """View a BF16 / int16 / uint16 CUDA tensor as 16-bit storage (no copy)."""
    torch = _torch()
    if not t.is_cuda:
        raise ValueError("W12 calls need CUDA (HIP) tensors")
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise ValueError(f"expected BF16 bits, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t


_WS = {}


def workspace(nbytes: int, device, purpose: str = "gemm"):
    """A workspace of at least nbytes on `device`, cached per purpose ("gemm" for both
    GEMM entry points, "verify", "encode") so that calls of different kinds queued on
    one stream never share scratch memory; grown on demand."""
    torch = _torch()
    dev = torch.device(device)
    key = (dev.index if dev.index is not None else torch.cuda.current_device(), purpose)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _WS[key] = buf
    return buf


@dataclass
class W12Tensor:
    """A W12-encoded weight [n, k] resident on the GPU."""
    n: int
    k: int
    n_esc: int
    codebook: tuple
    e_max: int
    tiles: object      # torch.uint8 [tiles_bytes]
    esc_off: object    # torch.int32 [n/16 + 1]
    esc: object        # torch.int32 [max(n_esc, 1)]

    def desc(self) -> W12Desc:
        d = W12Desc()
        d.n, d.k, d.n_esc = self.n, self.k, self.n_esc
        for i, c in enumerate(self.codebook):
            d.codebook[i] = c
        d.e_max = self.e_max
        d.tiles = self.tiles.data_ptr()
        d.esc_off = self.esc_off.data_ptr()
        d.esc = self.esc.data_ptr()
        return d

    @property
    def device(self):
        return self.tiles.device

    def nbytes(self) -> int:
        """Bytes of the format: tiles + escapes + offsets + the 64-byte header."""
        return self.tiles.numel() + 4 * self.n_esc + 4 * (self.n // 16 + 1) + 64

    def bits_per_weight(self) -> float:
        return 8.0 * self.nbytes() / (self.n * self.k)


def encode(w) -> W12Tensor:
    """Encode BF16 weights w [n, k] (CUDA) to W12 on the same device."""
    torch = _torch()
    w = _as_bits(w)
    n, k = w.shape
    L = lib()
    dev = w.device
    ws = workspace(workspace_bytes(OP_ENCODE, 1, n, k), dev, "encode")
    cb = (c_uint8 * 16)()
    emax = c_uint8()
    nesc = c_uint64()
    s = _stream(dev)
    _check("w12_encode_count", L.w12_encode_count(_ptr(w), n, k, ctypes.byref(cb), ctypes.byref(emax),
                                                  ctypes.byref(nesc), _ptr(ws), ws.numel(), s))
    t = W12Tensor(n=n, k=k, n_esc=int(nesc.value), codebook=tuple(cb), e_max=int(emax.value),
                  tiles=torch.empty(tiles_bytes(n, k), dtype=torch.uint8, device=dev),
                  esc_off=torch.empty(n // 16 + 1, dtype=torch.int32, device=dev),
                  esc=torch.empty(max(int(nesc.value), 1), dtype=torch.int32, device=dev))
    d = t.desc()
    _check("w12_encode", L.w12_encode(_ptr(w), ctypes.byref(d), _ptr(ws), ws.numel(), s))
    return t


def decode(t: W12Tensor, out=None):
    torch = _torch()
    if out is None:
        out = torch.empty((t.n, t.k), dtype=torch.bfloat16, device=t.device)
    d = t.desc()
    _check("w12_decode", lib().w12_decode(ctypes.byref(d), _ptr(_as_bits(out)), _stream(t.device)))
    return out


@dataclass
class F8Tensor:
    """An FP8 weight [n, k] of an FP8 target resident on the GPU: E4M3 codes in the GEMM's
    2 KB tiles (w12_f8_tile) and FP32 scales per 128 x 128 block [ceil(n/128), k/128]."""
    n: int
    k: int
    tiles: object      # torch.uint8 [n*k]
    scale: object      # torch.float32 [ceil(n/128), k/128]

    def nbytes(self) -> int:
        return self.tiles.numel() + 4 * self.scale.numel()


def f8_encode(q, scale) -> F8Tensor:
    """F8Tensor of row-major E4M3 codes q [n, k] (uint8, CUDA) and their block scales."""
    torch = _torch()
    n, k = q.shape
    if scale.dtype != torch.float32 or tuple(scale.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("f8_encode: scale must be float32 [ceil(n/128), k/128]")
    return F8Tensor(n, k, f8_tile(q), scale.contiguous())


def gemm(x, t, out=None, rms: bool = False):
    """y = x . W^T, x BF16 [m, k] (m <= MAX_M), y BF16 [m, n].  rms: each output row divided
    by the RMS of its x row (w12_gemm_rms).  A GEMM is routed by its weight's format: a
    W12Tensor to w12_gemm, an F8Tensor (the weight of an FP8 target) to w12_gemm_f8 (FP8 GEMM
    routing, review page "The mechanisms it found")."""
    torch = _torch()
    if isinstance(t, F8Tensor):
        return gemm_f8(x, t.tiles, t.scale, t.n, t.k, out, rms=rms)
    x = _as_bits(x)
    m = x.shape[0]
    if x.shape[1] != t.k:
        raise ValueError(f"x has {x.shape[1]} columns, W has k = {t.k}")
    if out is None:
        out = torch.empty((m, t.n), dtype=torch.bfloat16, device=x.device)
    ws = workspace(max(workspace_bytes(OP_GEMM, m, t.n, t.k), 256), x.device)
    d = t.desc()
    fn = "w12_gemm_rms" if rms else "w12_gemm"
    _check(fn, getattr(lib(), fn)(_ptr(x), m, ctypes.byref(d), _ptr(_as_bits(out)), _ptr(ws),
                                  ws.numel(), _stream(x.device)))
    return out


def gemm_noalloc(x, t: W12Tensor, out=None):
    """y = x . W^T through w12_gemm_noalloc: the library's own fixed scratch array instead
    of a workspace (for callers that cannot allocate; `out` must then be given)."""
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    if x.shape[1] != t.k:
        raise ValueError(f"x has {x.shape[1]} columns, W has k = {t.k}")
    if out is None:
        out = torch.empty((m, t.n), dtype=torch.bfloat16, device=x.device)
    d = t.desc()
    _check("w12_gemm_noalloc", lib().w12_gemm_noalloc(_ptr(x), m, ctypes.byref(d), _ptr(_as_bits(out)),
                                                      _stream(x.device)))
    return out


def stream_read(buf, offset: int, nbytes: int, workgroups: int, sink):
    """The streaming-read probe (w12_stream_read) over bytes [offset, offset + nbytes) of the
    uint8 device tensor buf; sink: int32 device tensor of at least 4 * workgroups."""
    if offset < 0 or offset + nbytes > buf.numel() or sink.numel() < 4 * workgroups:
        raise ValueError("stream_read: range outside buf, or sink too small")
    _check("w12_stream_read", lib().w12_stream_read(c_void_p(buf.data_ptr() + offset), nbytes,
                                                    workgroups, _ptr(sink), _stream(buf.device)))


def _group_args(x, ts, outs):
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    if not 1 <= len(ts) <= MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} weights")
    if any(t.k != x.shape[1] for t in ts):
        raise ValueError("every weight of a group must have k = x.shape[1]")
    if outs is None:
        outs = [torch.empty((m, t.n), dtype=torch.bfloat16, device=x.device) for t in ts]
    descs = [t.desc() for t in ts]
    darr = (ctypes.POINTER(W12Desc) * len(ts))(*[ctypes.pointer(d) for d in descs])
    yarr = (c_void_p * len(ts))(*[_as_bits(o).data_ptr() for o in outs])
    ws = workspace(max(workspace_bytes(OP_GEMM_GROUP, m, sum(t.n for t in ts), ts[0].k), 256),
                   x.device)
    args = (_ptr(x), m, ctypes.cast(darr, c_void_p), len(ts), ctypes.cast(yarr, c_void_p), _ptr(ws),
            ws.numel(), _stream(x.device))
    return args, outs, (x, ts, outs, ws, descs, darr, yarr)


def gemm_group(x, ts, outs=None, rms: bool = False):
    """y_i = x . W_i^T for the weights ts (1..4, same k) in one launch per codebook kind;
    rms as for gemm (w12_gemm_group_rms).  A group of F8Tensors goes to w12_gemm_f8_group."""
    if ts and all(isinstance(t, F8Tensor) for t in ts):
        return gemm_f8_group(x, [(t.tiles, t.scale, t.n) for t in ts], ts[0].k, outs, rms=rms)
    if any(isinstance(t, F8Tensor) for t in ts):
        raise ValueError("gemm_group: a group holds W12 weights or FP8 weights, not both")
    args, outs, keep = _group_args(x, ts, outs)
    fn = "w12_gemm_group_rms" if rms else "w12_gemm_group"
    _check(fn, getattr(lib(), fn)(*args))
    return outs


def gemm_bf16(x, w, out=None):
    """The same kernel family on plain BF16 weights w [n, k]."""
    torch = _torch()
    x = _as_bits(x)
    w = _as_bits(w)
    m = x.shape[0]
    n, k = w.shape
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    ws = workspace(max(workspace_bytes(OP_GEMM_BF16, m, n, k), 256), x.device)
    _check("w12_gemm_bf16", lib().w12_gemm_bf16(_ptr(x), m, _ptr(w), n, k, _ptr(_as_bits(out)),
                                                _ptr(ws), ws.numel(), _stream(x.device)))
    return out


def bf16_tile(w):
    """4 KB-tiled copy of BF16 weights w [n, k] (the second baseline's layout)."""
    torch = _torch()
    w = _as_bits(w)
    n, k = w.shape
    out = torch.empty(n * k * 2, dtype=torch.uint8, device=w.device)
    _check("w12_bf16_tile", lib().w12_bf16_tile(_ptr(w), n, k, _ptr(out), _stream(w.device)))
    return out


def gemm_bf16_tiled(x, w_tiled, n: int, k: int, out=None):
    """The same kernel family on 4 KB-tiled BF16 weights (from bf16_tile)."""
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    if x.shape[1] != k or w_tiled.numel() * w_tiled.element_size() != 2 * n * k:
        raise ValueError("gemm_bf16_tiled: x must be [m, k] and w_tiled n*k*2 bytes")
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    ws = workspace(max(workspace_bytes(OP_GEMM_BF16, m, n, k), 256), x.device)
    _check("w12_gemm_bf16_tiled", lib().w12_gemm_bf16_tiled(
        _ptr(x), m, _ptr(w_tiled), n, k, _ptr(_as_bits(out)), _ptr(ws), ws.numel(), _stream(x.device)))
    return out


def f8_tile(q):
    """2 KB-tiled copy of FP8 E4M3 codes q [n, k] (uint8 storage) for gemm_f8."""
    torch = _torch()
    if not q.is_cuda or q.dtype != torch.uint8 or not q.is_contiguous() or q.dim() != 2:
        raise ValueError("f8_tile: q must be a contiguous uint8 CUDA tensor [n, k]")
    n, k = q.shape
    out = torch.empty(n * k, dtype=torch.uint8, device=q.device)
    _check("w12_f8_tile", lib().w12_f8_tile(_ptr(q), n, k, _ptr(out), _stream(q.device)))
    return out


def gemm_f8(x, q_tiled, scale, n: int, k: int, out=None, rms: bool = False):
    """y = x . W^T for the FP8 weight W = E4M3(q) * block scale: q_tiled from f8_tile,
    scale float32 [ceil(n/128), k/128].  rms: each output row divided by the RMS of its x
    row (w12_gemm_f8_rms)."""
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    if x.shape[1] != k or q_tiled.numel() * q_tiled.element_size() != n * k:
        raise ValueError("gemm_f8: x must be [m, k] and q_tiled n*k bytes")
    if (not scale.is_cuda or scale.dtype != torch.float32 or not scale.is_contiguous()
            or scale.numel() != ((n + 127) // 128) * (k // 128)):
        raise ValueError("gemm_f8: scale must be a contiguous float32 CUDA tensor "
                         "[ceil(n/128), k/128]")
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    ws = workspace(max(workspace_bytes(OP_GEMM_F8, m, n, k), 256), x.device)
    fn = "w12_gemm_f8_rms" if rms else "w12_gemm_f8"
    _check(fn, getattr(lib(), fn)(
        _ptr(x), m, _ptr(q_tiled), _ptr(scale), n, k, _ptr(_as_bits(out)), _ptr(ws), ws.numel(),
        _stream(x.device)))
    return out


def _f8_group_args(x, weights, k: int, outs):
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    if x.shape[1] != k or not 1 <= len(weights) <= MAX_GROUP:
        raise ValueError("gemm_f8_group: x must be [m, k] and 1..MAX_GROUP weights given")
    for qt, sc, n in weights:
        if qt.numel() * qt.element_size() != n * k or sc.dtype != torch.float32 or \
                not sc.is_contiguous() or sc.numel() != ((n + 127) // 128) * (k // 128):
            raise ValueError("gemm_f8_group: each weight is (q_tiled of n*k bytes, float32 "
                             "scale [ceil(n/128), k/128], n)")
    if outs is None:
        outs = [torch.empty((m, n), dtype=torch.bfloat16, device=x.device) for _, _, n in weights]
    nw = len(weights)
    ptrs = (c_void_p * nw)(*[qt.data_ptr() for qt, _, _ in weights])
    scs = (c_void_p * nw)(*[sc.data_ptr() for _, sc, _ in weights])
    ns = (c_uint64 * nw)(*[n for _, _, n in weights])
    ys = (c_void_p * nw)(*[_as_bits(o).data_ptr() for o in outs])
    n_total = sum(n for _, _, n in weights)
    ws = workspace(max(workspace_bytes(OP_GEMM_GROUP, m, n_total, k), 256), x.device)
    args = (_ptr(x), m, ctypes.cast(ptrs, c_void_p), ctypes.cast(scs, c_void_p),
            ctypes.cast(ns, c_void_p), nw, k, ctypes.cast(ys, c_void_p), _ptr(ws), ws.numel(),
            _stream(x.device))
    return args, outs, (x, weights, outs, ws, ptrs, scs, ns, ys)


def gemm_f8_group(x, weights, k: int, outs=None, rms: bool = False):
    """One launch over up to MAX_GROUP FP8 weights that read x: weights is a list of
    (q_tiled, scale, n) as gemm_f8 takes them; returns the outputs [m, n_i].  rms as for
    gemm_f8 (w12_gemm_f8_group_rms)."""
    args, outs, _keep = _f8_group_args(x, weights, k, outs)
    fn = "w12_gemm_f8_group_rms" if rms else "w12_gemm_f8_group"
    _check(fn, getattr(lib(), fn)(*args))
    return outs


def lmhead_verify(x, t: W12Tensor, draft, argmax_out=None, accepted_out=None):
    """Exact-logit argmax per row (lowest index on ties) and accepted-prefix length."""
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    if argmax_out is None:
        argmax_out = torch.empty(m, dtype=torch.int32, device=x.device)
    if accepted_out is None:
        accepted_out = torch.empty(1, dtype=torch.int32, device=x.device)
    n_draft = int(draft.numel())
    ws = workspace(workspace_bytes(OP_VERIFY, m, t.n, t.k), x.device, "verify")
    d = t.desc()
    _check("w12_lmhead_verify", lib().w12_lmhead_verify(
        _ptr(x), m, ctypes.byref(d), _ptr(draft) if n_draft else None, n_draft, _ptr(argmax_out),
        _ptr(accepted_out), _ptr(ws), ws.numel(), _stream(x.device)))
    return argmax_out, accepted_out


def _batched_checked(x, t: W12Tensor, req_off, req_ndraft, draft, argmax_out, accepted_out):
    """Validated batched-verification tensors (the outputs allocated when not given)."""
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    n_req = int(req_ndraft.numel())
    for name, a, size in (("req_off", req_off, n_req + 1), ("req_ndraft", req_ndraft, n_req),
                          ("draft", draft, m)):
        if a.dtype != torch.int32 or a.numel() != size or a.device != x.device:
            raise ValueError(f"lmhead_verify_batched: {name} must be int32 [{size}] on {x.device}")
    if argmax_out is None:
        argmax_out = torch.empty(m, dtype=torch.int32, device=x.device)
    if accepted_out is None:
        accepted_out = torch.empty(n_req, dtype=torch.int32, device=x.device)
    return x, m, n_req, argmax_out, accepted_out


def _batched_args(x, t: W12Tensor, req_off, req_ndraft, draft, argmax_out, accepted_out):
    x, m, n_req, argmax_out, accepted_out = _batched_checked(x, t, req_off, req_ndraft, draft,
                                                             argmax_out, accepted_out)
    ws = workspace(workspace_bytes(OP_VERIFY, m, t.n, t.k), x.device, "verify")
    d = t.desc()
    args = (_ptr(x), m, ctypes.byref(d), _ptr(req_off), _ptr(req_ndraft), n_req, _ptr(draft),
            _ptr(argmax_out), _ptr(accepted_out), _ptr(ws), ws.numel(), _stream(x.device))
    return args, (x, t, req_off, req_ndraft, draft, argmax_out, accepted_out, ws, d)


def lmhead_verify_batched(x, t: W12Tensor, req_off, req_ndraft, draft, argmax_out=None,
                          accepted_out=None):
    """Several requests verified in one pass: request r owns rows req_off[r] ..
    req_off[r+1]-1 and drafts draft[req_off[r] + i] for i < req_ndraft[r] (int32 device
    tensors [n_req+1], [n_req], [m]).  Returns (argmax [m], accepted [n_req]); an invalid
    request entry gets accepted -1."""
    args, keep = _batched_args(x, t, req_off, req_ndraft, draft, argmax_out, accepted_out)
    _check("w12_lmhead_verify_batched", lib().w12_lmhead_verify_batched(*args))
    return keep[5], keep[6]


@dataclass
class ScreenCopy:
    """The screen copy of an LM head for two-level verification (w12_screen_encode):
    8-bit codes with a BF16 scale per 32 columns, plus the per-row bound constants."""
    n: int
    k: int
    buf: object        # torch.uint8 [w12_screen_bytes(n, k)]

    def nbytes(self) -> int:
        return int(self.buf.numel())


def screen_encode(w) -> ScreenCopy:
    """Screen copy of BF16 weights w [n, k] (CUDA) on the same device."""
    torch = _torch()
    w = _as_bits(w)
    n, k = w.shape
    nbytes = int(lib().w12_screen_bytes(n, k))
    if nbytes == 0:
        raise ValueError(f"screen copy needs n % 16 == 0, k % 128 == 0, 0 < k < 2^20 (got {n}x{k})")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _check("w12_screen_encode", lib().w12_screen_encode(_ptr(w), n, k, _ptr(buf), nbytes,
                                                        _stream(w.device)))
    return ScreenCopy(n=n, k=k, buf=buf)


def _verify2_ws(m: int, t: W12Tensor, dev):
    # zero-filled on allocation: its row tickets start at zero (every call leaves them so)
    return workspace(workspace_bytes(OP_VERIFY2, m, t.n, t.k), dev, "verify2")


def _check_screen(t: W12Tensor, sc: ScreenCopy):
    if (sc.n, sc.k) != (t.n, t.k):
        raise ValueError(f"screen copy is {sc.n}x{sc.k}, the head {t.n}x{t.k}")


def lmhead_verify2(x, t: W12Tensor, sc: ScreenCopy, draft, argmax_out=None, accepted_out=None):
    """Two-level verification: the same results as lmhead_verify, from the screen copy
    first and the W12 head for the logits it cannot rule out."""
    torch = _torch()
    _check_screen(t, sc)
    x = _as_bits(x)
    m = x.shape[0]
    if argmax_out is None:
        argmax_out = torch.empty(m, dtype=torch.int32, device=x.device)
    if accepted_out is None:
        accepted_out = torch.empty(1, dtype=torch.int32, device=x.device)
    n_draft = int(draft.numel())
    ws = _verify2_ws(m, t, x.device)
    d = t.desc()
    _check("w12_lmhead_verify2", lib().w12_lmhead_verify2(
        _ptr(x), m, ctypes.byref(d), _ptr(sc.buf), _ptr(draft) if n_draft else None, n_draft,
        _ptr(argmax_out), _ptr(accepted_out), _ptr(ws), ws.numel(), _stream(x.device)))
    return argmax_out, accepted_out


def _batched2_args(x, t: W12Tensor, sc: ScreenCopy, req_off, req_ndraft, draft, argmax_out,
                   accepted_out):
    _check_screen(t, sc)
    x, m, n_req, argmax_out, accepted_out = _batched_checked(x, t, req_off, req_ndraft, draft,
                                                             argmax_out, accepted_out)
    ws = _verify2_ws(m, t, x.device)
    d = t.desc()
    args = (_ptr(x), m, ctypes.byref(d), _ptr(sc.buf), _ptr(req_off), _ptr(req_ndraft), n_req,
            _ptr(draft), _ptr(argmax_out), _ptr(accepted_out), _ptr(ws), ws.numel(),
            _stream(x.device))
    return args, (x, t, sc, req_off, req_ndraft, draft, argmax_out, accepted_out, ws, d)


def lmhead_verify2_batched(x, t: W12Tensor, sc: ScreenCopy, req_off, req_ndraft, draft,
                           argmax_out=None, accepted_out=None):
    """Several requests in one two-level pass (requests as lmhead_verify_batched)."""
    args, keep = _batched2_args(x, t, sc, req_off, req_ndraft, draft, argmax_out, accepted_out)
    _check("w12_lmhead_verify2_batched", lib().w12_lmhead_verify2_batched(*args))
    return keep[6], keep[7]


def screen_logits_f32(x, t: W12Tensor, sc: ScreenCopy):
    """The screen logits z8^ [m, n] and their certified bounds [m, n] (FP32) from the first
    pass of the two-level verification."""
    torch = _torch()
    _check_screen(t, sc)
    x = _as_bits(x)
    m = x.shape[0]
    z = torch.empty((m, t.n), dtype=torch.float32, device=x.device)
    bnd = torch.empty((m, t.n), dtype=torch.float32, device=x.device)
    ws = _verify2_ws(m, t, x.device)
    d = t.desc()
    _check("w12_screen_logits_f32", lib().w12_screen_logits_f32(
        _ptr(x), m, ctypes.byref(d), _ptr(sc.buf), _ptr(z), _ptr(bnd), _ptr(ws), ws.numel(),
        _stream(x.device)))
    return z, bnd


def verify2_candidates(t: W12Tensor, m: int):
    """Per-row diagnostic counts of the last two-level verification on this device's
    workspace: int32 [m, 2] = (logits the screen could not rule out, those left after the
    FP64 recomputation; 1 means no exact sum was needed)."""
    torch = _torch()
    ws = _verify2_ws(m, t, t.device)
    return ws[4096:4096 + 8 * m].view(torch.int32).view(m, 2).clone()


def verify_candidates(t: W12Tensor, m: int):
    """Per-row diagnostic counts of the last verification on this device's workspace:
    int32 [m, 2] = (candidate logits screened in FP64, those left after the screen; 1
    means no exact sum was needed)."""
    torch = _torch()
    ws = workspace(workspace_bytes(OP_VERIFY, m, t.n, t.k), t.device, "verify")
    return ws[:8 * m].view(torch.int32).view(m, 2).clone()   # the counts open the workspace


def logits_f32(x, t: W12Tensor):
    """FP32 logits z^ [m, n] and error scales S [m, n] from the first pass of the
    verification (same kernels, same summation order).  S = X_m W_v rounded up, an upper
    bound of sum_k |x_k||w_vk| (Cauchy-Schwarz): W_v the first pass's bound of
    ||w_v||_2, X_m the second pass's bound of ||x_m||_2."""
    torch = _torch()
    x = _as_bits(x)
    m = x.shape[0]
    z = torch.empty((m, t.n), dtype=torch.float32, device=x.device)
    s = torch.empty((m, t.n), dtype=torch.float32, device=x.device)
    ws = workspace(workspace_bytes(OP_VERIFY, m, t.n, t.k), x.device, "verify")
    d = t.desc()
    _check("w12_logits_f32", lib().w12_logits_f32(_ptr(x), m, ctypes.byref(d), _ptr(z), _ptr(s),
                                                  _ptr(ws), ws.numel(), _stream(x.device)))
    return z, s


def rms_rescale(x, out=None):
    torch = _torch()
    x = _as_bits(x)
    m, k = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check("w12_rms_rescale", lib().w12_rms_rescale(_ptr(x), m, k, _ptr(_as_bits(out)), _stream(x.device)))
    return out


# ----------------------------------------------------------------------------- paged cache
@dataclass
class PageTable:
    """Block tables of up to max_req requests over one pool of pages (page_table makes an
    empty one).  Request r's token t lies in page table[r, t // page_size].  The free pages are
    ring[state[0]], ring[state[0] + 1], ... (state[1] of them, indices modulo n_pages).  With refs
    (page_refs) requests may share pages: kv_fork in place of kv_plan."""
    page_size: int
    table: object      # torch.int32 [max_req, max_pages]
    held: object       # torch.int32 [max_req]: pages each request holds
    ring: object       # torch.int32 [n_pages]
    state: object      # torch.int32 [4]: head, count, 0, 0
    refs: object = None    # torch.int32 [5 n_pages + 1024]: holders of each page, then words of the calls

    @property
    def n_pages(self) -> int:
        return self.ring.numel()

    @property
    def device(self):
        return self.table.device

    def desc(self) -> W12Pages:
        if self.table.dim() != 2:
            raise ValueError("PageTable: table must be [max_req, max_pages]")
        max_req, max_pages = self.table.shape
        for name, t, size in (("table", self.table, max_req * max_pages), ("held", self.held, max_req),
                              ("ring", self.ring, self.n_pages), ("state", self.state, 4)):
            _int32(f"PageTable: {name}", t, size, self.device)
        p = W12Pages()
        p.n_pages, p.page_size, p.max_req, p.max_pages = self.n_pages, self.page_size, max_req, max_pages
        p.table, p.held, p.ring, p.state = (t.data_ptr() for t in
                                            (self.table, self.held, self.ring, self.state))
        return p


def page_refs(n_pages: int, device="cuda"):
    """Zero counts for an empty pool (W12_REFS_WORDS).  For tables that hold pages already, the first
    n_pages entries are the number of entries table[r, c], c < held[r], that name each page."""
    torch = _torch()
    return torch.zeros(5 * n_pages + 1024, dtype=torch.int32, device=device)


def page_table(n_pages: int, page_size: int, max_req: int, max_pages: int, device="cuda",
               shared: bool = False) -> PageTable:
    """A pool of n_pages free pages and empty tables for max_req requests of at most
    max_pages pages each; shared: with counts, for requests that share pages (kv_fork)."""
    torch = _torch()
    i32 = dict(dtype=torch.int32, device=device)
    return PageTable(page_size, torch.full((max_req, max_pages), -1, **i32),
                     torch.zeros(max_req, **i32), torch.arange(n_pages, **i32),
                     torch.tensor([0, n_pages, 0, 0], **i32), page_refs(n_pages, device) if shared else None)


@dataclass
class KvCache:
    """One layer's paged keys and values: k [n_pages, n_kv_heads, page_size, head_dim] and v
    transposed inside its page, [n_pages, n_kv_heads, head_dim, page_size]; both bfloat16, or
    both float8_e4m3fn with a stored code standing for code * scale."""
    k: object
    v: object
    k_scale: float = 1.0
    v_scale: float = 1.0

    @property
    def device(self):
        return self.k.device

    def desc(self) -> W12Kv:
        torch = _torch()
        k, v = self.k, self.v
        if not k.is_cuda:
            raise ValueError("W12 calls need CUDA (HIP) tensors")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or v.dtype != k.dtype:
            raise ValueError("KvCache: k and v must both be bfloat16 or both float8_e4m3fn")
        if k.dim() != 4 or tuple(v.shape) != (k.shape[0], k.shape[1], k.shape[3], k.shape[2]) or \
                v.device != k.device or not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("KvCache: k must be [n_pages, n_kv_heads, page_size, head_dim] and v "
                             "[n_pages, n_kv_heads, head_dim, page_size], contiguous, on one device")
        d = W12Kv()
        d.n_pages, d.n_kv_heads, d.page_size, d.head_dim = k.shape
        d.dtype = KV_BF16 if k.dtype == torch.bfloat16 else KV_E4M3
        d.k_scale, d.v_scale = self.k_scale, self.v_scale
        d.k, d.v = k.data_ptr(), v.data_ptr()
        return d


def kv_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=None,
             k_scale: float = 1.0, v_scale: float = 1.0, device="cuda") -> KvCache:
    """An empty (zero) cache of n_pages pages; dtype bfloat16 (default) or float8_e4m3fn."""
    torch = _torch()
    dtype = dtype or torch.bfloat16
    bits = torch.int16 if dtype == torch.bfloat16 else torch.uint8
    k = torch.zeros((n_pages, n_kv_heads, page_size, head_dim), dtype=bits, device=device).view(dtype)
    v = torch.zeros((n_pages, n_kv_heads, head_dim, page_size), dtype=bits, device=device).view(dtype)
    return KvCache(k, v, k_scale, v_scale)


@dataclass
class Rope:
    """Norm and rotation of query and key heads: inv_freq float64 [rot_dim / 2] in radians per
    position (None: no rotation), BF16 norm weights [head_dim] (None: no norm), pairs
    (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved."""
    inv_freq: object = None
    q_norm: object = None
    k_norm: object = None
    eps: float = 1e-6
    interleaved: bool = False

    def desc(self, head_dim: int, device) -> W12Rope:
        torch = _torch()
        f = self.inv_freq
        if f is not None and (f.dtype != torch.float64 or f.device != device or not f.is_contiguous()):
            raise ValueError("Rope: inv_freq must be a contiguous float64 tensor on the cache's device")
        for w in (self.q_norm, self.k_norm):
            if w is not None and (_as_bits(w).numel() != head_dim or w.device != device):
                raise ValueError("Rope: norm weights must be BF16 [head_dim] on the cache's device")
        d = W12Rope()
        d.q_norm = self.q_norm.data_ptr() if self.q_norm is not None else None
        d.k_norm = self.k_norm.data_ptr() if self.k_norm is not None else None
        d.inv_freq = f.data_ptr() if f is not None and f.numel() else None
        d.rot_dim = 2 * f.numel() if f is not None else 0
        d.interleaved, d.eps = int(self.interleaved), self.eps
        return d


def _int32(name: str, t, size: int, device):
    if t.dtype != _torch().int32 or t.numel() != size or t.device != device or not t.is_cuda \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {size} on {device}")


def _heads(name: str, t, m: int, n: int, d: int, device) -> int:
    """Row stride (elements) of a BF16 tensor [m, n, d] whose rows hold n contiguous heads."""
    torch = _torch()
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be BF16 on {device}")
    if tuple(t.shape) != (m, n, d) or (m > 0 and (t.stride(2) != 1 or (n > 1 and t.stride(1) != d))):
        raise ValueError(f"{name} must be [{m}, {n}, {d}] with contiguous heads")
    if m > 1 and t.stride(0) < n * d:
        raise ValueError(f"{name}: rows overlap")
    return t.stride(0) if m > 1 else n * d


def _rows(t):
    """(address, bytes of a row, bytes between rows, rows) of a tensor [m, heads, d], or of any
    contiguous one as a single row."""
    shape, es = t.shape, t.element_size()
    if len(shape) == 3 and shape[0] > 1:
        return t.data_ptr(), shape[1] * shape[2] * es, t.stride(0) * es, shape[0]
    nbytes = t.numel() * es
    return t.data_ptr(), nbytes, nbytes, 1 if nbytes else 0


def _meet(a, b) -> bool:
    """Do two sets of rows (as _rows has them) share a byte?  Columns of one buffer do not."""
    (p, la, sa, ma), (q, lb, sb, mb) = a, b
    if not (ma and mb and la and lb) or p >= q + sb * (mb - 1) + lb or q >= p + sa * (ma - 1) + la:
        return False
    if ma == 1:
        sa = sb
    if mb == 1:
        sb = sa
    if sa != sb:
        return any(_meet((p + i * sa, la, sb, 1), b) for i in range(ma))
    # rows i and j meet where -lb < q - p + (j - i) sa < la: the smallest j - i past the left end
    k = max((p - q - lb) // sa + 1, 1 - ma)
    return k < mb and q - p + k * sa < la


def _disjoint(what: str, outs, ins):
    """Every tensor in outs {name: tensor} apart from the others and from those in ins."""
    spans = []
    for i, (name, t) in enumerate((*outs.items(), *ins.items())):
        if t is None:
            continue
        rows = p, length, stride, n = _rows(t)
        end = p + stride * (n - 1) + length
        for other, q, q_end, of in spans:
            if p < q_end and q < end and _meet(rows, of):
                raise ValueError(f"{what}: {other} overlaps {name}")
        if i < len(outs):
            spans.append((name, p, end, rows))


def _issue(name: str, args, device):
    torch = _torch()
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            _check(name, getattr(lib(), name)(*args))
    else:
        _check(name, getattr(lib(), name)(*args))


def _plan_args(pt: PageTable, length, req_off, kv_len, pos, slot):
    if pt.refs is not None:
        raise ValueError("kv_plan: the pool's pages are shared (refs): kv_fork")
    dev, n_req, m = pt.device, int(length.numel()), int(pos.numel())
    for name, t, size in (("length", length, n_req), ("req_off", req_off, n_req + 1),
                          ("kv_len", kv_len, n_req), ("pos", pos, m), ("slot", slot, m)):
        _int32(f"kv_plan: {name}", t, size, dev)
    d = pt.desc()
    _disjoint("kv_plan", {"kv_len": kv_len, "pos": pos, "slot": slot, "table": pt.table, "held": pt.held,
                          "ring": pt.ring, "state": pt.state}, {"length": length, "req_off": req_off})
    args = (ctypes.byref(d), _ptr(length), _ptr(req_off), n_req, m, _ptr(kv_len),
            _ptr(pos) if m else None, _ptr(slot) if m else None, _stream(dev))
    return args, (pt, length, req_off, kv_len, pos, slot, d)


def kv_plan(pt: PageTable, length, req_off, m: int, kv_len=None, pos=None, slot=None):
    """Bring the block tables in line with the requests' lengths and map the m new rows
    (w12_kv_plan): request r keeps length[r] tokens and adds rows req_off[r] ..
    req_off[r+1]-1.  Pages past its need go back to the pool (rejected drafts; everything at
    length 0 without rows), missing ones are taken.  length int32 [n_req], req_off int32
    [n_req + 1].  Returns int32 (kv_len [n_req], pos [m], slot [m]); -1 marks a request that
    found too few pages or has invalid lengths, and its rows."""
    torch = _torch()
    new = lambda n: torch.empty(n, dtype=torch.int32, device=pt.device)
    kv_len = new(length.numel()) if kv_len is None else kv_len
    pos = new(m) if pos is None else pos
    slot = new(m) if slot is None else slot
    if pos.numel() != m:
        raise ValueError(f"kv_plan: pos must have m = {m} entries")
    args, keep = _plan_args(pt, length, req_off, kv_len, pos, slot)
    _issue("w12_kv_plan", args, pt.device)
    return kv_len, pos, slot


def _rope_args(q, k, v, cache: KvCache, rope: Rope, pos, slot, q_out):
    c = cache.desc()
    dev, m, n, d = cache.device, q.shape[0], q.shape[1], c.head_dim
    strides = [_heads("qk_rope: q", q, m, n, d, dev), _heads("qk_rope: k", k, m, c.n_kv_heads, d, dev),
               _heads("qk_rope: v", v, m, c.n_kv_heads, d, dev),
               _heads("qk_rope: q_out", q_out, m, n, d, dev)]
    for name, t in (("pos", pos), ("slot", slot)):
        _int32(f"qk_rope: {name}", t, m, dev)
    if q_out.data_ptr() == q.data_ptr() and strides[3] != strides[0]:
        raise ValueError("qk_rope: q_out may be q itself, with the same strides")
    r = rope.desc(d, dev)
    ins = {"k": k, "v": v, "pos": pos, "slot": slot, "inv_freq": rope.inv_freq, "q_norm": rope.q_norm,
           "k_norm": rope.k_norm}
    if q_out.data_ptr() != q.data_ptr():
        ins["q"] = q
    _disjoint("qk_rope", {"q_out": q_out, "the cache's k": cache.k, "the cache's v": cache.v}, ins)
    args = (_ptr(q), strides[0], _ptr(k), strides[1], _ptr(v), strides[2], m, n, ctypes.byref(c),
            ctypes.byref(r), _ptr(pos), _ptr(slot), _ptr(q_out), strides[3], _stream(dev))
    return args, (q, k, v, cache, rope, pos, slot, q_out, c, r)


def qk_rope(q, k, v, cache: KvCache, rope: Rope, pos, slot, q_out=None):
    """Norm and rotate the heads of q [m, n_heads, head_dim] and k [m, n_kv_heads, head_dim] at
    the rows' positions, and append k and v to the cache at their slots (w12_qk_rope; pos and
    slot int32 [m] as kv_plan gives them).  Rows may be strided.  Rows with pos < 0 are passed
    over, rows without a slot leave the cache alone.  Returns q_out (BF16; may be q)."""
    if q.dim() != 3:
        raise ValueError("qk_rope: q must be [m, n_heads, head_dim]")
    if q_out is None:
        q_out = _torch().empty(tuple(q.shape), dtype=q.dtype, device=q.device)
    args, _keep = _rope_args(q, k, v, cache, rope, pos, slot, q_out)
    _issue("w12_qk_rope", args, cache.device)
    return q_out


_ATTN_WS = {}


def attn_workspace(device="cuda"):
    """A workspace for attn_paged (zero tickets), for callers that keep their own: one for each
    stream or captured graph that may run at the same time as others.  It is zeroed on the current
    stream: a call on another one has to wait for that."""
    torch = _torch()
    return torch.zeros(ATTN_WS_BYTES, dtype=torch.uint8, device=device)


def _attn_ws(dev, ws):
    """The caller's workspace, or one per device and stream.  Under graph capture without the
    caller's: memory of the graph itself, its tickets zeroed inside the graph, so no other
    graph or stream shares it."""
    torch = _torch()
    if ws is not None:
        if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"attn_paged: ws must be a contiguous uint8 tensor on {dev}")
        return ws
    with torch.cuda.device(dev):
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(ATTN_WS_BYTES, dtype=torch.uint8, device=dev)
            _check("w12_workspace_init", lib().w12_workspace_init(_ptr(ws), 4096, _stream(dev)))
            return ws
        key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
        if key not in _ATTN_WS:
            _ATTN_WS[key] = attn_workspace(dev)
        return _ATTN_WS[key]


def _attn_args(q, cache: KvCache, table, kv_len, req_off, out, scale, ws):
    c = cache.desc()
    dev, m, n, d, n_req = cache.device, q.shape[0], q.shape[1], c.head_dim, int(kv_len.numel())
    qs, os_ = _heads("attn_paged: q", q, m, n, d, dev), _heads("attn_paged: out", out, m, n, d, dev)
    if table.dim() != 2 or table.shape[0] < n_req:
        raise ValueError("attn_paged: table must be [>= n_req, max_pages]")
    _int32("attn_paged: table", table, table.shape[0] * table.shape[1], dev)
    _int32("attn_paged: kv_len", kv_len, n_req, dev)
    _int32("attn_paged: req_off", req_off, n_req + 1, dev)
    ws = _attn_ws(dev, ws)
    _disjoint("attn_paged", {"out": out, "ws": ws},
              {"q": q, "the cache's k": cache.k, "the cache's v": cache.v, "table": table,
               "kv_len": kv_len, "req_off": req_off})
    scale = d ** -0.5 if scale is None else float(scale)
    args = (_ptr(q), qs, m, n, ctypes.byref(c), _ptr(table), table.shape[1], _ptr(kv_len), _ptr(req_off),
            n_req, scale, _ptr(out), os_, _ptr(ws), ws.numel(), _stream(dev))
    return args, (q, cache, table, kv_len, req_off, out, ws, c)


def attn_paged(q, cache: KvCache, table, kv_len, req_off, out=None, scale=None, ws=None):
    """Attention of the new rows q [m, n_heads, head_dim] over the paged cache (w12_attn_paged):
    request r owns rows req_off[r] .. req_off[r+1]-1, the last kv_len[r] tokens' newest; row i
    sees the tokens up to its own.  table int32 [>= n_req, max_pages], kv_len int32 [n_req],
    req_off int32 [n_req + 1]; scale defaults to head_dim ** -0.5; n_heads any multiple of the
    cache's heads.  Returns out (BF16; rows of no request are left as they were)."""
    if q.dim() != 3:
        raise ValueError("attn_paged: q must be [m, n_heads, head_dim]")
    if out is None:
        out = _torch().zeros(tuple(q.shape), dtype=q.dtype, device=q.device)
    args, _keep = _attn_args(q, cache, table, kv_len, req_off, out, scale, ws)
    _issue("w12_attn_paged", args, cache.device)
    return out


# ----------------------------------------------------------------------------- shared pages
def _refs(what: str, pt: PageTable):
    if pt.refs is None:
        raise ValueError(f"{what}: the pool has no counts of its pages' holders (refs: page_refs)")
    _int32(f"{what}: refs", pt.refs, 5 * pt.n_pages + 1024, pt.device)
    return pt.refs


def _quads(name: str, t, n: int, device):
    if t.dim() != 2 or t.shape[1] != 4:
        raise ValueError(f"{name} must be [n, 4]")
    _int32(name, t, 4 * n, device)


def _fork_args(pt: PageTable, parent, length, req_off, kv_len, pos, slot, copies):
    dev, n_req, m = pt.device, int(length.numel()), int(pos.numel())
    for name, t, size in (("parent", parent, n_req), ("length", length, n_req), ("req_off", req_off, n_req + 1),
                          ("kv_len", kv_len, n_req), ("pos", pos, m), ("slot", slot, m)):
        if t is not None or name != "parent":
            _int32(f"kv_fork: {name}", t, size, dev)
    _quads("kv_fork: copies", copies, n_req, dev)
    d, refs = pt.desc(), _refs("kv_fork", pt)
    _disjoint("kv_fork", {"kv_len": kv_len, "pos": pos, "slot": slot, "copies": copies, "table": pt.table,
                          "held": pt.held, "ring": pt.ring, "state": pt.state, "refs": refs},
              {"parent": parent, "length": length, "req_off": req_off})
    args = (ctypes.byref(d), _ptr(refs), _ptr(parent) if parent is not None else None, _ptr(length), _ptr(req_off),
            n_req, m, _ptr(kv_len), _ptr(pos) if m else None, _ptr(slot) if m else None, _ptr(copies), _stream(dev))
    return args, (pt, parent, length, req_off, kv_len, pos, slot, copies, d)


def kv_fork(pt: PageTable, parent, length, req_off, m: int, kv_len=None, pos=None, slot=None, copies=None):
    """kv_plan for requests that share pages (w12_kv_fork): request r becomes the first length[r]
    tokens of request parent[r] as it was (parent None: its own; -1: none) and rows req_off[r] ..
    req_off[r+1]-1.  Full pages are shared; where a request will write into a page that another
    one holds, copies[r] = (page, new page, tokens, 0) says what kv_copy has to copy before the rows are
    appended.  Served whole or, if the pool has too few pages, not at all (everything -1).
    Returns int32 (kv_len [n_req], pos [m], slot [m], copies [n_req, 4])."""
    torch = _torch()
    new = lambda *n: torch.empty(n, dtype=torch.int32, device=pt.device)
    kv_len = new(length.numel()) if kv_len is None else kv_len
    pos = new(m) if pos is None else pos
    slot = new(m) if slot is None else slot
    copies = new(length.numel(), 4) if copies is None else copies
    if pos.numel() != m:
        raise ValueError(f"kv_fork: pos must have m = {m} entries")
    args, _keep = _fork_args(pt, parent, length, req_off, kv_len, pos, slot, copies)
    _issue("w12_kv_fork", args, pt.device)
    return kv_len, pos, slot, copies


def _copy_args(caches, copies):
    caches = list(caches)
    if not caches:
        raise ValueError("kv_copy: no caches")
    dev = caches[0].device
    if any(c.device != dev for c in caches):
        raise ValueError("kv_copy: the caches must be on one device")
    _quads("kv_copy: copies", copies, copies.shape[0], dev)
    d = (W12Kv * len(caches))(*(c.desc() for c in caches))
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                   for t in (copies, *(x for c in caches for x in (c.k, c.v))) if t.numel())
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError("kv_copy: the caches, or a cache and copies, overlap")
    args = (d, len(caches), _ptr(copies) if copies.shape[0] else None, copies.shape[0], _stream(dev))
    return args, (caches, copies, d), dev


def kv_copy(caches, copies):
    """Copy pages in the caches of all layers (w12_kv_copy): copies int32 [n, 4] as kv_fork or
    kv_compact give them."""
    args, _keep, dev = _copy_args(caches, copies)
    _issue("w12_kv_copy", args, dev)


def _compact_args(pt: PageTable, first: int, moves, moved):
    dev = pt.device
    _quads("kv_compact: moves", moves, moves.shape[0], dev)
    _int32("kv_compact: moved", moved, 1, dev)
    d, refs = pt.desc(), _refs("kv_compact", pt)
    if first < 0 or not 1 <= moves.shape[0] <= pt.n_pages - first:
        raise ValueError("kv_compact: the range leaves the pool")
    _disjoint("kv_compact", {"moves": moves, "moved": moved, "table": pt.table, "ring": pt.ring, "state": pt.state,
                             "refs": refs}, {"held": pt.held})
    args = (ctypes.byref(d), _ptr(refs), first, moves.shape[0], _ptr(moves), _ptr(moved), _stream(dev))
    return args, (pt, moves, moved, d)


def kv_compact(pt: PageTable, first: int, n_clear: int, moves=None, moved=None):
    """Clear the pages first .. first + n_clear - 1 of the pool (w12_kv_compact): those in use move to
    free pages outside, and the tables follow; kv_copy with the returned moves [n_clear, 4] moves
    the contents.  moved [1] is their number, -1 (and nothing changed) if there are too few
    outside.  Afterwards the range is the end of the free ring."""
    torch = _torch()
    new = lambda *n: torch.empty(n, dtype=torch.int32, device=pt.device)
    if n_clear < 1:
        raise ValueError("kv_compact: an empty range")
    moves = new(n_clear, 4) if moves is None else moves
    moved = new(1) if moved is None else moved
    if moves.shape[0] != n_clear:
        raise ValueError(f"kv_compact: moves must be [{n_clear}, 4]")
    args, _keep = _compact_args(pt, first, moves, moved)
    _issue("w12_kv_compact", args, pt.device)
    return moves, moved


_SHARED_WS = {}


def attn_shared_workspace(m: int, n_heads: int, head_dim: int, device="cuda"):
    """A workspace for attn_shared of up to m rows, n_heads heads and head_dim values, in no particular
    state, for callers that keep their own: one for each stream or captured graph that may run at the
    same time as others."""
    n = int(lib().w12_attn_shared_ws_bytes(m, n_heads, head_dim))
    if n == 0:
        raise ValueError("attn_shared_workspace: no such call")
    return _torch().empty(n, dtype=_torch().uint8, device=device)


def _shared_ws(dev, ws, m, n_heads, d):
    """The caller's workspace, or one per device and stream; under graph capture memory of the graph."""
    torch = _torch()
    if ws is not None:
        if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"attn_shared: ws must be a contiguous uint8 tensor on {dev}")
        return ws
    with torch.cuda.device(dev):
        if torch.cuda.is_current_stream_capturing():
            return attn_shared_workspace(m, n_heads, d, dev)
        key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
        have = _SHARED_WS.get(key)
        if have is None or have.numel() < lib().w12_attn_shared_ws_bytes(m, n_heads, d):
            have = _SHARED_WS[key] = attn_shared_workspace(m, n_heads, d, dev)
        return have


def _shared_args(q, cache: KvCache, table, kv_len, req_off, grp_off, grp_len, out, scale, ws):
    c = cache.desc()
    dev, m, n, d, n_req = cache.device, q.shape[0], q.shape[1], c.head_dim, int(kv_len.numel())
    n_grp = int(grp_len.numel())
    qs, os_ = _heads("attn_shared: q", q, m, n, d, dev), _heads("attn_shared: out", out, m, n, d, dev)
    if table.dim() != 2 or table.shape[0] < n_req:
        raise ValueError("attn_shared: table must be [>= n_req, max_pages]")
    _int32("attn_shared: table", table, table.shape[0] * table.shape[1], dev)
    for name, t, size in (("kv_len", kv_len, n_req), ("req_off", req_off, n_req + 1),
                          ("grp_off", grp_off, n_grp + 1), ("grp_len", grp_len, n_grp)):
        _int32(f"attn_shared: {name}", t, size, dev)
    if m * n > MAX_SHARED_ROWS:
        raise ValueError(f"attn_shared: at most {MAX_SHARED_ROWS} query rows (m * n_heads)")
    ws = _shared_ws(dev, ws, m, n, d)
    _disjoint("attn_shared", {"out": out, "ws": ws},
              {"q": q, "the cache's k": cache.k, "the cache's v": cache.v, "table": table,
               "kv_len": kv_len, "req_off": req_off, "grp_off": grp_off, "grp_len": grp_len})
    scale = d ** -0.5 if scale is None else float(scale)
    args = (_ptr(q), qs, m, n, ctypes.byref(c), _ptr(table), table.shape[1], _ptr(kv_len), _ptr(req_off),
            n_req, _ptr(grp_off), _ptr(grp_len), n_grp, scale, _ptr(out), os_, _ptr(ws), ws.numel(), _stream(dev))
    return args, (q, cache, table, kv_len, req_off, grp_off, grp_len, out, ws, c)


def attn_shared(q, cache: KvCache, table, kv_len, req_off, grp_off, grp_len, out=None, scale=None, ws=None):
    """attn_paged for requests that share their first tokens (w12_attn_shared): the first grp_len[g]
    tokens of requests grp_off[g] .. grp_off[g+1]-1 are the same (in the same pages or copies of them)
    and are read once for all of them.  grp_off int32 [n_grp + 1] from 0 to n_req, grp_len int32 [n_grp].  Returns out (BF16; rows
    of no request are left as they were)."""
    if q.dim() != 3:
        raise ValueError("attn_shared: q must be [m, n_heads, head_dim]")
    if out is None:
        out = _torch().zeros(tuple(q.shape), dtype=q.dtype, device=q.device)
    args, _keep = _shared_args(q, cache, table, kv_len, req_off, grp_off, grp_len, out, scale, ws)
    _issue("w12_attn_shared", args, cache.device)
    return out


# ----------------------------------------------------------------------------- beams
_BEAM_WS = {}


def beam_workspace(n: int, vocab: int, k: int, device="cuda"):
    """A workspace for beam_select (zero tickets) of up to n rows, vocab logits and k pairs, for callers
    that keep their own: one for each stream or captured graph that may run at the same time as others.
    It is zeroed on the current stream."""
    size = int(lib().w12_beam_ws_bytes(n, vocab, k))
    if size == 0:
        raise ValueError("beam_workspace: no such call")
    return _torch().zeros(size, dtype=_torch().uint8, device=device)


def _beam_ws(dev, ws, n, vocab, k):
    """The caller's workspace, or one per device and stream; under graph capture memory of the
    graph, its tickets zeroed inside the graph."""
    torch = _torch()
    if ws is not None:
        if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"beam_select: ws must be a contiguous uint8 tensor on {dev}")
        return ws
    size = int(lib().w12_beam_ws_bytes(n, vocab, k))
    with torch.cuda.device(dev):
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(max(size, 16384), dtype=torch.uint8, device=dev)
            _check("w12_workspace_init", lib().w12_workspace_init(_ptr(ws), 16384, _stream(dev)))
            return ws
        key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
        if key not in _BEAM_WS or _BEAM_WS[key].numel() < size:
            _BEAM_WS[key] = torch.zeros(max(size, 16384), dtype=torch.uint8, device=dev)
        return _BEAM_WS[key]


def _beam_args(logits, scores, grp_off, parent, token, score_out, ws):
    torch = _torch()
    if not logits.is_cuda:
        raise ValueError("W12 calls need CUDA (HIP) tensors")
    if logits.dim() != 2 or logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("beam_select: logits must be [n, vocab], bfloat16 or float32")
    dev, (n, vocab) = logits.device, logits.shape
    if n and vocab > 1 and logits.stride(1) != 1 or n > 1 and logits.stride(0) < vocab:
        raise ValueError("beam_select: a row's logits must be contiguous, and rows apart")
    stride = logits.stride(0) if n > 1 else vocab
    if parent.dim() != 2:
        raise ValueError("beam_select: parent must be [n_grp, k]")
    n_grp, k = parent.shape
    _int32("beam_select: grp_off", grp_off, n_grp + 1, dev)
    for name, t in (("parent", parent), ("token", token)):
        _int32(f"beam_select: {name}", t, n_grp * k, dev)
    for name, t, size in (("scores", scores, n), ("score_out", score_out, n_grp * k)):
        if t.dtype != torch.float32 or t.numel() != size or t.device != dev or not t.is_contiguous():
            raise ValueError(f"beam_select: {name} must be a contiguous float32 tensor of {size} on {dev}")
    ws = _beam_ws(dev, ws, n, vocab, k)
    _disjoint("beam_select", {"parent": parent, "token": token, "score_out": score_out, "ws": ws},
              {"logits": logits.unsqueeze(1), "scores": scores, "grp_off": grp_off})
    args = (_ptr(logits) if n else None, LOGITS_F32 if logits.dtype == torch.float32 else LOGITS_BF16, stride, n, vocab,
            _ptr(scores) if n else None, _ptr(grp_off), n_grp, k, _ptr(parent), _ptr(token), _ptr(score_out), _ptr(ws),
            ws.numel(), _stream(dev))
    return args, (logits, scores, grp_off, parent, token, score_out, ws), dev


def beam_select(logits, scores, grp_off, k: int, parent=None, token=None, score_out=None, ws=None):
    """The k best pairs of a row and a token of each group of rows grp_off[g] .. grp_off[g+1]-1, by
    scores[row] + log softmax(logits[row])[token] (w12_beam_select).  logits [n, vocab] bfloat16 or
    float32 (rows may be strided), scores float32 [n], grp_off int32 [n_grp + 1].  Returns (parent int32,
    token int32, score float32), each [n_grp, k], the best first; with k beams to a group, parent as
    it is goes to kv_fork."""
    torch = _torch()
    n_grp = grp_off.numel() - 1
    new = lambda dtype: torch.empty((n_grp, k), dtype=dtype, device=logits.device)
    parent = new(torch.int32) if parent is None else parent
    token = new(torch.int32) if token is None else token
    score_out = new(torch.float32) if score_out is None else score_out
    if tuple(parent.shape) != (n_grp, k):
        raise ValueError(f"beam_select: parent must be [{n_grp}, {k}]")
    args, _keep, dev = _beam_args(logits, scores, grp_off, parent, token, score_out, ws)
    _issue("w12_beam_select", args, dev)
    return parent, token, score_out


# ----------------------------------------------------------------------------- prepared calls
class Prepared:
    """One library call with its arguments marshalled once (device pointers, descriptor,
    workspace, stream); calling it re-issues the call with no other Python work.  The
    tensors it refers to must stay alive, and the stream is the one current when it was
    prepared."""

    def __init__(self, name: str, fn, args, keep):
        self.name, self._fn, self._args, self._keep = name, fn, args, keep

    def __call__(self):
        st = self._fn(*self._args)
        if st != 0:
            raise W12Error(self.name, st)


def prepare_gemm(x, t: W12Tensor, out, rms: bool = False) -> Prepared:
    x, out = _as_bits(x), _as_bits(out)
    m = x.shape[0]
    if x.shape[1] != t.k or tuple(out.shape) != (m, t.n):
        raise ValueError("prepare_gemm: x must be [m, k] and out [m, n]")
    ws = workspace(max(workspace_bytes(OP_GEMM, m, t.n, t.k), 256), x.device)
    d = t.desc()
    args = (_ptr(x), m, ctypes.byref(d), _ptr(out), _ptr(ws), ws.numel(), _stream(x.device))
    fn = "w12_gemm_rms" if rms else "w12_gemm"
    return Prepared(fn, getattr(lib(), fn), args, (x, t, out, ws, d))


def prepare_gemm_group(x, ts, outs, rms: bool = False) -> Prepared:
    args, outs, keep = _group_args(x, ts, outs)
    fn = "w12_gemm_group_rms" if rms else "w12_gemm_group"
    return Prepared(fn, getattr(lib(), fn), args, keep)


def prepare_gemm_f8(x, q_tiled, scale, n: int, k: int, out, rms: bool = False) -> Prepared:
    x, out = _as_bits(x), _as_bits(out)
    m = x.shape[0]
    if x.shape[1] != k or tuple(out.shape) != (m, n) or q_tiled.numel() * q_tiled.element_size() != n * k:
        raise ValueError("prepare_gemm_f8: x must be [m, k], out [m, n], q_tiled n*k bytes")
    ws = workspace(max(workspace_bytes(OP_GEMM_F8, m, n, k), 256), x.device)
    args = (_ptr(x), m, _ptr(q_tiled), _ptr(scale), n, k, _ptr(out), _ptr(ws), ws.numel(),
            _stream(x.device))
    fn = "w12_gemm_f8_rms" if rms else "w12_gemm_f8"
    return Prepared(fn, getattr(lib(), fn), args, (x, q_tiled, scale, out, ws))


def prepare_gemm_f8_group(x, weights, k: int, outs, rms: bool = False) -> Prepared:
    args, outs, keep = _f8_group_args(x, weights, k, outs)
    fn = "w12_gemm_f8_group_rms" if rms else "w12_gemm_f8_group"
    return Prepared(fn, getattr(lib(), fn), args, keep)


def prepare_rms(x, out) -> Prepared:
    x, out = _as_bits(x), _as_bits(out)
    m, k = x.shape
    args = (_ptr(x), m, k, _ptr(out), _stream(x.device))
    return Prepared("w12_rms_rescale", lib().w12_rms_rescale, args, (x, out))


def prepare_verify(x, t: W12Tensor, draft, argmax_out, accepted_out) -> Prepared:
    x = _as_bits(x)
    m = x.shape[0]
    n_draft = int(draft.numel())
    ws = workspace(workspace_bytes(OP_VERIFY, m, t.n, t.k), x.device, "verify")
    d = t.desc()
    args = (_ptr(x), m, ctypes.byref(d), _ptr(draft) if n_draft else None, n_draft,
            _ptr(argmax_out), _ptr(accepted_out), _ptr(ws), ws.numel(), _stream(x.device))
    return Prepared("w12_lmhead_verify", lib().w12_lmhead_verify, args,
                    (x, t, draft, argmax_out, accepted_out, ws, d))


def prepare_verify2(x, t: W12Tensor, sc: ScreenCopy, draft, argmax_out, accepted_out) -> Prepared:
    _check_screen(t, sc)
    x = _as_bits(x)
    m = x.shape[0]
    n_draft = int(draft.numel())
    ws = _verify2_ws(m, t, x.device)
    d = t.desc()
    args = (_ptr(x), m, ctypes.byref(d), _ptr(sc.buf), _ptr(draft) if n_draft else None, n_draft,
            _ptr(argmax_out), _ptr(accepted_out), _ptr(ws), ws.numel(), _stream(x.device))
    return Prepared("w12_lmhead_verify2", lib().w12_lmhead_verify2, args,
                    (x, t, sc, draft, argmax_out, accepted_out, ws, d))


def prepare_verify2_batched(x, t: W12Tensor, sc: ScreenCopy, req_off, req_ndraft, draft,
                            argmax_out, accepted_out) -> Prepared:
    args, keep = _batched2_args(x, t, sc, req_off, req_ndraft, draft, argmax_out, accepted_out)
    return Prepared("w12_lmhead_verify2_batched", lib().w12_lmhead_verify2_batched, args, keep)


def prepare_verify_batched(x, t: W12Tensor, req_off, req_ndraft, draft, argmax_out,
                           accepted_out) -> Prepared:
    args, keep = _batched_args(x, t, req_off, req_ndraft, draft, argmax_out, accepted_out)
    return Prepared("w12_lmhead_verify_batched", lib().w12_lmhead_verify_batched, args, keep)


class _PreparedOn(Prepared):
    """A prepared call that is issued with its tensors' device current."""

    def __init__(self, name: str, fn, args, keep, device):
        super().__init__(name, fn, args, keep)
        self._device = device

    def __call__(self):
        with _torch().cuda.device(self._device):
            super().__call__()


def _prepared(name: str, args, keep, device) -> Prepared:
    fn = getattr(lib(), name)
    if _torch().cuda.device_count() == 1:
        return Prepared(name, fn, args, keep)
    return _PreparedOn(name, fn, args, keep, device)


def prepare_kv_plan(pt: PageTable, length, req_off, kv_len, pos, slot) -> Prepared:
    """kv_plan of m = pos.numel() rows into kv_len, pos and slot."""
    args, keep = _plan_args(pt, length, req_off, kv_len, pos, slot)
    return _prepared("w12_kv_plan", args, keep, pt.device)


def prepare_qk_rope(q, k, v, cache: KvCache, rope: Rope, pos, slot, q_out) -> Prepared:
    args, keep = _rope_args(q, k, v, cache, rope, pos, slot, q_out)
    return _prepared("w12_qk_rope", args, keep, cache.device)


def prepare_attn_paged(q, cache: KvCache, table, kv_len, req_off, out, scale=None, ws=None) -> Prepared:
    """attn_paged into out.  A captured prepared call keeps its workspace, by default that of the
    stream it was prepared on: graphs that may run at the same time, or beside calls on that
    stream, are prepared with a ws of their own (attn_workspace)."""
    args, keep = _attn_args(q, cache, table, kv_len, req_off, out, scale, ws)
    return _prepared("w12_attn_paged", args, keep, cache.device)


def prepare_kv_fork(pt: PageTable, parent, length, req_off, kv_len, pos, slot, copies) -> Prepared:
    """kv_fork of m = pos.numel() rows into kv_len, pos, slot and copies."""
    args, keep = _fork_args(pt, parent, length, req_off, kv_len, pos, slot, copies)
    return _prepared("w12_kv_fork", args, keep, pt.device)


def prepare_kv_copy(caches, copies) -> Prepared:
    args, keep, dev = _copy_args(caches, copies)
    return _prepared("w12_kv_copy", args, keep, dev)


def prepare_kv_compact(pt: PageTable, first: int, moves, moved) -> Prepared:
    """kv_compact of moves.shape[0] pages from page first on."""
    args, keep = _compact_args(pt, first, moves, moved)
    return _prepared("w12_kv_compact", args, keep, pt.device)


def prepare_attn_shared(q, cache: KvCache, table, kv_len, req_off, grp_off, grp_len, out, scale=None,
                        ws=None) -> Prepared:
    """attn_shared into out.  As with prepare_attn_paged, graphs and streams that may run at the same
    time are prepared with a ws of their own (attn_shared_workspace)."""
    args, keep = _shared_args(q, cache, table, kv_len, req_off, grp_off, grp_len, out, scale, ws)
    return _prepared("w12_attn_shared", args, keep, cache.device)


def prepare_beam_select(logits, scores, grp_off, parent, token, score_out, ws=None) -> Prepared:
    """beam_select of k = parent.shape[1] pairs.  As with prepare_attn_paged, graphs and streams that may run
    at the same time are prepared with a ws of their own (beam_workspace)."""
    args, keep, dev = _beam_args(logits, scores, grp_off, parent, token, score_out, ws)
    return _prepared("w12_beam_select", args, keep, dev)
