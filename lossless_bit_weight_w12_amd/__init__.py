"""W12 on MI355X: lossless 12-bit BF16 weights decoded inside the GEMM, plus greedy
verification with a certified exact-argmax LM head, in one pass over the W12 head or in
two levels (an 8-bit screen copy first), the GEMMs of FP8 targets (E4M3 weights with
128 x 128 block scales) in the same kernel family, and the attention side of a decode step
(block tables, norm and rotation with the cache append, attention over the paged cache), also of
several continuations of one prompt (shared pages and their copies, attention that reads shared
tokens once, the choice of beams).
The compute lives in libw12.so (HIP kernels for gfx950 behind a C ABI, declared in
include/w12.h); this package is its thin Python binding."""
from .w12 import (ATTN_WS_BYTES, ENCODE_TOTAL_OFFSET, EXPORTS, F8Tensor, KV_BF16, KV_E4M3,
                  KvCache, LOGITS_BF16, LOGITS_F32, MAX_BEAMS, MAX_BEAM_K, MAX_COPIES,
                  MAX_GROUP, MAX_HEADS, MAX_KV_ROWS, MAX_LAYERS, MAX_M, MAX_REQ,
                  MAX_SHARED_ROWS, MAX_VOCAB, NOALLOC_SCRATCH_BYTES, OP_DECODE, OP_ENCODE,
                  OP_GEMM, OP_GEMM_BF16, OP_GEMM_F8, OP_GEMM_GROUP, OP_VERIFY, OP_VERIFY2,
                  PageTable, Prepared, Rope, ScreenCopy, W12Desc, W12Error, W12Tensor,
                  attn_paged, attn_shared, attn_shared_workspace, attn_workspace, beam_select,
                  beam_workspace, bf16_tile, decode, encode, f8_encode, f8_tile, gemm,
                  gemm_bf16, gemm_bf16_tiled, gemm_f8, gemm_f8_group, gemm_group, gemm_noalloc,
                  kv_cache, kv_compact, kv_copy, kv_fork, kv_plan, lib, lib_path, lmhead_verify,
                  lmhead_verify2, lmhead_verify2_batched, lmhead_verify_batched, logits_f32,
                  page_refs, page_table, prepare_attn_paged, prepare_attn_shared,
                  prepare_beam_select, prepare_gemm, prepare_gemm_f8, prepare_gemm_f8_group,
                  prepare_gemm_group, prepare_kv_compact, prepare_kv_copy, prepare_kv_fork,
                  prepare_kv_plan, prepare_qk_rope, prepare_rms, prepare_verify,
                  prepare_verify2, prepare_verify2_batched, prepare_verify_batched, qk_rope,
                  rms_rescale, screen_encode, screen_logits_f32, status_str, stream_read,
                  tiles_bytes, verify2_candidates, verify_candidates, workspace,
                  workspace_bytes)

__all__ = ["ATTN_WS_BYTES", "ENCODE_TOTAL_OFFSET", "EXPORTS", "F8Tensor", "KV_BF16", "KV_E4M3",
           "KvCache", "LOGITS_BF16", "LOGITS_F32", "MAX_BEAMS", "MAX_BEAM_K", "MAX_COPIES",
           "MAX_GROUP", "MAX_HEADS", "MAX_KV_ROWS", "MAX_LAYERS", "MAX_M", "MAX_REQ",
           "MAX_SHARED_ROWS", "MAX_VOCAB", "NOALLOC_SCRATCH_BYTES", "OP_DECODE", "OP_ENCODE",
           "OP_GEMM", "OP_GEMM_BF16", "OP_GEMM_F8", "OP_GEMM_GROUP", "OP_VERIFY", "OP_VERIFY2",
           "PageTable", "Prepared", "Rope", "ScreenCopy", "W12Desc", "W12Error", "W12Tensor",
           "attn_paged", "attn_shared", "attn_shared_workspace", "attn_workspace",
           "beam_select", "beam_workspace", "bf16_tile", "decode", "encode", "f8_encode",
           "f8_tile", "gemm", "gemm_bf16", "gemm_bf16_tiled", "gemm_f8", "gemm_f8_group",
           "gemm_group", "gemm_noalloc", "kv_cache", "kv_compact", "kv_copy", "kv_fork",
           "kv_plan", "lib", "lib_path", "lmhead_verify", "lmhead_verify2",
           "lmhead_verify2_batched", "lmhead_verify_batched", "logits_f32", "page_refs",
           "page_table", "prepare_attn_paged", "prepare_attn_shared", "prepare_beam_select",
           "prepare_gemm", "prepare_gemm_f8", "prepare_gemm_f8_group", "prepare_gemm_group",
           "prepare_kv_compact", "prepare_kv_copy", "prepare_kv_fork", "prepare_kv_plan",
           "prepare_qk_rope", "prepare_rms", "prepare_verify", "prepare_verify2",
           "prepare_verify2_batched", "prepare_verify_batched", "qk_rope", "rms_rescale",
           "screen_encode", "screen_logits_f32", "status_str", "stream_read", "tiles_bytes",
           "verify2_candidates", "verify_candidates", "workspace", "workspace_bytes"]
