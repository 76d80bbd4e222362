"""ctypes mirror of include/dsv4.h, dsv4_gqa.h and dsv4_loop.h, and the loader of the in-tree libdsv4.so.

Argument marshalling only: every step of the decode path runs in the library's CUDA kernels.
Importing this module fails loudly if the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libdsv4.so")

F32, BF16, FP8_DS_MLA, I8_ROWSCALE, MXFP4 = 0, 1, 2, 3, 4
E4M3_PAGE = 5  # per-head caches: e4m3 codes with one UE8M0 exponent per page and head
OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_BOUNDS, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
LATENT_DIM, VALUE_DIM, ROPE_DIM, FP8_DS_MLA_BYTES = 576, 512, 64, 656
ABI_VERSION = 3

vp, i32, i64, u32, f32, f64 = C.c_void_p, C.c_int32, C.c_int64, C.c_uint32, C.c_float, C.c_double


class KvInsertParams(C.Structure):
    _fields_ = [("struct_size", u32), ("kv_new", vp), ("kv_dtype", i32), ("slot_mapping", vp), ("cache", vp),
                ("cache_dtype", i32), ("T", i32), ("page_size", i32), ("num_pages", i64), ("positions", vp),
                ("cos_sin", vp), ("max_pos", i32), ("after_independent", i32)]


class QnormRopeKvInsertParams(C.Structure):
    _fields_ = [("struct_size", u32), ("q", vp), ("q_out", vp), ("H", i32), ("H_pad", i32), ("q_norm_weight", vp),
                ("apply_q_norm", i32), ("apply_q_rope", i32), ("eps", f32), ("kv_new", vp), ("slot_mapping", vp),
                ("cache", vp), ("cache_dtype", i32), ("page_size", i32), ("num_pages", i64),
                ("apply_kv_rope", i32), ("act_dtype", i32), ("T", i32), ("positions", vp), ("cos_sin", vp),
                ("max_pos", i32), ("after_independent", i32)]


class CompressUpdateParams(C.Structure):
    _fields_ = [("struct_size", u32), ("kv_score", vp), ("positions", vp), ("T", i32), ("B", i32),
                ("q_per_seq", i32), ("ratio", i32), ("coff", i32), ("state", vp), ("ape", vp),
                ("norm_weight", vp), ("eps", f32), ("cos_sin", vp), ("max_pos", i32), ("main_cache", vp),
                ("cache_dtype", i32), ("page_size", i32), ("num_pages", i64), ("block_table", vp),
                ("max_pages_per_seq", i32), ("after_independent", i32), ("wk", vp), ("ik_norm_weight", vp),
                ("ik_eps", f32), ("ik_dim", i32), ("ik_cache", vp), ("ik_dtype", i32), ("ik_num_pages", i64),
                ("ik_block_table", vp), ("ik_max_pages", i32)]


class IndexerTopkParams(C.Structure):
    _fields_ = [("struct_size", u32), ("q", vp), ("q_dtype", i32), ("weights", vp), ("k_cache", vp),
                ("k_dtype", i32), ("num_pages", i64), ("block_table", vp), ("max_pages_per_seq", i32),
                ("positions", vp), ("T", i32), ("B", i32), ("q_per_seq", i32), ("ratio", i32),
                ("n_heads", i32), ("head_dim", i32), ("topk", i32), ("page_size", i32), ("max_context", i32),
                ("topk_idx", vp), ("topk_score", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t),
                ("workspace_zeroed", i32), ("cand_blocks", vp), ("cand_block_size", i32), ("cand_topk", i32),
                ("cand_write", i32)]


class SparseMlaDecodeParams(C.Structure):
    _fields_ = [("struct_size", u32), ("q", vp), ("q_dtype", i32), ("T", i32), ("B", i32), ("q_per_seq", i32),
                ("H", i32), ("positions", vp), ("swa_cache", vp), ("swa_block_table", vp), ("swa_max_pages", i32),
                ("swa_num_pages", i64), ("main_cache", vp), ("main_block_table", vp), ("main_max_pages", i32),
                ("main_num_pages", i64), ("cache_dtype", i32), ("page_size", i32), ("ratio", i32),
                ("window", i32), ("topk_idx", vp), ("topk", i32), ("sink", vp), ("softmax_scale", f32),
                ("out", vp), ("out_dtype", i32), ("lse", vp), ("max_context", i32), ("workspace", vp),
                ("workspace_bytes", C.c_size_t)]


class GqaAppendParams(C.Structure):
    _fields_ = [("struct_size", u32), ("k_new", vp), ("v_new", vp), ("k_token_stride", i64), ("k_head_stride", i64),
                ("v_token_stride", i64), ("v_head_stride", i64), ("q", vp), ("q_out", vp), ("q_token_stride", i64),
                ("q_head_stride", i64), ("q_out_token_stride", i64), ("q_out_head_stride", i64), ("k_cache", vp),
                ("v_cache", vp), ("k_page_stride", i64), ("k_cache_head_stride", i64), ("k_row_stride", i64),
                ("v_page_stride", i64), ("v_cache_head_stride", i64), ("v_row_stride", i64), ("k_exp", vp),
                ("v_exp", vp), ("cache_dtype", i32), ("T", i32), ("B", i32), ("q_heads", i32), ("kv_heads", i32),
                ("head_dim", i32), ("page_size", i32), ("num_pages", i64), ("block_table", vp),
                ("max_pages_per_seq", i32), ("q_start", vp), ("kv_len", vp), ("max_q_len", i32), ("cos_sin", vp),
                ("max_pos", i32), ("rope_first", i32), ("rope_dim", i32), ("rope_halves", i32)]


class GqaAttentionParams(C.Structure):
    _fields_ = [("struct_size", u32), ("q", vp), ("q_token_stride", i64), ("q_head_stride", i64), ("k_cache", vp),
                ("v_cache", vp), ("k_page_stride", i64), ("k_cache_head_stride", i64), ("k_row_stride", i64),
                ("v_page_stride", i64), ("v_cache_head_stride", i64), ("v_row_stride", i64), ("k_exp", vp),
                ("v_exp", vp), ("cache_dtype", i32), ("T", i32), ("B", i32), ("q_heads", i32), ("kv_heads", i32),
                ("head_dim", i32), ("page_size", i32), ("num_pages", i64), ("block_table", vp),
                ("max_pages_per_seq", i32), ("q_start", vp), ("kv_len", vp), ("max_q_len", i32),
                ("max_kv_len", i32), ("softmax_scale", f32), ("causal", i32), ("prefix_len", vp), ("kv_start", vp),
                ("window", i32), ("softcap", f32), ("slopes", vp), ("sink", vp), ("out", vp), ("out_dtype", i32),
                ("lse", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


class RopeFreqsParams(C.Structure):
    _fields_ = [("struct_size", u32), ("rope_dim", i32), ("scaling", i32), ("theta", f64), ("factor", f64),
                ("original_len", f64), ("beta_fast", f64), ("beta_slow", f64), ("low_turns", f64), ("high_turns", f64)]


class RopeParams(C.Structure):
    _fields_ = [("struct_size", u32), ("x", vp), ("y", vp), ("x_token_stride", i64), ("x_head_stride", i64),
                ("y_token_stride", i64), ("y_head_stride", i64), ("x2", vp), ("y2", vp), ("x2_token_stride", i64),
                ("x2_head_stride", i64), ("y2_token_stride", i64), ("y2_head_stride", i64), ("heads", i32),
                ("heads2", i32), ("dtype", i32), ("T", i32), ("head_dim", i32), ("positions", vp), ("freqs", vp),
                ("rope_first", i32), ("rope_dim", i32), ("rope_halves", i32), ("inverse", i32), ("scale", f32)]


class RopeTableParams(C.Structure):
    _fields_ = [("struct_size", u32), ("table", vp), ("rows", i32), ("rope_dim", i32), ("first_position", i32),
                ("scale", f32), ("freqs", vp)]


class PlanCache(C.Structure):
    _fields_ = [("page_size", i32), ("ratio", i32), ("window", i32), ("max_pages_per_seq", i32), ("num_pages", i64),
                ("block_table", vp), ("held", vp), ("held_out", vp), ("first", vp), ("first_out", vp),
                ("free_pages", vp), ("free_count", vp), ("free_count_out", vp), ("slots", vp)]


PLAN_MAX_CACHES, PLAN_MAX_REQUESTS, PLAN_MAX_TOKENS = 4, 4096, 1 << 19


class BatchPlanParams(C.Structure):
    _fields_ = [("struct_size", u32), ("B", i32), ("T", i32), ("num_caches", i32), ("ctx", vp), ("ctx_add", vp),
                ("n_new", vp), ("ctx_out", vp), ("q_start", vp), ("kv_len", vp), ("positions", vp),
                ("token_seq", vp), ("caches", PlanCache * PLAN_MAX_CACHES)]


class DraftVerifyParams(C.Structure):
    _fields_ = [("struct_size", u32), ("target", vp), ("target_stride", i64), ("target_dtype", i32),
                ("target_probs", i32), ("draft", vp), ("draft_stride", i64), ("draft_rows", i64),
                ("draft_dtype", i32), ("draft_probs", i32), ("draft_row", vp), ("tokens", vp), ("q_start", vp),
                ("T", i32), ("B", i32), ("vocab", i32), ("max_q_len", i32), ("temperature", vp), ("u", vp),
                ("noise", vp), ("noise_stride", i64), ("out_tokens", vp), ("n_out", vp), ("logp", vp)]


EXPORTS = ["dsv4_kv_insert", "dsv4_compress_update", "dsv4_indexer_topk_workspace_bytes", "dsv4_indexer_topk",
           "dsv4_sparse_mla_decode_workspace_bytes", "dsv4_sparse_mla_decode", "dsv4_abi_version",
           "dsv4_status_string", "dsv4_last_cuda_error", "dsv4_read_device_flags", "dsv4_indexer_topk_noalloc",
           "dsv4_qnorm_rope_kv_insert", "dsv4_padded_num_q_heads", "dsv4_kernel_launches"]

# the grouped-query calls (include/dsv4_gqa.h)
GQA_EXPORTS = ["dsv4_gqa_append", "dsv4_gqa_attention_workspace_bytes", "dsv4_gqa_attention"]

# the calls around the layers (include/dsv4_loop.h)
LOOP_EXPORTS = ["dsv4_rope_freqs", "dsv4_rope", "dsv4_rope_table", "dsv4_batch_plan", "dsv4_draft_verify"]
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "yarn": 3, "bands": 4}

# bytes of the scratch array built into the library for dsv4_indexer_topk_noalloc
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024

_lib = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Loads libdsv4.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libdsv4.so is not built ({path}); run __graft_entry__.build() or "
                           "python -m deepseek_v4_hybrid_gb300.build")
    lib = C.CDLL(path)
    for name, st in (("dsv4_kv_insert", KvInsertParams), ("dsv4_compress_update", CompressUpdateParams),
                     ("dsv4_qnorm_rope_kv_insert", QnormRopeKvInsertParams),
                     ("dsv4_indexer_topk", IndexerTopkParams), ("dsv4_sparse_mla_decode", SparseMlaDecodeParams),
                     ("dsv4_indexer_topk_noalloc", IndexerTopkParams), ("dsv4_gqa_append", GqaAppendParams),
                     ("dsv4_gqa_attention", GqaAttentionParams), ("dsv4_rope", RopeParams),
                     ("dsv4_rope_table", RopeTableParams), ("dsv4_batch_plan", BatchPlanParams),
                     ("dsv4_draft_verify", DraftVerifyParams)):
        fn = getattr(lib, name)
        fn.argtypes = [C.POINTER(st), vp]
        fn.restype = C.c_int
    for name, st in (("dsv4_indexer_topk_workspace_bytes", IndexerTopkParams),
                     ("dsv4_sparse_mla_decode_workspace_bytes", SparseMlaDecodeParams),
                     ("dsv4_gqa_attention_workspace_bytes", GqaAttentionParams)):
        fn = getattr(lib, name)
        fn.argtypes = [C.POINTER(st)]
        fn.restype = C.c_size_t
    lib.dsv4_rope_freqs.argtypes = [C.POINTER(RopeFreqsParams), C.POINTER(C.c_uint64)]
    lib.dsv4_rope_freqs.restype = C.c_int
    lib.dsv4_padded_num_q_heads.argtypes = [C.c_int, C.c_int]
    lib.dsv4_padded_num_q_heads.restype = C.c_int
    lib.dsv4_abi_version.restype = C.c_int
    lib.dsv4_status_string.argtypes = [C.c_int]
    lib.dsv4_status_string.restype = C.c_char_p
    lib.dsv4_last_cuda_error.restype = C.c_int
    lib.dsv4_kernel_launches.argtypes = []
    lib.dsv4_kernel_launches.restype = C.c_uint64
    lib.dsv4_read_device_flags.argtypes = [C.POINTER(u32)]
    lib.dsv4_read_device_flags.restype = C.c_int
    if lib.dsv4_abi_version() != ABI_VERSION:
        raise RuntimeError("libdsv4.so ABI version mismatch")
    _lib = lib
    return lib


def make(struct_type, **fields):
    s = struct_type()
    s.struct_size = C.sizeof(struct_type)
    for k, v in fields.items():
        setattr(s, k, v)
    return s


class Dsv4Error(RuntimeError):
    def __init__(self, call: str, status: int):
        lib = load()
        msg = lib.dsv4_status_string(status).decode()
        if status == ERR_CUDA:
            msg += f" (cudaError {lib.dsv4_last_cuda_error()})"
        super().__init__(f"{call}: {msg}")
        self.status = status


def check(call: str, status: int) -> None:
    if status != OK:
        raise Dsv4Error(call, status)
