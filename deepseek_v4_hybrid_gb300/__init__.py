"""DeepSeek-V4 hybrid compressed-attention decode step on one GB300 (sm_103a).

Thin Python binding of libdsv4.so (include/dsv4.h, dsv4_gqa.h, dsv4_loop.h).  The functions below take torch CUDA tensors,
fill the C parameter structs and call the library on the current torch stream; every step of the
decode path runs in the library's CUDA kernels.  There is no CPU fallback: the import fails if
the library is not built.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _abi
from ._abi import BF16, E4M3_PAGE, F32, FP8_DS_MLA, I8_ROWSCALE, MXFP4, Dsv4Error  # noqa: F401

_lib = _abi.load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    # (the handle itself: making a stream object of it costs more than a kernel's launch, 2.8 us of a call's 5.9)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def dsv4_kv_insert(kv_new, kv_dtype, slot_mapping, cache, cache_dtype, page_size, positions=None, cos_sin=None,
                   stream=None, after_independent=False):
    """Writes kv_new[T, 576] into the paged SWA cache at slot_mapping[T] (int64, -1 skips).
    after_independent: see include/dsv4.h (the kernel before it on the stream touches nothing this call does)."""
    T = slot_mapping.shape[0]
    p = _abi.make(_abi.KvInsertParams, kv_new=_ptr(kv_new), kv_dtype=kv_dtype, slot_mapping=_ptr(slot_mapping),
                  cache=_ptr(cache), cache_dtype=cache_dtype, T=T, page_size=page_size,
                  num_pages=cache.shape[0], positions=_ptr(positions), cos_sin=_ptr(cos_sin),
                  max_pos=0 if cos_sin is None else cos_sin.shape[0], after_independent=int(after_independent))
    _abi.check("dsv4_kv_insert", _lib.dsv4_kv_insert(p, _stream(stream)))


def dsv4_qnorm_rope_kv_insert(q, q_out, act_dtype, kv_new, slot_mapping, cache, cache_dtype, page_size, positions,
                              cos_sin, q_norm_weight=None, eps=1e-6, apply_q_norm=True, apply_q_rope=True,
                              apply_kv_rope=True, stream=None, after_independent=False):
    """Per-head RMSNorm + GPT-J RoPE of q[T, H, 576] into q_out[T, H_pad, 576] (heads >= H zero) and the
    kv rows' RoPE + store into the paged SWA cache, in one launch (see include/dsv4.h)."""
    T, H, _ = q.shape
    p = _abi.make(_abi.QnormRopeKvInsertParams, q=_ptr(q), q_out=_ptr(q_out), H=H, H_pad=q_out.shape[1],
                  q_norm_weight=_ptr(q_norm_weight), apply_q_norm=int(apply_q_norm), apply_q_rope=int(apply_q_rope),
                  eps=eps, kv_new=_ptr(kv_new), slot_mapping=_ptr(slot_mapping), cache=_ptr(cache),
                  cache_dtype=cache_dtype, page_size=page_size, num_pages=cache.shape[0],
                  apply_kv_rope=int(apply_kv_rope), act_dtype=act_dtype, T=T, positions=_ptr(positions),
                  cos_sin=_ptr(cos_sin), max_pos=0 if cos_sin is None else cos_sin.shape[0],
                  after_independent=int(after_independent))
    _abi.check("dsv4_qnorm_rope_kv_insert", _lib.dsv4_qnorm_rope_kv_insert(p, _stream(stream)))


def dsv4_padded_num_q_heads(H, cache_dtype) -> int:
    """Query heads the attention's q and output buffers hold for H heads with this cache dtype."""
    n = int(_lib.dsv4_padded_num_q_heads(int(H), int(cache_dtype)))
    if n < 0:
        raise ValueError(f"no padded head count for H={H}, cache dtype {cache_dtype}")
    return n


def dsv4_compress_update(kv_score, positions, q_per_seq, ratio, coff, state, ape, norm_weight, eps, cos_sin,
                         main_cache, cache_dtype, block_table, page_size, stream=None, after_independent=False,
                         wk=None, ik_norm_weight=None, ik_eps=1e-6, ik_cache=None, ik_dtype=BF16,
                         ik_block_table=None):
    """Compressor state store + fold of the new tokens, and (with wk) the index key of every new entry
    into the indexer cache (see include/dsv4.h)."""
    T = positions.shape[0]
    p = _abi.make(_abi.CompressUpdateParams, kv_score=_ptr(kv_score), positions=_ptr(positions), T=T,
                  B=T // q_per_seq, q_per_seq=q_per_seq, ratio=ratio, coff=coff, state=_ptr(state), ape=_ptr(ape),
                  norm_weight=_ptr(norm_weight), eps=eps, cos_sin=_ptr(cos_sin), max_pos=cos_sin.shape[0],
                  main_cache=_ptr(main_cache), cache_dtype=cache_dtype, page_size=page_size,
                  num_pages=main_cache.shape[0], block_table=_ptr(block_table),
                  max_pages_per_seq=block_table.shape[1], after_independent=int(after_independent))
    if wk is not None:
        p.wk, p.ik_norm_weight, p.ik_eps, p.ik_dim = _ptr(wk), _ptr(ik_norm_weight), ik_eps, wk.shape[0]
        p.ik_cache, p.ik_dtype, p.ik_num_pages = _ptr(ik_cache), ik_dtype, ik_cache.shape[0]
        p.ik_block_table, p.ik_max_pages = _ptr(ik_block_table), ik_block_table.shape[1]
    _abi.check("dsv4_compress_update", _lib.dsv4_compress_update(p, _stream(stream)))


def indexer_topk_params(q, q_dtype, weights, k_cache, k_dtype, block_table, positions, q_per_seq, ratio, topk,
                        page_size, max_context, topk_idx=None, topk_score=None, workspace=None, cand_blocks=None,
                        cand_block_size=0, cand_write=False):
    """Parameter struct of dsv4_indexer_topk.  cand_blocks ([T, cand_topk] int32) with cand_block_size > 0
    turns on two-level candidate filtering: read by a consumer, written by the source (cand_write)."""
    T, n_heads, head_dim = q.shape
    return _abi.make(_abi.IndexerTopkParams, q=_ptr(q), q_dtype=q_dtype, weights=_ptr(weights),
                     k_cache=_ptr(k_cache), k_dtype=k_dtype, num_pages=k_cache.shape[0],
                     block_table=_ptr(block_table), max_pages_per_seq=block_table.shape[1],
                     positions=_ptr(positions), T=T, B=T // q_per_seq, q_per_seq=q_per_seq, ratio=ratio,
                     n_heads=n_heads, head_dim=head_dim, topk=topk, page_size=page_size, max_context=max_context,
                     topk_idx=_ptr(topk_idx), topk_score=_ptr(topk_score), workspace=_ptr(workspace),
                     workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size(),
                     cand_blocks=_ptr(cand_blocks), cand_block_size=cand_block_size if cand_blocks is not None else 0,
                     cand_topk=0 if cand_blocks is None else cand_blocks.shape[1], cand_write=int(cand_write))


def dsv4_indexer_topk_workspace_bytes(params) -> int:
    return int(_lib.dsv4_indexer_topk_workspace_bytes(params))


def dsv4_indexer_topk(params, stream=None):
    """Lightning-Indexer scores + per-query top-k into params.topk_idx (see include/dsv4.h)."""
    _abi.check("dsv4_indexer_topk", _lib.dsv4_indexer_topk(params, _stream(stream)))


def sparse_mla_params(q, q_dtype, positions, q_per_seq, swa_cache, swa_block_table, main_cache, main_block_table,
                      cache_dtype, page_size, ratio, window, topk_idx, sink, softmax_scale, out, out_dtype, lse,
                      max_context, workspace=None):
    T, H, _ = q.shape
    return _abi.make(_abi.SparseMlaDecodeParams, q=_ptr(q), q_dtype=q_dtype, T=T, B=T // q_per_seq,
                     q_per_seq=q_per_seq, H=H, positions=_ptr(positions), swa_cache=_ptr(swa_cache),
                     swa_block_table=_ptr(swa_block_table), swa_max_pages=swa_block_table.shape[1],
                     swa_num_pages=swa_cache.shape[0], main_cache=_ptr(main_cache),
                     main_block_table=_ptr(main_block_table),
                     main_max_pages=0 if main_block_table is None else main_block_table.shape[1],
                     main_num_pages=0 if main_cache is None else main_cache.shape[0], cache_dtype=cache_dtype,
                     page_size=page_size, ratio=ratio, window=window, topk_idx=_ptr(topk_idx),
                     topk=0 if topk_idx is None else topk_idx.shape[1], sink=_ptr(sink),
                     softmax_scale=softmax_scale, out=_ptr(out), out_dtype=out_dtype, lse=_ptr(lse),
                     max_context=max_context, workspace=_ptr(workspace),
                     workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size())


def dsv4_sparse_mla_decode_workspace_bytes(params) -> int:
    return int(_lib.dsv4_sparse_mla_decode_workspace_bytes(params))


def dsv4_sparse_mla_decode(params, stream=None):
    """Shared-KV sparse MLA decode attention into params.out (see include/dsv4.h)."""
    _abi.check("dsv4_sparse_mla_decode", _lib.dsv4_sparse_mla_decode(params, _stream(stream)))


# ---------------------------------------------------------------------------------------------------------
# grouped-query operators (include/dsv4_gqa.h).  The parameter structs are built once over fixed buffers
# (they keep their tensors alive) and passed to any number of calls; the calls run on the tensors' device.
# ---------------------------------------------------------------------------------------------------------
def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _need_tensor(t, name, dtypes, shape, device):
    """t is a tensor of one of dtypes on device; shape entries of None are free; the last dim is contiguous."""
    _need(isinstance(t, torch.Tensor) and t.dtype in dtypes, f"{name}: dtype {getattr(t, 'dtype', type(t))} is none of {dtypes}")
    _need(t.dim() == len(shape) and all(w is None or s == w for s, w in zip(t.shape, shape)),
          f"{name}: shape {tuple(t.shape)}, wanted {tuple('*' if w is None else w for w in shape)}")
    _need(t.device == device, f"{name}: on {t.device}, wanted {device}")
    _need(t.numel() == 0 or t.shape[-1] == 1 or t.stride(-1) == 1, f"{name}: the last dimension is not contiguous")


def _need_flat(t, name, dtype, shape, device):
    _need_tensor(t, name, (dtype,), shape, device)
    _need(t.is_contiguous(), f"{name}: not contiguous")


def _gqa_common(k_cache, v_cache, k_scale, v_scale, block_table, q_start, kv_len, max_q_len):
    """Fields that both grouped-query calls share."""
    dev = k_cache.device
    _need(dev.type == "cuda", f"k_cache: on {dev}, wanted a CUDA device")
    e4m3 = (torch.uint8, torch.float8_e4m3fn)
    scaled = k_cache.dtype in e4m3
    _need_tensor(k_cache, "k_cache", e4m3 if scaled else (torch.bfloat16,), (None,) * 4, dev)
    pages, heads, page_size, dim = k_cache.shape
    _need_tensor(v_cache, "v_cache", e4m3 if scaled else (torch.bfloat16,), (pages, heads, page_size, dim), dev)
    _need((k_scale is not None) == scaled and (v_scale is not None) == scaled,
          "k_scale and v_scale go with an e4m3 cache, and only with one")
    if scaled:
        _need_flat(k_scale, "k_scale", torch.uint8, (pages, heads), dev)
        _need_flat(v_scale, "v_scale", torch.uint8, (pages, heads), dev)
    _need_flat(kv_len, "kv_len", torch.int32, (None,), dev)
    B = kv_len.shape[0]
    _need_flat(q_start, "q_start", torch.int32, (B + 1,), dev)
    _need_flat(block_table, "block_table", torch.int32, (B, None), dev)
    ks, vs = k_cache.stride(), v_cache.stride()
    return dev, dict(k_cache=_ptr(k_cache), v_cache=_ptr(v_cache), k_page_stride=ks[0], k_cache_head_stride=ks[1],
                     k_row_stride=ks[2], v_page_stride=vs[0], v_cache_head_stride=vs[1], v_row_stride=vs[2],
                     k_exp=_ptr(k_scale), v_exp=_ptr(v_scale), cache_dtype=E4M3_PAGE if scaled else BF16, B=B,
                     kv_heads=heads, head_dim=dim, page_size=page_size, num_pages=pages,
                     block_table=_ptr(block_table), max_pages_per_seq=block_table.shape[1], q_start=_ptr(q_start),
                     kv_len=_ptr(kv_len), max_q_len=max_q_len)


def gqa_append_params(k_new, v_new, k_cache, v_cache, block_table, q_start, kv_len, max_q_len, k_scale=None,
                      v_scale=None, cos_sin=None, rope_first=0, rope_halves=False, q=None, q_out=None):
    """Parameter struct of dsv4_gqa_append.  k_new, v_new [T, kv_heads, dim] and q, q_out [T, q_heads, dim] bf16,
    rows of any strides (slices of a fused projection); caches [pages, kv_heads, page_size, dim] in any order
    of the first three, bf16, or e4m3 codes (uint8 or float8_e4m3fn) with k_scale, v_scale [pages, kv_heads] of
    UE8M0 bytes; q_start [B + 1], kv_len [B] (rows including the new ones), block_table [B, n] int32;
    cos_sin [max_pos, rope_dim] fp32 rotates keys and queries (rope_halves: pairs (i, i + rope_dim / 2))."""
    dev, f = _gqa_common(k_cache, v_cache, k_scale, v_scale, block_table, q_start, kv_len, max_q_len)
    act, heads, dim = (torch.bfloat16,), f["kv_heads"], f["head_dim"]
    _need_tensor(k_new, "k_new", act, (None, heads, dim), dev)
    T = k_new.shape[0]
    _need_tensor(v_new, "v_new", act, (T, heads, dim), dev)
    _need((q is None) == (q_out is None), "q and q_out go together")
    p = _abi.make(_abi.GqaAppendParams, T=T, k_new=_ptr(k_new), v_new=_ptr(v_new), k_token_stride=k_new.stride(0),
                  k_head_stride=k_new.stride(1), v_token_stride=v_new.stride(0), v_head_stride=v_new.stride(1),
                  q_heads=1, **f)
    if q is not None:
        _need_tensor(q, "q", act, (T, None, dim), dev)
        _need_tensor(q_out, "q_out", act, (T, q.shape[1], dim), dev)
        p.q, p.q_out, p.q_heads = _ptr(q), _ptr(q_out), q.shape[1]
        p.q_token_stride, p.q_head_stride = q.stride(0), q.stride(1)
        p.q_out_token_stride, p.q_out_head_stride = q_out.stride(0), q_out.stride(1)
    if cos_sin is not None:
        _need_flat(cos_sin, "cos_sin", torch.float32, (None, None), dev)
        p.cos_sin, p.max_pos, p.rope_dim = _ptr(cos_sin), cos_sin.shape[0], cos_sin.shape[1]
        p.rope_first, p.rope_halves = rope_first, int(rope_halves)
    p.device = dev
    p.tensors = (k_new, v_new, k_cache, v_cache, block_table, q_start, kv_len, k_scale, v_scale, cos_sin, q, q_out)
    return p


def gqa_attention_params(q, k_cache, v_cache, block_table, q_start, kv_len, max_q_len, max_kv_len, softmax_scale, out,
                         lse=None, k_scale=None, v_scale=None, causal=True, prefix_len=None, kv_start=None, window=0,
                         softcap=0.0, slopes=None, sink=None, workspace=None):
    """Parameter struct of dsv4_gqa_attention (caches and batch as in gqa_append_params).  q [T, q_heads, dim]
    bf16 of any strides; out [T, q_heads, dim] bf16 or fp32 and lse [T, q_heads] fp32, contiguous; prefix_len [B]
    and kv_start [T] int32; slopes and sink [q_heads] fp32."""
    dev, f = _gqa_common(k_cache, v_cache, k_scale, v_scale, block_table, q_start, kv_len, max_q_len)
    dim = f["head_dim"]
    _need_tensor(q, "q", (torch.bfloat16,), (None, None, dim), dev)
    T, H, _ = q.shape
    _need(out.dtype in (torch.bfloat16, torch.float32), f"out: dtype {out.dtype}")
    _need_flat(out, "out", out.dtype, (T, H, dim), dev)
    for t, name, dt, shape in ((lse, "lse", torch.float32, (T, H)), (prefix_len, "prefix_len", torch.int32, (f["B"],)),
                               (kv_start, "kv_start", torch.int32, (T,)), (slopes, "slopes", torch.float32, (H,)),
                               (sink, "sink", torch.float32, (H,))):
        if t is not None:
            _need_flat(t, name, dt, shape, dev)
    p = _abi.make(_abi.GqaAttentionParams, q=_ptr(q), q_token_stride=q.stride(0), q_head_stride=q.stride(1), T=T,
                  q_heads=H, max_kv_len=max_kv_len, softmax_scale=softmax_scale, causal=int(causal),
                  prefix_len=_ptr(prefix_len), kv_start=_ptr(kv_start), window=window, softcap=softcap,
                  slopes=_ptr(slopes), sink=_ptr(sink), out=_ptr(out),
                  out_dtype=BF16 if out.dtype == torch.bfloat16 else F32, lse=_ptr(lse), **f)
    p.device = dev
    p.tensors = (q, k_cache, v_cache, block_table, q_start, kv_len, out, lse, k_scale, v_scale, prefix_len, kv_start,
                 slopes, sink)
    if workspace is not None:
        gqa_set_workspace(p, workspace)
    return p


def dsv4_gqa_attention_workspace_bytes(params) -> int:
    with torch.cuda.device(params.device):
        n = int(_lib.dsv4_gqa_attention_workspace_bytes(params))
    if n == 0:  # refused: the call itself says why
        _abi.check("dsv4_gqa_attention_workspace_bytes", _abi.ERR_INVALID)
    return n


def gqa_set_workspace(params, workspace):
    """Gives the params a workspace (a tensor of at least dsv4_gqa_attention_workspace_bytes(params) bytes).  Calls
    that may overlap on the GPU need one each."""
    _need(workspace.device == params.device and workspace.is_contiguous(), "workspace: wrong device, or not contiguous")
    params.workspace, params.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    params.workspace_tensor = workspace


def _call(name, fn, params, stream):
    dev = params.device
    if dev.index is not None and dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = fn(params, _stream(stream))
    else:
        status = fn(params, _stream(stream))
    _abi.check(name, status)


def dsv4_gqa_append(params, stream=None):
    """Rotates and stores the new tokens' keys and values, and rotates their queries (see include/dsv4_gqa.h)."""
    _call("dsv4_gqa_append", _lib.dsv4_gqa_append, params, stream)


def dsv4_gqa_attention(params, stream=None):
    """Attention of the new tokens over the paged per-head caches into params' out and lse (see include/dsv4_gqa.h)."""
    _call("dsv4_gqa_attention", _lib.dsv4_gqa_attention, params, stream)


# ---------------------------------------------------------------------------------------------------------
# what surrounds the layers of a decode step (include/dsv4_loop.h): like the grouped-query calls, over parameter
# structs that are built once and keep their tensors alive.
# ---------------------------------------------------------------------------------------------------------
def rope_freqs(rope_dim, theta=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0,
               low_turns=1.0, high_turns=4.0, device="cuda"):
    """Frequencies of rope_params and rope_table_params: [rope_dim / 2] int64 on the device, scaled for long contexts
    by "none", "linear", "base", "yarn" or "bands" (see include/dsv4_loop.h)."""
    _need(scaling in _abi.ROPE_SCALINGS, f"scaling: {scaling!r} is none of {tuple(_abi.ROPE_SCALINGS)}")
    _need(isinstance(rope_dim, int) and 2 <= rope_dim <= 1024, f"rope_dim: {rope_dim}")
    out = torch.empty(rope_dim // 2, dtype=torch.int64)
    p = _abi.make(_abi.RopeFreqsParams, rope_dim=rope_dim, scaling=_abi.ROPE_SCALINGS[scaling], theta=theta,
                  factor=factor, original_len=original_len, beta_fast=beta_fast, beta_slow=beta_slow,
                  low_turns=low_turns, high_turns=high_turns)
    _abi.check("dsv4_rope_freqs", _lib.dsv4_rope_freqs(p, C.cast(out.data_ptr(), C.POINTER(C.c_uint64))))
    return out.to(device)


def _act(t, name):
    _need(isinstance(t, torch.Tensor) and t.dtype in (torch.bfloat16, torch.float32),
          f"{name}: dtype {getattr(t, 'dtype', type(t))} is neither bfloat16 nor float32")
    _need(t.device.type == "cuda", f"{name}: on {t.device}, wanted a CUDA device")
    return BF16 if t.dtype == torch.bfloat16 else F32


def rope_params(x, out, positions, freqs, x2=None, out2=None, rope_first=0, rope_halves=False, inverse=False,
                scale=1.0):
    """Parameter struct of dsv4_rope.  x, out [T, heads, dim] and x2, out2 [T, heads2, dim] bf16 or fp32, rows of
    any strides (slices of a fused projection); out is x itself (in place) or apart; positions [T] int32 (negative:
    skipped); freqs of rope_freqs; inverse turns back (the gradient)."""
    dt, dev = _act(x, "x"), x.device
    _need(x.dim() == 3, f"x: shape {tuple(x.shape)}, wanted three dimensions")
    T, heads, dim = x.shape
    _need((x2 is None) == (out2 is None), "x2 and out2 go together")
    _need_tensor(x, "x", (x.dtype,), (T, heads, dim), dev)
    _need_tensor(out, "out", (x.dtype,), (T, heads, dim), dev)
    _need_flat(positions, "positions", torch.int32, (T,), dev)
    _need_flat(freqs, "freqs", torch.int64, (None,), dev)
    p = _abi.make(_abi.RopeParams, x=_ptr(x), y=_ptr(out), x_token_stride=x.stride(0), x_head_stride=x.stride(1),
                  y_token_stride=out.stride(0), y_head_stride=out.stride(1), heads=heads, heads2=1, dtype=dt, T=T,
                  head_dim=dim, positions=_ptr(positions), freqs=_ptr(freqs), rope_first=rope_first,
                  rope_dim=2 * freqs.shape[0], rope_halves=int(rope_halves), inverse=int(inverse), scale=scale)
    if x2 is not None:
        _need_tensor(x2, "x2", (x.dtype,), (T, None, dim), dev)
        _need_tensor(out2, "out2", (x.dtype,), (T, x2.shape[1], dim), dev)
        p.x2, p.y2, p.heads2 = _ptr(x2), _ptr(out2), x2.shape[1]
        p.x2_token_stride, p.x2_head_stride = x2.stride(0), x2.stride(1)
        p.y2_token_stride, p.y2_head_stride = out2.stride(0), out2.stride(1)
    p.device = dev
    p.tensors = (x, out, positions, freqs, x2, out2)
    return p


def dsv4_rope(params, stream=None):
    """Turns rows by their tokens' positions (see include/dsv4_loop.h)."""
    _call("dsv4_rope", _lib.dsv4_rope, params, stream)


def rope_table_params(table, freqs, first_position=0, scale=1.0):
    """Parameter struct of dsv4_rope_table: table [rows, rope_dim] fp32 becomes the cos_sin table of the positions from
    first_position on."""
    _need(isinstance(table, torch.Tensor) and table.device.type == "cuda", "table: wanted a tensor on a CUDA device")
    _need_flat(freqs, "freqs", torch.int64, (None,), table.device)
    _need_flat(table, "table", torch.float32, (None, 2 * freqs.shape[0]), table.device)
    p = _abi.make(_abi.RopeTableParams, table=_ptr(table), rows=table.shape[0], rope_dim=table.shape[1],
                  first_position=first_position, scale=scale, freqs=_ptr(freqs))
    p.device = table.device
    p.tensors = (table, freqs)
    return p


def dsv4_rope_table(params, stream=None):
    """Writes a cos_sin table (see include/dsv4_loop.h)."""
    _call("dsv4_rope_table", _lib.dsv4_rope_table, params, stream)


def plan_cache(block_table, held, free_pages, free_count, page_size, held_out=None, free_count_out=None, ratio=1,
               window=0, first=None, first_out=None, slots=None):
    """One paged cache of batch_plan_params: block_table [B, n], held [B], free_pages [num_pages] and free_count [1] int32;
    window: with first [B], the begin of each request's table entries; slots [T] int64.  The outputs are
    the inputs themselves where they are not given (held, first and free_count then advance in place)."""
    held_out = held if held_out is None else held_out
    free_count_out = free_count if free_count_out is None else free_count_out
    first_out = first if first_out is None else first_out
    _need(isinstance(block_table, torch.Tensor) and block_table.device.type == "cuda",
          "block_table: wanted a tensor on a CUDA device")
    dev = block_table.device
    _need_flat(block_table, "block_table", torch.int32, (None, None), dev)
    B = block_table.shape[0]
    for t, name in ((held, "held"), (held_out, "held_out"), (first, "first"), (first_out, "first_out")):
        if t is not None or name.startswith("held"):
            _need_flat(t, name, torch.int32, (B,), dev)
    _need_flat(free_pages, "free_pages", torch.int32, (None,), dev)
    _need_flat(free_count, "free_count", torch.int32, (1,), dev)
    _need_flat(free_count_out, "free_count_out", torch.int32, (1,), dev)
    if slots is not None:
        _need_flat(slots, "slots", torch.int64, (None,), dev)
    c = _abi.PlanCache(page_size=page_size, ratio=ratio, window=window, max_pages_per_seq=block_table.shape[1],
                       num_pages=free_pages.shape[0], block_table=_ptr(block_table), held=_ptr(held),
                       held_out=_ptr(held_out), first=_ptr(first), first_out=_ptr(first_out),
                       free_pages=_ptr(free_pages), free_count=_ptr(free_count), free_count_out=_ptr(free_count_out),
                       slots=_ptr(slots))
    c.shape, c.device = (B, None if slots is None else slots.shape[0]), dev
    c.tensors = (block_table, held, held_out, first, first_out, free_pages, free_count, free_count_out, slots)
    return c


def batch_plan_params(ctx, n_new, q_start, kv_len, caches, ctx_add=None, ctx_out=None, positions=None, token_seq=None,
                      max_tokens=None):
    """Parameter struct of dsv4_batch_plan.  ctx, n_new, kv_len, ctx_add, ctx_out [B], q_start [B + 1], positions and
    token_seq [T] int32; caches: 1 to 4 of plan_cache; max_tokens: T, where neither positions, token_seq nor
    slots say it."""
    _need(isinstance(ctx, torch.Tensor) and ctx.device.type == "cuda", "ctx: wanted a tensor on a CUDA device")
    dev, B = ctx.device, ctx.shape[0]
    _need(1 <= len(caches) <= _abi.PLAN_MAX_CACHES, f"caches: {len(caches)}, wanted 1 to {_abi.PLAN_MAX_CACHES}")
    for t, name, shape in ((ctx, "ctx", (B,)), (n_new, "n_new", (B,)), (q_start, "q_start", (B + 1,)),
                           (kv_len, "kv_len", (B,)), (ctx_add, "ctx_add", (B,)), (ctx_out, "ctx_out", (B,)),
                           (positions, "positions", (None,)), (token_seq, "token_seq", (None,))):
        if t is not None or name in ("ctx", "n_new", "q_start", "kv_len"):
            _need_flat(t, name, torch.int32, shape, dev)
    sizes = {t.shape[0] for t in (positions, token_seq) if t is not None}
    sizes |= {c.shape[1] for c in caches if c.shape[1] is not None} | ({max_tokens} if max_tokens is not None else set())
    _need(len(sizes) == 1, f"positions, token_seq, slots and max_tokens: sizes {sorted(sizes)}, wanted one")
    for c in caches:
        _need(c.device == dev and c.shape[0] == B, f"cache: {c.shape[0]} requests on {c.device}, wanted {B} on {dev}")
    p = _abi.make(_abi.BatchPlanParams, B=B, T=sizes.pop(), num_caches=len(caches), ctx=_ptr(ctx), ctx_add=_ptr(ctx_add),
                  n_new=_ptr(n_new), ctx_out=_ptr(ctx_out), q_start=_ptr(q_start), kv_len=_ptr(kv_len),
                  positions=_ptr(positions), token_seq=_ptr(token_seq))
    for i, c in enumerate(caches):
        p.caches[i] = c
    p.device = dev
    p.tensors = (ctx, n_new, q_start, kv_len, ctx_add, ctx_out, positions, token_seq, tuple(c.tensors for c in caches))
    return p


def dsv4_batch_plan(params, stream=None):
    """Gives back and takes pages and writes the next step's tables, slots and positions (see include/dsv4_loop.h)."""
    _call("dsv4_batch_plan", _lib.dsv4_batch_plan, params, stream)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def draft_verify_params(target, tokens, q_start, max_q_len, out_tokens, n_out, draft=None, draft_row=None,
                        temperature=None, u=None, noise=None, logp=None, target_probs=False, draft_probs=False):
    """Parameter struct of dsv4_draft_verify.  target [T, vocab] logits (or probabilities) and draft [rows, vocab], bf16
    or fp32, rows of any stride (without draft_row: the drafted tokens' rows in order); tokens, draft_row [T],
    q_start [B + 1], out_tokens [B, max_q_len], n_out [B] int32; temperature [B], u [T], noise [B, vocab],
    logp [B, max_q_len] fp32."""
    dt, dev = _act(target, "target"), target.device
    _need_tensor(target, "target", (target.dtype,), (None, None), dev)
    T, V = target.shape
    _need_flat(n_out, "n_out", torch.int32, (None,), dev)
    B = n_out.shape[0]
    _need_flat(q_start, "q_start", torch.int32, (B + 1,), dev)
    _need_flat(tokens, "tokens", torch.int32, (T,), dev)
    _need_flat(out_tokens, "out_tokens", torch.int32, (B, max_q_len), dev)
    for t, name, dtype, shape in ((draft_row, "draft_row", torch.int32, (T,)), (temperature, "temperature", torch.float32, (B,)),
                                  (u, "u", torch.float32, (T,)), (logp, "logp", torch.float32, (B, max_q_len))):
        if t is not None:
            _need_flat(t, name, dtype, shape, dev)
    _need((u is None) == (noise is None), "u and noise go together")
    p = _abi.make(_abi.DraftVerifyParams, target=_ptr(target), target_stride=_row_stride(target), target_dtype=dt,
                  target_probs=int(target_probs), draft_row=_ptr(draft_row), tokens=_ptr(tokens), q_start=_ptr(q_start),
                  T=T, B=B, vocab=V, max_q_len=max_q_len, temperature=_ptr(temperature), u=_ptr(u), noise=_ptr(noise),
                  out_tokens=_ptr(out_tokens), n_out=_ptr(n_out), logp=_ptr(logp), draft_probs=int(draft_probs))
    if draft is not None:
        p.draft_dtype = _act(draft, "draft")
        _need_tensor(draft, "draft", (draft.dtype,), (None, V), dev)
        # (an empty tensor has no address, which would mean that there is no draft; nothing is read from it)
        p.draft, p.draft_rows, p.draft_stride = _ptr(draft) or 16, draft.shape[0], _row_stride(draft)
    if noise is not None:
        _need_tensor(noise, "noise", (torch.float32,), (B, V), dev)
        p.noise_stride = _row_stride(noise)
    p.device = dev
    p.tensors = (target, tokens, q_start, out_tokens, n_out, draft, draft_row, temperature, u, noise, logp)
    return p


def dsv4_draft_verify(params, stream=None):
    """Verifies drafted tokens and draws the token that follows them (see include/dsv4_loop.h)."""
    _call("dsv4_draft_verify", _lib.dsv4_draft_verify, params, stream)


def dsv4_kernel_launches() -> int:
    """Kernels the library has enqueued (or recorded into a graph) since it was loaded."""
    return int(_lib.dsv4_kernel_launches())


def dsv4_read_device_flags() -> int:
    """Synchronises and returns (and clears) the kernels' range-check flags."""
    f = _abi.u32(0)
    st = _lib.dsv4_read_device_flags(f)
    if st not in (_abi.OK, _abi.ERR_BOUNDS, _abi.ERR_TIMEOUT):
        _abi.check("dsv4_read_device_flags", st)
    return int(f.value)
