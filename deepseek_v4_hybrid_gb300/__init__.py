"""DeepSeek-V4 hybrid compressed-attention decode step on one GB300 (sm_103a).

Thin Python binding of libdsv4.so (include/dsv4.h, include/dsv4_gqa.h).  The functions below take torch CUDA tensors,
fill the C parameter structs and call the library on the current torch stream; every step of the
decode path runs in the library's CUDA kernels.  There is no CPU fallback: the import fails if
the library is not built.
"""
from __future__ import annotations

import torch

from . import _abi
from ._abi import BF16, E4M3_PAGE, F32, FP8_DS_MLA, I8_ROWSCALE, MXFP4, Dsv4Error  # noqa: F401

_lib = _abi.load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


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


def _gqa_call(name, fn, params, stream):
    dev = params.device
    if dev.index is not None and dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = fn(params, _stream(stream))
    else:
        status = fn(params, _stream(stream))
    _abi.check(name, status)


def dsv4_gqa_append(params, stream=None):
    """Rotates and stores the new tokens' keys and values, and rotates their queries (see include/dsv4_gqa.h)."""
    _gqa_call("dsv4_gqa_append", _lib.dsv4_gqa_append, params, stream)


def dsv4_gqa_attention(params, stream=None):
    """Attention of the new tokens over the paged per-head caches into params' out and lse (see include/dsv4_gqa.h)."""
    _gqa_call("dsv4_gqa_attention", _lib.dsv4_gqa_attention, params, stream)


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
