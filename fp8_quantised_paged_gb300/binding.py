"""FP8-quantised paged decode attention for GB300 (sm_103a).

The main calls, hand-written CUDA kernels behind a C ABI (``include/fp8pa.h``):

* :func:`kv_append_quant` -- absmax-scale each new token's K/V rows, round
  them to E4M3 or E5M2 (or symmetric INT8 codes) and scatter codes and
  scales into the paged cache.
* :func:`paged_decode_attention` -- grouped-query (or shared-latent MLA)
  attention of one query token per request over its paged FP8 cache, split
  across the GPU and merged.
* :func:`kv_append_rope` -- the append behind a rotation of q and k by their
  positions.
* :func:`paged_decode_attention_mod` -- the decode with a window, an
  always-visible prefix, capped scores and a distance bias.
* :func:`paged_prefill_attention` -- ragged query chunks of any length, with
  the same modifiers.
* :func:`paged_tree_attention` -- trees of drafted tokens, with the same modifiers.
* :func:`kv_keep_accepted`, :func:`kv_fork`, :func:`kv_resize`, :func:`kv_compact` --
  the pages of sequences that branch.

These wrappers only check torch tensors and pass their device pointers and
the current CUDA stream to the library.  PyTorch provides memory and streams;
all arithmetic runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from ._native import (E4M3, E5M2, INT8, MAX_TREE, OUT_BF16, OUT_F32, SCALE_CHANNEL_STATIC,
                      SCALE_MX_BLOCK,
                      SCALE_SEGMENT, SCALE_TOKEN_GROUP, SCALE_TOKEN_HEAD, SEGMENT_TOKENS,
                      Fp8paError)

__all__ = ["kv_append_quant", "kv_append_quant_segment", "segment_scale_heads",
           "kv_channel_scales", "kv_channel_absmax_update",
           "kv_scales_from_absmax", "paged_decode_attention", "paged_multiquery_attention",
           "kv_append_rope", "paged_decode_attention_mod", "paged_prefill_attention",
           "prefill_workspace_bytes", "paged_tree_attention",
           "tree_workspace_bytes", "MAX_TREE", "KvPages", "kv_keep_accepted", "kv_fork", "kv_resize",
           "kv_compact", "pages_workspace_bytes", "decode_step", "decode_workspace_bytes",
           "get_device_error", "set_decode_workers",
           "version", "E4M3", "E5M2", "INT8", "SCALE_TOKEN_HEAD", "SCALE_CHANNEL_STATIC",
           "SCALE_TOKEN_GROUP", "SCALE_MX_BLOCK", "SCALE_SEGMENT", "SEGMENT_TOKENS", "OUT_BF16",
           "OUT_F32", "Fp8paError"]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class _Nop:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


_NOP = _Nop()


def _on(dev):
    """Make `dev` current for a call (a no-op when it already is)."""
    return _NOP if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _scale_dtype(scale_mode):
    """fp32 scales, or E8M0 exponent bytes for the MX block mode."""
    return torch.uint8 if scale_mode == SCALE_MX_BLOCK else torch.float32


def _need(t, dtype, name, device=None):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _alloc(shape, dtype, dev, stream, result=True):
    """Memory for a call on `stream` (None: the current one), from the pool of that
    stream: the block's earlier uses are that stream's own, so the call's kernels come
    behind them.  A result is read on the current stream, too: its memory is not handed
    out again before what that stream holds when the result is freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if result:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def version() -> int:
    return int(N.lib.fp8pa_version())


def set_decode_workers(workers: int) -> None:
    N.check(N.lib.fp8pa_set_decode_workers(int(workers)), "set_decode_workers")
    _decode_need.cache_clear()


def kv_append_quant(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, fmt=E4M3,
                    scale_mode=SCALE_TOKEN_HEAD, group_size=64, stream=None):
    """k, v: bf16 [num_tokens, Hkv, D] (v may be None for the MLA latent);
    slot_mapping: int32 [num_tokens]; caches: uint8 [num_blocks, Hkv, bs, D];
    scales: float32 per the scale mode, uint8 E8M0 exponents for SCALE_MX_BLOCK
    (see include/fp8pa.h)."""
    _need(k, torch.bfloat16, "k")
    dev = k.device
    _need(v, torch.bfloat16, "v", dev)
    _need(slot_mapping, torch.int32, "slot_mapping", dev)
    _need(k_cache, torch.uint8, "k_cache", dev)
    _need(v_cache, torch.uint8, "v_cache", dev)
    _need(k_scale, _scale_dtype(scale_mode), "k_scale", dev)
    _need(v_scale, _scale_dtype(scale_mode), "v_scale", dev)
    n, hkv, d = k.shape
    nb, _, bs, _ = k_cache.shape
    with _on(dev):
        rc = N.lib.fp8pa_kv_append_quant(_ptr(k), _ptr(v), _ptr(slot_mapping), n, hkv, d, fmt,
                                         scale_mode, group_size, _ptr(k_cache), _ptr(v_cache),
                                         _ptr(k_scale), _ptr(v_scale), nb, bs, _stream(stream))
    N.check(rc, "kv_append_quant")


def segment_scale_heads(n_kv_heads: int) -> int:
    """Row length of a SCALE_SEGMENT scale tensor: KV heads rounded up to 4."""
    return (n_kv_heads + 3) // 4 * 4


def kv_append_quant_segment(k, v, slot_mapping, seq_offsets, seq_start_pos, k_cache, v_cache,
                            k_scale, v_scale, seg_state, fmt=E4M3, stream=None):
    """Append with block-wise cumulative rescaling (SCALE_SEGMENT).
    k, v: bf16 [num_tokens, Hkv, D] (v may be None); seq_offsets: int32
    [num_seqs + 1]; seq_start_pos: int32 [num_seqs] (each sequence's cached
    length before the call); scales: float32 [num_blocks, round_up(Hkv, 4)];
    seg_state: float32 [num_seqs, 2, Hkv, 2], carried between calls (see
    include/fp8pa.h)."""
    _need(k, torch.bfloat16, "k")
    dev = k.device
    _need(v, torch.bfloat16, "v", dev)
    _need(slot_mapping, torch.int32, "slot_mapping", dev)
    _need(seq_offsets, torch.int32, "seq_offsets", dev)
    _need(seq_start_pos, torch.int32, "seq_start_pos", dev)
    _need(k_cache, torch.uint8, "k_cache", dev)
    _need(v_cache, torch.uint8, "v_cache", dev)
    _need(k_scale, torch.float32, "k_scale", dev)
    _need(v_scale, torch.float32, "v_scale", dev)
    _need(seg_state, torch.float32, "seg_state", dev)
    n, hkv, d = k.shape
    nb, _, bs, _ = k_cache.shape
    ns = seq_start_pos.numel()
    if seq_offsets.numel() != ns + 1 or tuple(seg_state.shape) != (ns, 2, hkv, 2):
        raise ValueError("seq_offsets must have num_seqs + 1 entries and seg_state "
                         "[num_seqs, 2, Hkv, 2]")
    if tuple(k_scale.shape) != (nb, segment_scale_heads(hkv)):
        raise ValueError("k_scale must be [num_blocks, round_up(Hkv, 4)]")
    with _on(dev):
        rc = N.lib.fp8pa_kv_append_quant_segment(
            _ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(seq_offsets), _ptr(seq_start_pos), ns,
            hkv, d, fmt, _ptr(seg_state), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
            _ptr(v_scale), nb, bs, _stream(stream))
    N.check(rc, "kv_append_quant_segment")


def kv_channel_scales(x, fmt=E5M2, out=None, stream=None):
    """Static per-channel scales max(absmax over tokens / FMAX, 1e-12) of a
    bf16 [N, Hkv, D] tensor; returns float32 [Hkv, D]."""
    _need(x, torch.bfloat16, "x")
    n, hkv, d = x.shape
    if out is None:
        out = _alloc((hkv, d), torch.float32, x.device, stream)
    _need(out, torch.float32, "out", x.device)
    with torch.cuda.device(x.device):
        rc = N.lib.fp8pa_kv_channel_scales(_ptr(x), n, hkv, d, fmt, _ptr(out), _stream(stream))
    N.check(rc, "kv_channel_scales")
    return out


def kv_channel_absmax_update(x, running_absmax, stream=None):
    """Fold a prefill batch x (bf16 [N, Hkv, D]) into a running per-channel
    absmax (float32 [Hkv, D], zero-initialised by the caller)."""
    _need(x, torch.bfloat16, "x")
    _need(running_absmax, torch.float32, "running_absmax", x.device)
    n, hkv, d = x.shape
    with torch.cuda.device(x.device):
        rc = N.lib.fp8pa_kv_channel_absmax_update(_ptr(x), n, hkv, d, _ptr(running_absmax),
                                                  _stream(stream))
    N.check(rc, "kv_channel_absmax_update")
    return running_absmax


def kv_scales_from_absmax(absmax, fmt=E5M2, out=None, stream=None):
    """Static scales max(absmax / FMAX, 1e-12) from a running absmax."""
    _need(absmax, torch.float32, "absmax")
    if out is None:
        out = _alloc(absmax.shape, torch.float32, absmax.device, stream)
    _need(out, torch.float32, "out", absmax.device)
    with torch.cuda.device(absmax.device):
        rc = N.lib.fp8pa_kv_scales_from_absmax(_ptr(absmax), absmax.numel(), fmt, _ptr(out),
                                               _stream(stream))
    N.check(rc, "kv_scales_from_absmax")
    return out


def decode_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim, head_dim_v, block_size,
                           max_blocks_per_seq, device=None, q_len=1) -> int:
    """Workspace bytes for the decode (q_len = 1) or a causal chunk of q_len
    queries per request (paged_multiquery_attention, decode_step)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        nbytes = int(N.lib.fp8pa_multiquery_workspace_bytes(batch, q_len, n_q_heads, n_kv_heads,
                                                            head_dim, head_dim_v, block_size,
                                                            max_blocks_per_seq))
    if nbytes == 0:
        raise Fp8paError(N.ERR_UNSUPPORTED, "decode_workspace_bytes")
    return nbytes


def paged_decode_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens,
                           n_kv_heads, sm_scale, fmt=E4M3, scale_mode=SCALE_TOKEN_HEAD,
                           group_size=64, head_dim_v=None, out=None, out_dtype=None,
                           workspace=None, stream=None):
    """q: bf16 [B, Hq, Dk]; caches/scales as written by kv_append_quant
    (v_cache/v_scale may be the same tensors as k_cache/k_scale for MLA);
    block_tables: int32 [B, max_blocks]; seq_lens: int32 [B].
    Returns out [B, Hq, Dv] (bf16 unless out_dtype=torch.float32)."""
    _need(q, torch.bfloat16, "q")
    dev = q.device
    for t, dt, name in ((k_cache, torch.uint8, "k_cache"), (v_cache, torch.uint8, "v_cache"),
                        (k_scale, _scale_dtype(scale_mode), "k_scale"),
                        (v_scale, _scale_dtype(scale_mode), "v_scale"),
                        (block_tables, torch.int32, "block_tables"),
                        (seq_lens, torch.int32, "seq_lens")):
        _need(t, dt, name, dev)
    B, hq, dk = q.shape
    dv = dk if head_dim_v is None else head_dim_v
    nb, _, bs, _ = k_cache.shape
    max_blocks = block_tables.shape[1]
    if out is None:
        out = _alloc((B, hq, dv), out_dtype or torch.bfloat16, dev, stream)
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be bf16 or float32")
    _need(out, out.dtype, "out", dev)
    with _on(dev):
        if workspace is None:
            need = int(N.lib.fp8pa_decode_workspace_bytes(B, hq, n_kv_heads, dk, dv, bs,
                                                          max_blocks))
            if need > 0:
                workspace = _alloc(need, torch.uint8, dev, stream, result=False)
        # need == 0 means the shapes are rejected: the call below returns the
        # precise status code.
        _need(workspace, torch.uint8, "workspace", dev)
        rc = N.lib.fp8pa_paged_decode_attention(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_tables), max_blocks, _ptr(seq_lens), B, bs, hq, n_kv_heads, dk, dv, fmt,
            scale_mode, group_size, float(sm_scale), nb, _ptr(out), odt, _ptr(workspace),
            0 if workspace is None else workspace.numel(), _stream(stream))
    N.check(rc, "paged_decode_attention")
    return out


def paged_multiquery_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens,
                               n_kv_heads, sm_scale, fmt=E4M3, scale_mode=SCALE_TOKEN_HEAD,
                               group_size=64, head_dim_v=None, out=None, out_dtype=None,
                               workspace=None, stream=None):
    """A causal chunk of q_len queries per request: q bf16 [B, q_len, Hq, Dk],
    the chunk already appended to the cache, seq_lens counting it.  Query i
    sees the first seq_lens[b] - (q_len - 1 - i) tokens.
    Returns out [B, q_len, Hq, Dv]."""
    _need(q, torch.bfloat16, "q")
    dev = q.device
    for t, dt, name in ((k_cache, torch.uint8, "k_cache"), (v_cache, torch.uint8, "v_cache"),
                        (k_scale, _scale_dtype(scale_mode), "k_scale"),
                        (v_scale, _scale_dtype(scale_mode), "v_scale"),
                        (block_tables, torch.int32, "block_tables"),
                        (seq_lens, torch.int32, "seq_lens")):
        _need(t, dt, name, dev)
    B, qlen, hq, dk = q.shape
    dv = dk if head_dim_v is None else head_dim_v
    nb, _, bs, _ = k_cache.shape
    max_blocks = block_tables.shape[1]
    if out is None:
        out = _alloc((B, qlen, hq, dv), out_dtype or torch.bfloat16, dev, stream)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be bf16 or float32")
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _need(out, out.dtype, "out", dev)
    with _on(dev):
        if workspace is None:
            need = int(N.lib.fp8pa_multiquery_workspace_bytes(B, qlen, hq, n_kv_heads, dk, dv,
                                                              bs, max_blocks))
            if need > 0:
                workspace = _alloc(need, torch.uint8, dev, stream, result=False)
        _need(workspace, torch.uint8, "workspace", dev)
        rc = N.lib.fp8pa_paged_multiquery_attention(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_tables), max_blocks, _ptr(seq_lens), B, qlen, bs, hq, n_kv_heads, dk, dv,
            fmt, scale_mode, group_size, float(sm_scale), nb, _ptr(out), odt, _ptr(workspace),
            0 if workspace is None else workspace.numel(), _stream(stream))
    N.check(rc, "paged_multiquery_attention")
    return out


def decode_step(k_new, v_new, slot_mapping, q, k_cache, v_cache, k_scale, v_scale,
                block_tables, seq_lens, n_kv_heads, sm_scale, fmt=E4M3,
                scale_mode=SCALE_TOKEN_HEAD, group_size=64, head_dim_v=None, out=None,
                out_dtype=None, workspace=None, stream=None):
    """Append the new rows (as kv_append_quant), then attend (as
    paged_decode_attention for q [B, Hq, Dk], or paged_multiquery_attention
    for q [B, q_len, Hq, Dk]) in one call.  For MLA pass v_new=None and
    v_cache/v_scale equal to k_cache/k_scale.  Returns out."""
    _need(q, torch.bfloat16, "q")
    dev = q.device
    _need(k_new, torch.bfloat16, "k_new", dev)
    _need(v_new, torch.bfloat16, "v_new", dev)
    for t, dt, name in ((k_cache, torch.uint8, "k_cache"), (v_cache, torch.uint8, "v_cache"),
                        (k_scale, _scale_dtype(scale_mode), "k_scale"),
                        (v_scale, _scale_dtype(scale_mode), "v_scale"),
                        (block_tables, torch.int32, "block_tables"),
                        (seq_lens, torch.int32, "seq_lens"),
                        (slot_mapping, torch.int32, "slot_mapping")):
        _need(t, dt, name, dev)
    multi = q.dim() == 4
    B, qlen, hq, dk = q.shape if multi else (q.shape[0], 1, q.shape[1], q.shape[2])
    dv = dk if head_dim_v is None else head_dim_v
    nb, _, bs, _ = k_cache.shape
    max_blocks = block_tables.shape[1]
    n_new = k_new.shape[0]
    if out is None:
        shape = (B, qlen, hq, dv) if multi else (B, hq, dv)
        out = _alloc(shape, out_dtype or torch.bfloat16, dev, stream)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be bf16 or float32")
    odt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _need(out, out.dtype, "out", dev)
    with _on(dev):
        if workspace is None:
            need = int(N.lib.fp8pa_multiquery_workspace_bytes(B, qlen, hq, n_kv_heads, dk, dv,
                                                              bs, max_blocks))
            if need > 0:
                workspace = _alloc(need, torch.uint8, dev, stream, result=False)
        _need(workspace, torch.uint8, "workspace", dev)
        rc = N.lib.fp8pa_decode_step(
            _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n_new, _ptr(q), _ptr(k_cache),
            _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), max_blocks,
            _ptr(seq_lens), B, qlen, bs, hq, n_kv_heads, dk, dv, fmt, scale_mode, group_size,
            float(sm_scale), nb, _ptr(out), odt, _ptr(workspace),
            0 if workspace is None else workspace.numel(), _stream(stream))
    N.check(rc, "decode_step")
    return out


# The wrappers below run next to kernels of a few microseconds, so their checks
# touch each tensor as little as they can.
def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, dev):
    """The handle of `stream`, or of the current stream of device `dev`."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _want(t, dtype, name, dev):
    if t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        _need(t, dtype, name, dev)


def _check_cache(k_cache, v_cache, k_scale, v_scale, n_kv_heads, head_dim, scale_mode,
                 group_size, dev):
    """The shapes of a paged cache and its scales; returns (num_blocks, block_size)."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[1] != n_kv_heads or shape[3] != head_dim:
        raise ValueError(f"k_cache must be [num_blocks, {n_kv_heads}, block_size, {head_dim}], "
                         f"got {tuple(shape)}")
    nb, _, bs, _ = shape
    sdt = torch.float32
    if scale_mode == SCALE_TOKEN_HEAD:
        numel = nb * n_kv_heads * bs
    elif scale_mode == SCALE_CHANNEL_STATIC:
        numel = n_kv_heads * head_dim
    elif scale_mode == SCALE_SEGMENT:
        numel = nb * segment_scale_heads(n_kv_heads)
    else:
        numel = nb * n_kv_heads * bs * (head_dim // max(int(group_size), 1))
        if scale_mode == SCALE_MX_BLOCK:
            sdt = torch.uint8
    _want(k_cache, torch.uint8, "k_cache", dev)
    _want(k_scale, sdt, "k_scale", dev)
    if k_scale.numel() != numel:
        raise ValueError(f"k_scale must hold {numel} values, got {k_scale.numel()}")
    if v_cache is not None or v_scale is not None:
        if v_cache is None or v_scale is None:
            raise ValueError("v_cache and v_scale come together")
        _want(v_cache, torch.uint8, "v_cache", dev)
        _want(v_scale, sdt, "v_scale", dev)
        if v_cache.shape != shape:
            raise ValueError("v_cache must have k_cache's shape")
        if v_scale.numel() != numel:
            raise ValueError(f"v_scale must hold {numel} values, got {v_scale.numel()}")
    return nb, bs


def _rows(t, name, n, heads, d, dev):
    """A bf16 [n, heads, d] tensor whose tokens may be strided; returns the stride."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    if t.device != dev or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != (n, heads, d):
        raise ValueError(f"{name} must be {(n, heads, d)}, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (heads > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s0 if n > 1 else heads * d


def kv_append_rope(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, k_scale, v_scale,
                   rot_offset=0, interleaved=False, fmt=E4M3, scale_mode=SCALE_TOKEN_HEAD,
                   group_size=64, q_out=None, stream=None):
    """Turn q and k by their tokens' rotary angles, then quantise K and V into
    the paged cache.  q: bf16 [N, Hq, D] (None: no queries); k, v: bf16
    [N, Hkv, D] (v None for the MLA latent); their tokens may be strided (slices
    of a fused projection).  positions: int32 [N]; cos_sin: float32
    [max_position, rot_dim], cosines then sines of rot_dim / 2 angles; the dims
    rot_offset .. rot_offset + rot_dim - 1 of each row are turned, halves paired
    (or neighbours, interleaved=True).  Returns q_out (q_out=q: in place)."""
    if k.dim() != 3:
        raise ValueError("k must be [num_tokens, n_kv_heads, head_dim]")
    dev = k.device
    n, hkv, d = k.shape
    ks = _rows(k, "k", n, hkv, d, dev)
    vs = 0 if v is None else _rows(v, "v", n, hkv, d, dev)
    hq = qs = qos = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [num_tokens, n_q_heads, head_dim]")
        hq = q.shape[1]
        qs = _rows(q, "q", n, hq, d, dev)
        if q_out is None:
            q_out = _alloc((n, hq, d), torch.bfloat16, dev, stream)
        qos = _rows(q_out, "q_out", n, hq, d, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _want(positions, torch.int32, "positions", dev)
    _want(slot_mapping, torch.int32, "slot_mapping", dev)
    _want(cos_sin, torch.float32, "cos_sin", dev)
    if positions.numel() != n or slot_mapping.numel() != n:
        raise ValueError(f"positions and slot_mapping must hold {n} entries")
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position, rot_dim]")
    if v is None:
        v_cache = v_scale = None
    elif v_cache is None or v_scale is None:
        raise ValueError("v needs v_cache and v_scale")
    nb, bs = _check_cache(k_cache, v_cache, k_scale, v_scale, hkv, d, scale_mode, group_size, dev)
    max_position, rot_dim = cos_sin.shape
    with _on(dev):
        rc = N.lib.fp8pa_kv_append_rope(
            _addr(q), _addr(q_out), k.data_ptr(), _addr(v), qs, qos, ks, vs, positions.data_ptr(),
            cos_sin.data_ptr(), max_position, rot_dim, rot_offset, 1 if interleaved else 0,
            slot_mapping.data_ptr(), n, hq, hkv, d, fmt, scale_mode, group_size,
            k_cache.data_ptr(), _addr(v_cache), k_scale.data_ptr(), _addr(v_scale), nb, bs,
            _raw_stream(stream, dev))
    if rc:
        N.check(rc, "kv_append_rope")
    return q_out


def _check_mods(prefix_lens, alibi_slopes, batch, hq, dev):
    if prefix_lens is not None:
        _want(prefix_lens, torch.int32, "prefix_lens", dev)
        if prefix_lens.numel() != batch:
            raise ValueError(f"prefix_lens must hold {batch} entries")
    if alibi_slopes is not None:
        _want(alibi_slopes, torch.float32, "alibi_slopes", dev)
        if alibi_slopes.numel() != hq:
            raise ValueError(f"alibi_slopes must hold {hq} entries")


def _window(window):
    """A window as the library takes it (one wider than any context leaves all of it)."""
    return max(-1, min(window, 0x7FFFFFFF))


def _check_tables(block_tables, seq_lens, dev):
    _want(block_tables, torch.int32, "block_tables", dev)
    _want(seq_lens, torch.int32, "seq_lens", dev)
    shape = block_tables.shape
    if len(shape) != 2 or seq_lens.dim() != 1 or shape[0] != seq_lens.shape[0]:
        raise ValueError("block_tables must be [batch, max_blocks] and seq_lens [batch]")
    return shape


def _output(out, shape, out_dtype, dev, stream):
    """The output tensor and its element code."""
    if out is None:
        out = _alloc(shape, out_dtype or torch.bfloat16, dev, stream)
    elif out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    dt = out.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise TypeError("out must be bf16 or float32")
    _want(out, dt, "out", dev)
    return out, OUT_F32 if dt is torch.float32 else OUT_BF16


def _scratch(need, dev, stream):
    """Workspace of one call (None where the sizes are refused)."""
    return _alloc(need, torch.uint8, dev, stream, result=False) if need else None


@functools.lru_cache(maxsize=4096)
def _decode_need(device_index, *sizes):
    """Workspace size of a decode of these sizes (device_index is current);
    forgotten by set_decode_workers."""
    return int(N.lib.fp8pa_decode_workspace_bytes(*sizes))


@functools.lru_cache(maxsize=4096)
def _prefill_need(device_index, *sizes):
    """Workspace size of a prefill of these sizes (device_index is current)."""
    return int(N.lib.fp8pa_prefill_workspace_bytes(*sizes))


def paged_decode_attention_mod(q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens,
                               n_kv_heads, sm_scale, window=0, prefix_lens=None, logit_cap=0.0,
                               alibi_slopes=None, fmt=E4M3, scale_mode=SCALE_TOKEN_HEAD,
                               group_size=64, out=None, out_dtype=None, workspace=None,
                               stream=None):
    """paged_decode_attention (GQA layout) with score modifiers: a sliding
    window of `window` tokens (0: none), the first prefix_lens[b] tokens (int32
    [B]) always visible, scores capped as logit_cap * tanh(z / logit_cap)
    (0: not), and alibi_slopes[h] (float32 [Hq]) times the distance subtracted.
    Pages without a visible token are not read.  Returns out [B, Hq, D]."""
    _need(q, torch.bfloat16, "q")
    if q.dim() != 3:
        raise ValueError("q must be [batch, n_q_heads, head_dim]")
    dev = q.device
    B, hq, d = q.shape
    rows, max_blocks = _check_tables(block_tables, seq_lens, dev)
    if rows != B:
        raise ValueError(f"block_tables and seq_lens must have {B} rows")
    if v_cache is None or v_scale is None:
        raise ValueError("v_cache and v_scale are required")
    nb, bs = _check_cache(k_cache, v_cache, k_scale, v_scale, n_kv_heads, d, scale_mode,
                          group_size, dev)
    _check_mods(prefix_lens, alibi_slopes, B, hq, dev)
    out, odt = _output(out, (B, hq, d), out_dtype, dev, stream)
    with _on(dev):
        if workspace is None:
            workspace = _scratch(_decode_need(dev.index, B, hq, n_kv_heads, d, d, bs, max_blocks),
                                 dev, stream)
        else:
            _want(workspace, torch.uint8, "workspace", dev)
        rc = N.lib.fp8pa_paged_decode_attention_mod(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), block_tables.data_ptr(), max_blocks, seq_lens.data_ptr(), B, bs,
            hq, n_kv_heads, d, fmt, scale_mode, group_size, sm_scale, _window(window),
            _addr(prefix_lens), logit_cap, _addr(alibi_slopes), nb, out.data_ptr(), odt,
            _addr(workspace), 0 if workspace is None else workspace.numel(),
            _raw_stream(stream, dev))
    if rc:
        N.check(rc, "paged_decode_attention_mod")
    return out


def prefill_workspace_bytes(total_q, batch, n_q_heads, n_kv_heads, head_dim, block_size,
                            max_blocks_per_seq, device=None) -> int:
    """Workspace bytes of paged_prefill_attention for these sizes.  A workspace made for
    a larger batch is taken, too, but may not hold the tiles converted once."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        nbytes = int(N.lib.fp8pa_prefill_workspace_bytes(total_q, batch, n_q_heads, n_kv_heads,
                                                         head_dim, block_size,
                                                         max_blocks_per_seq))
    if nbytes == 0:
        raise Fp8paError(N.ERR_UNSUPPORTED, "prefill_workspace_bytes")
    return nbytes


def paged_prefill_attention(q, q_offsets, k_cache, v_cache, k_scale, v_scale, block_tables,
                            seq_lens, n_kv_heads, sm_scale, window=0, prefix_lens=None,
                            logit_cap=0.0, alibi_slopes=None, fmt=E4M3,
                            scale_mode=SCALE_TOKEN_HEAD, group_size=64, out=None, out_dtype=None,
                            workspace=None, stream=None):
    """Causal attention of ragged query chunks over the paged cache, with the
    score modifiers of paged_decode_attention_mod.  q: bf16 [total_q, Hq, D],
    request b's chunk in rows q_offsets[b] .. q_offsets[b+1]-1 (int32 [B + 1]),
    already appended; seq_lens counts it.  The first prefix_lens[b] tokens are
    visible to every query, also to those before them.  Rows outside every
    chunk are left as they were.  Returns out [total_q, Hq, D]."""
    _need(q, torch.bfloat16, "q")
    if q.dim() != 3:
        raise ValueError("q must be [total_q, n_q_heads, head_dim]")
    dev = q.device
    total, hq, d = q.shape
    B, max_blocks = _check_tables(block_tables, seq_lens, dev)
    _want(q_offsets, torch.int32, "q_offsets", dev)
    if q_offsets.numel() != B + 1:
        raise ValueError(f"q_offsets must hold {B + 1} entries")
    if v_cache is None or v_scale is None:
        raise ValueError("v_cache and v_scale are required")
    nb, bs = _check_cache(k_cache, v_cache, k_scale, v_scale, n_kv_heads, d, scale_mode,
                          group_size, dev)
    _check_mods(prefix_lens, alibi_slopes, B, hq, dev)
    out, odt = _output(out, (total, hq, d), out_dtype, dev, stream)
    with _on(dev):
        if workspace is None:
            workspace = _scratch(_prefill_need(dev.index, total, B, hq, n_kv_heads, d, bs,
                                               max_blocks), dev, stream)
        else:
            _want(workspace, torch.uint8, "workspace", dev)
        rc = N.lib.fp8pa_paged_prefill_attention(
            q.data_ptr(), q_offsets.data_ptr(), total, k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(), max_blocks,
            seq_lens.data_ptr(), B, bs, hq, n_kv_heads, d, fmt, scale_mode, group_size, sm_scale,
            _window(window), _addr(prefix_lens), logit_cap, _addr(alibi_slopes), nb,
            out.data_ptr(), odt, _addr(workspace),
            0 if workspace is None else workspace.numel(), _raw_stream(stream, dev))
    if rc:
        N.check(rc, "paged_prefill_attention")
    return out


@functools.lru_cache(maxsize=4096)
def _tree_need(device_index, *sizes):
    """Workspace size of a tree attention of these sizes (device_index is current)."""
    return int(N.lib.fp8pa_tree_workspace_bytes(*sizes))


def tree_workspace_bytes(total_q, batch, n_q_heads, n_kv_heads, head_dim, block_size,
                         max_blocks_per_seq, device=None) -> int:
    """Workspace bytes of paged_tree_attention for these sizes; enough for every smaller
    batch of the same heads."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        nbytes = int(N.lib.fp8pa_tree_workspace_bytes(total_q, batch, n_q_heads, n_kv_heads,
                                                      head_dim, block_size, max_blocks_per_seq))
    if nbytes == 0:
        raise Fp8paError(N.ERR_UNSUPPORTED, "tree_workspace_bytes")
    return nbytes


def paged_tree_attention(q, q_offsets, parents, k_cache, v_cache, k_scale, v_scale, block_tables,
                         seq_lens, n_kv_heads, sm_scale, window=0, prefix_lens=None,
                         logit_cap=0.0, alibi_slopes=None, fmt=E4M3, scale_mode=SCALE_TOKEN_HEAD,
                         group_size=64, out=None, out_dtype=None, workspace=None, stream=None):
    """Attention for trees of drafted tokens over the paged cache.  q: bf16 [total_q, Hq, D],
    request b's nodes in rows q_offsets[b] .. q_offsets[b+1]-1 (int32 [B + 1]), already
    appended as its last tokens; seq_lens counts them.  parents: int32 [total_q], a node's
    parent within its tree (a smaller number), -1 for a child of the last token ahead of
    the tree.  A node sees the tokens ahead of the tree, its ancestors and itself; score
    modifiers as paged_prefill_attention, counted along its line.  At most MAX_TREE nodes a
    request.  Rows outside every tree are left as they were.  Returns out [total_q, Hq, D]."""
    _need(q, torch.bfloat16, "q")
    if q.dim() != 3:
        raise ValueError("q must be [total_q, n_q_heads, head_dim]")
    dev = q.device
    total, hq, d = q.shape
    B, max_blocks = _check_tables(block_tables, seq_lens, dev)
    _want(q_offsets, torch.int32, "q_offsets", dev)
    _want(parents, torch.int32, "parents", dev)
    if q_offsets.numel() != B + 1 or parents.numel() != total:
        raise ValueError(f"q_offsets must hold {B + 1} entries and parents {total}")
    if v_cache is None or v_scale is None:
        raise ValueError("v_cache and v_scale are required")
    nb, bs = _check_cache(k_cache, v_cache, k_scale, v_scale, n_kv_heads, d, scale_mode,
                          group_size, dev)
    _check_mods(prefix_lens, alibi_slopes, B, hq, dev)
    out, odt = _output(out, (total, hq, d), out_dtype, dev, stream)
    with _on(dev):
        if workspace is None:
            workspace = _scratch(_tree_need(dev.index, total, B, hq, n_kv_heads, d, bs,
                                            max_blocks), dev, stream)
        else:
            _want(workspace, torch.uint8, "workspace", dev)
        rc = N.lib.fp8pa_paged_tree_attention(
            q.data_ptr(), q_offsets.data_ptr(), total, parents.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(),
            max_blocks, seq_lens.data_ptr(), B, bs, hq, n_kv_heads, d, fmt, scale_mode,
            group_size, sm_scale, _window(window), _addr(prefix_lens), logit_cap,
            _addr(alibi_slopes), nb, out.data_ptr(), odt, _addr(workspace),
            0 if workspace is None else workspace.numel(), _raw_stream(stream, dev))
    if rc:
        N.check(rc, "paged_tree_attention")
    return out


class KvPages:
    """The arrays of a cache whose pages the page operators move: codes and scales of
    every layer's K and V, each contiguous with the pages as its first dimension and a
    multiple of 16 bytes a page, no two overlapping (static channel scales are not among
    them).  Made once,
    next to the cache; it holds the tensors."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        if not self.tensors:
            raise ValueError("KvPages needs a tensor")
        self.device, self.num_blocks = self.tensors[0].device, self.tensors[0].shape[0]
        rows = None
        for i, t in enumerate(self.tensors):
            _need(t, t.dtype, f"tensors[{i}]", self.device)
            if t.dim() < 2 or t.shape[0] != self.num_blocks:
                raise ValueError(f"tensors[{i}] must hold {self.num_blocks} pages, got "
                                 f"{tuple(t.shape)}")
            if t.dim() == 4:
                if rows not in (None, tuple(t.shape[1:3])):
                    raise ValueError(f"tensors[{i}]: heads and block size differ from the "
                                     f"others'")
                rows = tuple(t.shape[1:3])
        # an array given twice would have its rows moved twice, by threads at once
        spans = sorted((t.data_ptr(), t.numel() * t.element_size(), i)
                       for i, t in enumerate(self.tensors))
        for (p, n, i), (q, _, j) in zip(spans, spans[1:]):
            if p + n > q:
                raise ValueError(f"tensors[{i}] and tensors[{j}] overlap")
        self.n_kv_heads, self.block_size = rows or (None, None)
        # whether every array has a row per token and head
        self.per_token = all(t.dim() == 4 for t in self.tensors)
        n = len(self.tensors)
        self._ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.tensors])
        self._bytes = (ctypes.c_longlong * n)(*[t[0].numel() * t.element_size()
                                                for t in self.tensors])
        self._args = (ctypes.cast(self._ptrs, ctypes.c_void_p),
                      ctypes.cast(self._bytes, ctypes.c_void_p), n)


def pages_workspace_bytes(rows, num_blocks) -> int:
    """Workspace bytes of kv_fork, kv_resize and kv_compact."""
    nbytes = int(N.lib.fp8pa_pages_workspace_bytes(rows, num_blocks))
    if nbytes == 0:
        raise Fp8paError(N.ERR_BAD_SHAPE, "pages_workspace_bytes")
    return nbytes


def _pages_scratch(workspace, rows, num_blocks, dev, stream):
    if workspace is None:
        return _scratch(int(N.lib.fp8pa_pages_workspace_bytes(rows, num_blocks)), dev, stream)
    _want(workspace, torch.uint8, "workspace", dev)
    return workspace


def _check_pages(pages, block_tables, seq_lens, ref_counts):
    """Tables, lengths and counts of a cache's rows; returns (device, rows, max_blocks)."""
    dev = pages.device
    rows, max_blocks = _check_tables(block_tables, seq_lens, dev)
    if ref_counts is not None:
        _want(ref_counts, torch.int32, "ref_counts", dev)
        if ref_counts.numel() != pages.num_blocks:
            raise ValueError(f"ref_counts must hold {pages.num_blocks} entries")
    if pages.block_size is None:
        raise ValueError("the pages hold no [num_blocks, n_kv_heads, block_size, ...] tensor")
    return dev, rows, max_blocks


def kv_keep_accepted(accepted, q_offsets, block_tables, seq_lens, pages, new_lens=None,
                     stream=None, ref_counts=None):
    """After a drafted tree's verification: move the accepted path's cached rows to the
    front of the tree's tokens.  accepted: int32 [B, max_accepted], the path's node
    numbers, then -1; request b's tree is its last q_offsets[b+1] - q_offsets[b] tokens.
    pages: a KvPages of per-token arrays, not the codes of SCALE_SEGMENT (a row there has
    its page's scale).  A row with a tree is not forked before this call; with ref_counts
    (as kv_fork's) a request whose rows would move into a page that another row holds, too,
    is left as it was (DEVERR_SHARED), without them it is not noticed.  Returns the new
    lengths (int32 [B]); the pages behind them stay the rows' until kv_resize."""
    dev, B, max_blocks = _check_pages(pages, block_tables, seq_lens, ref_counts)
    if not pages.per_token:
        raise ValueError("kv_keep_accepted needs arrays of rows per token and head")
    _want(accepted, torch.int32, "accepted", dev)
    _want(q_offsets, torch.int32, "q_offsets", dev)
    if accepted.dim() != 2 or accepted.shape[0] != B or q_offsets.numel() != B + 1:
        raise ValueError(f"accepted must be [{B}, max_accepted] and q_offsets hold {B + 1}")
    if new_lens is None:
        new_lens = _alloc((B,), torch.int32, dev, stream)
    _want(new_lens, torch.int32, "new_lens", dev)
    if new_lens.numel() != B:
        raise ValueError(f"new_lens must hold {B} entries")
    head = (accepted.data_ptr(), accepted.shape[1], q_offsets.data_ptr(), block_tables.data_ptr(),
            max_blocks, seq_lens.data_ptr(), B)
    tail = (*pages._args, pages.n_kv_heads, pages.num_blocks, pages.block_size,
            new_lens.data_ptr(), _raw_stream(stream, dev))
    with _on(dev):
        if ref_counts is None:
            rc = N.lib.fp8pa_kv_keep_accepted(*head, *tail)
        else:
            rc = N.lib.fp8pa_kv_keep_accepted_counted(*head, ref_counts.data_ptr(), *tail)
    if rc:
        N.check(rc, "kv_keep_accepted")
    return new_lens


def kv_fork(src_rows, dst_rows, block_tables, seq_lens, ref_counts, pages, workspace=None,
            stream=None):
    """Make row dst_rows[i] (of length 0) a copy of the sequence in row src_rows[i]: full
    pages are shared, a last page that is not full is copied to a free one.  src_rows,
    dst_rows: int32 [n]; block_tables, seq_lens and ref_counts (int32 [num_blocks], the
    table entries that hold a page) change in place."""
    dev, rows, max_blocks = _check_pages(pages, block_tables, seq_lens, ref_counts)
    _want(src_rows, torch.int32, "src_rows", dev)
    _want(dst_rows, torch.int32, "dst_rows", dev)
    n = src_rows.numel()
    if dst_rows.numel() != n:
        raise ValueError("src_rows and dst_rows must be of one length")
    workspace = _pages_scratch(workspace, rows, pages.num_blocks, dev, stream)
    with _on(dev):
        rc = N.lib.fp8pa_kv_fork(
            src_rows.data_ptr(), dst_rows.data_ptr(), n, block_tables.data_ptr(), max_blocks,
            seq_lens.data_ptr(), rows, ref_counts.data_ptr(), *pages._args, pages.num_blocks,
            pages.block_size, workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if rc:
        N.check(rc, "kv_fork")


def kv_resize(new_lens, block_tables, seq_lens, ref_counts, block_size, workspace=None,
              stream=None):
    """Give every row the length new_lens[r] (int32 [rows]): pages behind it are given
    back, missing ones taken from the free pages, the lowest first; 0 frees the row.
    block_tables, seq_lens and ref_counts change in place."""
    _need(ref_counts, torch.int32, "ref_counts")
    dev = ref_counts.device
    rows, max_blocks = _check_tables(block_tables, seq_lens, dev)
    _want(new_lens, torch.int32, "new_lens", dev)
    if new_lens.numel() != rows:
        raise ValueError(f"new_lens must hold {rows} entries")
    nb = ref_counts.numel()
    workspace = _pages_scratch(workspace, rows, nb, dev, stream)
    with _on(dev):
        rc = N.lib.fp8pa_kv_resize(
            new_lens.data_ptr(), block_tables.data_ptr(), max_blocks, seq_lens.data_ptr(), rows,
            ref_counts.data_ptr(), nb, block_size, _addr(workspace),
            0 if workspace is None else workspace.numel(), _raw_stream(stream, dev))
    if rc:
        N.check(rc, "kv_resize")


def kv_compact(block_tables, seq_lens, ref_counts, pages, page_map=None, workspace=None,
               stream=None):
    """Move the live pages behind the number of live ones to the free pages before it, in
    every array; block_tables and ref_counts follow in place.  Returns page_map (int32
    [num_blocks]): the new number of each page, -1 for a free one."""
    dev, rows, max_blocks = _check_pages(pages, block_tables, seq_lens, ref_counts)
    nb = pages.num_blocks
    if page_map is None:
        page_map = _alloc((nb,), torch.int32, dev, stream)
    _want(page_map, torch.int32, "page_map", dev)
    if page_map.numel() != nb:
        raise ValueError(f"page_map must hold {nb} entries")
    workspace = _pages_scratch(workspace, rows, nb, dev, stream)
    with _on(dev):
        rc = N.lib.fp8pa_kv_compact(
            block_tables.data_ptr(), max_blocks, seq_lens.data_ptr(), rows, ref_counts.data_ptr(),
            *pages._args, nb, pages.block_size, page_map.data_ptr(), workspace.data_ptr(),
            workspace.numel(), _raw_stream(stream, dev))
    if rc:
        N.check(rc, "kv_compact")
    return page_map


def get_device_error(stream=None, device=None) -> int:
    """Synchronise the stream, then read and clear the device error word."""
    flags = ctypes.c_uint32(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        N.check(N.lib.fp8pa_get_device_error(_stream(stream), ctypes.byref(flags)),
                "get_device_error")
    return int(flags.value)
