"""Python binding of libgemma_attn.so (the C ABI in include/gemma_attn.h).

Argument marshalling only: every step of the attention path runs in the CUDA
library. Tensors may be torch tensors (device memory) or raw integer addresses;
``None`` passes a NULL pointer. Each wrapper raises ``GemmaAttnError`` on a
non-zero status. Importing this module raises ImportError when the library has
not been built (``python -m global_interleaved_layers_b200.build``): there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemma_attn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python global_interleaved_layers_b200/build.py` "
                      "(or __graft_entry__.build())")

_lib = ctypes.CDLL(LIB_PATH)

LOCAL = 0
GLOBAL = 1
BIDIR = 2  # vision patches: bidirectional, 2D RoPE; positions are [T, 2] (h, w); prefill only
CACHE_CONTIGUOUS = 0
CACHE_RING = 1
CACHE_KEYS_ROTATED = 0x100  # OR-ed into the layout (local layers): cached keys stored rotated
OUT_BF16 = 0
OUT_F32 = 1

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_MISALIGNED = -4
ERR_LAUNCH = -5
ERR_TIMEOUT = -6
ERR_DEVICE = -7
ERR_SEQLEN = -8
ERR_PAGE = -9
PAGES_BF16 = 0
PAGES_E4M3 = 1
PROBS_F32 = 0
PROBS_BF16 = 1


class GemmaAttnParams(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("window", ctypes.c_int32), ("rope_p", ctypes.c_float),
                ("rope_base", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class GemmaAttnPagedCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class GemmaAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gemma_attn_error_string(status)} ({status})")


_P = ctypes.c_void_p
_I = ctypes.c_int32
_PP = ctypes.POINTER(GemmaAttnParams)

_lib.gemma_attn_error_string.argtypes = [ctypes.c_int]
_lib.gemma_attn_error_string.restype = ctypes.c_char_p
_lib.gemma_attn_last_launch_count.argtypes = []
_lib.gemma_attn_last_launch_count.restype = ctypes.c_int
_lib.gemma_attn_prefill_workspace_size.argtypes = [_PP, _I, ctypes.POINTER(ctypes.c_size_t)]
_lib.gemma_attn_prefill.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, ctypes.c_size_t, _P]
_lib.gemma_attn_prefill_rotate.argtypes = _lib.gemma_attn_prefill.argtypes
_lib.gemma_attn_prefill_attend.argtypes = _lib.gemma_attn_prefill.argtypes
_lib.gemma_attn_decode.argtypes = [_PP, _P, _P, _P, _P, _P, _I, _I, _P, _I, _I, _I, _P, _P, _I, _P]
_lib.gemma_attn_decode_num_splits.argtypes = [_PP, _I, _I, _I, ctypes.POINTER(ctypes.c_int32)]
_lib.gemma_attn_combine.argtypes = [_P, _P, _I, _I, _I, _I, _P, _P, _P]
_lib.gemma_attn_tile_plan.argtypes = [_I, _I, _P, _I, _I, _I, _P, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
_lib.gemma_attn_decode_noalloc.argtypes = [_PP, _P, _P, _P, _P, _P, _I, _I, _P, _I, _I, _I, _I, _P, _P, _P]
_lib.gemma_attn_cache_append.argtypes = [_PP, _P, _P, _P, _P, _I, _I, _P, _I, _I, _P]
_lib.gemma_attn_decode_shard.argtypes = [_PP, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P]
_PC = ctypes.POINTER(GemmaAttnPagedCache)
_lib.gemma_attn_paged_append.argtypes = [_PP, _PC, _P, _P, _P, _P, _I, _I, _P]
_lib.gemma_attn_paged_gather.argtypes = [_PP, _PC, _P, _P, _P, _P, _I, _I, _P]
_lib.gemma_attn_paged_workspace_size.argtypes = [_PP, _PC, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]
_lib.gemma_attn_paged_attend.argtypes = [_PP, _PC, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]
_lib.gemma_attn_draft_verify.argtypes = [_P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P]
_lib.gemma_attn_check.argtypes = [_P]
_lib.gemma_attn_selftest_umma.argtypes = [_I, _P, _P, _P, _P, _P]
_lib.gemma_attn_selftest_timeout.argtypes = [_P, _P]
for _f in ("gemma_attn_prefill_workspace_size", "gemma_attn_prefill", "gemma_attn_decode",
           "gemma_attn_decode_num_splits", "gemma_attn_combine", "gemma_attn_tile_plan", "gemma_attn_check",
           "gemma_attn_selftest_umma", "gemma_attn_decode_noalloc", "gemma_attn_selftest_timeout",
           "gemma_attn_cache_append", "gemma_attn_decode_shard",
           "gemma_attn_prefill_rotate", "gemma_attn_prefill_attend", "gemma_attn_paged_append",
           "gemma_attn_paged_gather", "gemma_attn_paged_workspace_size", "gemma_attn_paged_attend",
           "gemma_attn_draft_verify"):
    getattr(_lib, _f).restype = ctypes.c_int


def params(kind: int, num_q_heads: int, num_kv_heads: int, head_dim: int, window: int = 0,
           rope_p: float = 1.0, rope_base: float = 10000.0, softmax_scale: Optional[float] = None,
           out_dtype: int = OUT_BF16) -> GemmaAttnParams:
    if softmax_scale is None:
        softmax_scale = head_dim ** -0.5
    return GemmaAttnParams(kind, window, rope_p, rope_base, softmax_scale, num_q_heads, num_kv_heads, head_dim,
                           out_dtype)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):          # numpy (host) arrays, for the host-only entry points
        return x.ctypes.data
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _stream(stream) -> Optional[int]:
    if stream is None:
        try:
            import torch
            return torch.cuda.current_stream().cuda_stream
        except Exception:  # no torch / no device: the legacy default stream
            return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise GemmaAttnError(rc, where)


def gemma_attn_error_string(status: int) -> str:
    return _lib.gemma_attn_error_string(status).decode()


def gemma_attn_last_launch_count() -> int:
    return int(_lib.gemma_attn_last_launch_count())


def gemma_attn_prefill_workspace_size(p: GemmaAttnParams, total_tokens: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.gemma_attn_prefill_workspace_size(ctypes.byref(p), total_tokens, ctypes.byref(n)),
           "gemma_attn_prefill_workspace_size")
    return int(n.value)


def gemma_attn_prefill(p: GemmaAttnParams, q, k, v, out, lse, positions, cu_seqlens, num_seqs: int,
                       total_tokens: int, max_seqlen: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(_lib.gemma_attn_prefill(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                   _ptr(positions), _ptr(cu_seqlens), num_seqs, total_tokens, max_seqlen,
                                   _ptr(workspace), workspace_bytes, _stream(stream)), "gemma_attn_prefill")


def gemma_attn_prefill_rotate(p: GemmaAttnParams, q, k, v, out, lse, positions, cu_seqlens, num_seqs: int,
                              total_tokens: int, max_seqlen: int, workspace, workspace_bytes: int,
                              stream=None) -> None:
    _check(_lib.gemma_attn_prefill_rotate(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                          _ptr(positions), _ptr(cu_seqlens), num_seqs, total_tokens, max_seqlen,
                                          _ptr(workspace), workspace_bytes, _stream(stream)),
           "gemma_attn_prefill_rotate")


def gemma_attn_prefill_attend(p: GemmaAttnParams, q, k, v, out, lse, positions, cu_seqlens, num_seqs: int,
                              total_tokens: int, max_seqlen: int, workspace, workspace_bytes: int,
                              stream=None) -> None:
    _check(_lib.gemma_attn_prefill_attend(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                          _ptr(positions), _ptr(cu_seqlens), num_seqs, total_tokens, max_seqlen,
                                          _ptr(workspace), workspace_bytes, _stream(stream)),
           "gemma_attn_prefill_attend")


def gemma_attn_decode(p: GemmaAttnParams, q, new_k, new_v, k_cache, v_cache, cache_layout: int,
                      cache_capacity: int, cache_seqlens, batch: int, n_q: int, max_cache_len: int,
                      partial_o, partial_lse, num_splits: int, stream=None) -> None:
    _check(_lib.gemma_attn_decode(ctypes.byref(p), _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(k_cache),
                                  _ptr(v_cache), cache_layout, cache_capacity, _ptr(cache_seqlens), batch, n_q,
                                  max_cache_len, _ptr(partial_o), _ptr(partial_lse), num_splits, _stream(stream)),
           "gemma_attn_decode")


def gemma_attn_decode_shard(p: GemmaAttnParams, q, new_k, k_cache, cache_capacity: int, shard_seqlens,
                            q_pos_offset, include_new: bool, batch: int, n_q: int, max_shard_len: int, partial_o,
                            partial_lse, num_splits: int, stream=None) -> None:
    """Split-KV partials over one key-range shard of a longer K=V history (global layers)."""
    _check(_lib.gemma_attn_decode_shard(ctypes.byref(p), _ptr(q), _ptr(new_k), _ptr(k_cache), cache_capacity,
                                        _ptr(shard_seqlens), _ptr(q_pos_offset), 1 if include_new else 0, batch,
                                        n_q, max_shard_len, _ptr(partial_o), _ptr(partial_lse), num_splits,
                                        _stream(stream)), "gemma_attn_decode_shard")


NOALLOC_SCRATCH_BYTES = 16 << 20


def gemma_attn_decode_noalloc(p: GemmaAttnParams, q, new_k, new_v, k_cache, v_cache, cache_layout: int,
                              cache_capacity: int, cache_seqlens, batch: int, n_q: int, max_cache_len: int,
                              num_splits: int, out, lse, stream=None) -> None:
    """Decode + combine with the split partials in the library's static device array (no allocation)."""
    _check(_lib.gemma_attn_decode_noalloc(ctypes.byref(p), _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(k_cache),
                                          _ptr(v_cache), cache_layout, cache_capacity, _ptr(cache_seqlens), batch,
                                          n_q, max_cache_len, num_splits, _ptr(out), _ptr(lse), _stream(stream)),
           "gemma_attn_decode_noalloc")


def gemma_attn_cache_append(p: GemmaAttnParams, new_k, new_v, k_cache, v_cache, cache_layout: int,
                            cache_capacity: int, cache_seqlens, batch: int, n_q: int, stream=None) -> None:
    """New tokens' K (and V) rows into the cache at slot position mod window (ring) or row position."""
    _check(_lib.gemma_attn_cache_append(ctypes.byref(p), _ptr(new_k), _ptr(new_v), _ptr(k_cache), _ptr(v_cache),
                                        cache_layout, cache_capacity, _ptr(cache_seqlens), batch, n_q,
                                        _stream(stream)), "gemma_attn_cache_append")


def gemma_attn_decode_num_splits(p: GemmaAttnParams, batch: int, n_q: int, max_cache_len: int) -> int:
    n = ctypes.c_int32(0)
    _check(_lib.gemma_attn_decode_num_splits(ctypes.byref(p), batch, n_q, max_cache_len, ctypes.byref(n)),
           "gemma_attn_decode_num_splits")
    return int(n.value)


def gemma_attn_combine(partial_o, partial_lse, num_splits: int, rows: int, head_dim: int, out_dtype: int, out,
                       lse, stream=None) -> None:
    _check(_lib.gemma_attn_combine(_ptr(partial_o), _ptr(partial_lse), num_splits, rows, head_dim, out_dtype,
                                   _ptr(out), _ptr(lse), _stream(stream)), "gemma_attn_combine")


def gemma_attn_tile_plan(kind: int, window: int, cu_seqlens_host, bm: int, bn: int):
    """Host-side tile plan; cu_seqlens_host is a numpy int32 array. Returns an int32 [n, 4] numpy array."""
    import numpy as np
    cu = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    n = ctypes.c_int64(0)
    _check(_lib.gemma_attn_tile_plan(kind, window, _ptr(cu), cu.shape[0] - 1, bm, bn, None, 0, ctypes.byref(n)),
           "gemma_attn_tile_plan")
    out = np.zeros((max(int(n.value), 1), 4), dtype=np.int32)
    _check(_lib.gemma_attn_tile_plan(kind, window, _ptr(cu), cu.shape[0] - 1, bm, bn, _ptr(out), n.value,
                                     ctypes.byref(n)), "gemma_attn_tile_plan")
    return out[: int(n.value)]


def _refuse(where: str, what: str) -> None:
    e = GemmaAttnError(ERR_INVALID_ARG, where)
    e.args = (f"{e.args[0]}: {what}",)
    raise e


def _tensor(x, where: str, name: str, dtype, shape=None, device=None):
    """Address of a torch tensor argument of a paged-cache or draft call, after checks of its type, shape,
    layout and device (raw addresses and None pass). A decode step makes a handful of these checks, so
    messages are put together only on the way out."""
    if x is None or type(x) is int:
        return x
    if x.dtype is not dtype:
        _refuse(where, f"{name} is {x.dtype}, not {dtype}")
    if not x.is_contiguous():
        _refuse(where, f"{name} is not contiguous")
    if shape is not None and x.shape != shape:
        _refuse(where, f"{name} has shape {tuple(x.shape)}, not {shape}")
    if device is not None and x.device != device:
        _refuse(where, f"{name} is on {x.device}, not {device}")
    return x.data_ptr()


def paged_cache(k_pages, v_pages, block_table, k_scales=None, v_scales=None) -> GemmaAttnPagedCache:
    """Handle of a paged cache over torch tensors, which it keeps alive: k_pages (and v_pages; None for
    global layers) [num_pages, kv_heads, page_size, head_dim] in bfloat16 or float8_e4m3fn, the latter
    with float32 scales [num_pages, kv_heads, page_size]; block_table [batch, max_blocks] int32."""
    import torch
    where = "paged_cache"
    if k_pages.dim() != 4 or block_table.dim() != 2:
        _refuse(where, "k_pages has 4 dimensions, block_table 2")
    if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        _refuse(where, f"k_pages is {k_pages.dtype}")
    e4m3 = k_pages.dtype == torch.float8_e4m3fn
    if e4m3 != (k_scales is not None) or (e4m3 and v_pages is not None) != (v_scales is not None):
        _refuse(where, "float8_e4m3fn pages have scales, bfloat16 pages none")
    dev, shape = k_pages.device, tuple(k_pages.shape)
    k = _tensor(k_pages, where, "k_pages", k_pages.dtype)
    v = _tensor(v_pages, where, "v_pages", k_pages.dtype, shape, dev)
    ks = _tensor(k_scales, where, "k_scales", torch.float32, shape[:3], dev)
    vs = _tensor(v_scales, where, "v_scales", torch.float32, shape[:3], dev)
    tab = _tensor(block_table, where, "block_table", torch.int32, None, dev)
    c = GemmaAttnPagedCache(k, v, ks, vs, tab, shape[0], shape[2], block_table.shape[1],
                            PAGES_E4M3 if e4m3 else PAGES_BF16)
    c.tensors = (k_pages, v_pages, block_table, k_scales, v_scales)
    c.fits = (shape[1], shape[3], block_table.shape[0], dev)
    return c


def _device_of(device, *tensors):
    """The device that a call's tensors have to be on: the handle's, else that of the first tensor
    among the arguments; None when all of them are raw addresses."""
    if device is None:
        for x in tensors:
            if x is not None and type(x) is not int:
                return x.device
    return device


def _call(fn, where: str, device, stream, *args) -> None:
    """fn(*args, stream) with `device` (of the call's tensors, or None) current; by default the stream
    is that device's current one. Tensors that are not on a CUDA device are refused here, after all
    other checks: their addresses mean nothing to a kernel."""
    if device is None:
        _check(fn(*args, _stream(stream)), where)
        return
    if device.type != "cuda":
        _refuse(where, f"tensors are on {device}, not on a CUDA device")
    import torch
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            _check(fn(*args, _stream(stream)), where)
        return
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        st = stream if type(stream) is int else stream.cuda_stream
    rc = fn(*args, st)
    if rc != OK:
        raise GemmaAttnError(rc, where)


def _cache_fits(p: GemmaAttnParams, cache: GemmaAttnPagedCache, batch: int, where: str):
    """The handle's tensors (when it was made from tensors) against the layer; returns their device."""
    fits = getattr(cache, "fits", None)
    if fits is None:
        return None
    heads, dim, rows, dev = fits
    if heads != p.num_kv_heads or dim != p.head_dim:
        _refuse(where, f"k_pages has {heads} heads of {dim} dims, the layer {p.num_kv_heads} of {p.head_dim}")
    if rows < batch:
        _refuse(where, f"block_table has {rows} rows for {batch} sequences")
    return dev


def gemma_attn_paged_append(p: GemmaAttnParams, cache: GemmaAttnPagedCache, new_k, new_v, cu_q, cache_seqlens,
                            batch: int, total_q: int, stream=None) -> None:
    """New rows into a paged cache: row cu_q[b] + i goes to position cache_seqlens[b] + i of sequence b."""
    import torch
    where = "gemma_attn_paged_append"
    dev = _device_of(_cache_fits(p, cache, batch, where), new_k, new_v, cu_q, cache_seqlens)
    shape = (total_q, p.num_kv_heads, p.head_dim)
    _call(_lib.gemma_attn_paged_append, where, dev, stream, ctypes.byref(p), ctypes.byref(cache),
          _tensor(new_k, where, "new_k", torch.bfloat16, shape, dev),
          _tensor(new_v, where, "new_v", torch.bfloat16, shape, dev),
          _tensor(cu_q, where, "cu_q", torch.int32, (batch + 1,), dev),
          _tensor(cache_seqlens, where, "cache_seqlens", torch.int32, (batch,), dev), batch, total_q)


def gemma_attn_paged_gather(p: GemmaAttnParams, cache: GemmaAttnPagedCache, starts, cu_out, out_k, out_v, batch: int,
                            total_out: int, stream=None) -> None:
    """Rows read back: row cu_out[b] + i receives position starts[b] + i of sequence b (params' out_dtype)."""
    import torch
    where = "gemma_attn_paged_gather"
    dev = _device_of(_cache_fits(p, cache, batch, where), starts, cu_out, out_k, out_v)
    shape = (total_out, p.num_kv_heads, p.head_dim)
    dt = torch.float32 if p.out_dtype == OUT_F32 else torch.bfloat16
    _call(_lib.gemma_attn_paged_gather, where, dev, stream, ctypes.byref(p), ctypes.byref(cache),
          _tensor(starts, where, "starts", torch.int32, (batch,), dev),
          _tensor(cu_out, where, "cu_out", torch.int32, (batch + 1,), dev),
          _tensor(out_k, where, "out_k", dt, shape, dev), _tensor(out_v, where, "out_v", dt, shape, dev), batch,
          total_out)


def gemma_attn_paged_workspace_size(p: GemmaAttnParams, cache: GemmaAttnPagedCache, batch: int, total_q: int,
                                    max_q: int, max_cache_len: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.gemma_attn_paged_workspace_size(ctypes.byref(p), ctypes.byref(cache), batch, total_q, max_q,
                                                max_cache_len, ctypes.byref(n)), "gemma_attn_paged_workspace_size")
    return int(n.value)


def gemma_attn_paged_attend(p: GemmaAttnParams, cache: GemmaAttnPagedCache, q, cu_q, cache_seqlens, out, lse,
                            batch: int, total_q: int, max_q: int, max_cache_len: int, workspace, workspace_bytes: int,
                            stream=None) -> None:
    """Attention of a chunk of new tokens over a paged cache that already holds their rows."""
    import torch
    where = "gemma_attn_paged_attend"
    dev = _device_of(_cache_fits(p, cache, batch, where), q, cu_q, cache_seqlens, out, lse, workspace)
    shape = (total_q, p.num_q_heads, p.head_dim)
    ws = workspace
    if ws is not None and type(ws) is not int:
        if not ws.is_contiguous() or ws.numel() * ws.element_size() < workspace_bytes or dev not in (None, ws.device):
            _refuse(where, "workspace is not workspace_bytes of the cache's device")
        ws = ws.data_ptr()
    _call(_lib.gemma_attn_paged_attend, where, dev, stream, ctypes.byref(p), ctypes.byref(cache),
          _tensor(q, where, "q", torch.bfloat16, shape, dev),
          _tensor(cu_q, where, "cu_q", torch.int32, (batch + 1,), dev),
          _tensor(cache_seqlens, where, "cache_seqlens", torch.int32, (batch,), dev),
          _tensor(out, where, "out", torch.float32 if p.out_dtype == OUT_F32 else torch.bfloat16, shape, dev),
          _tensor(lse, where, "lse", torch.float32, shape[:2], dev), batch, total_q, max_q, max_cache_len, ws,
          workspace_bytes)


def gemma_attn_draft_verify(target_probs, draft_probs, draft_tokens, draft_lens, uniforms, noise, num_accepted,
                            out_tokens, stream=None) -> None:
    """Drafted tokens accepted or replaced: target_probs [batch, max_draft + 1, vocab] float32 or bfloat16,
    draft_probs [batch, max_draft, vocab] or None (certain drafts), draft_tokens [batch, max_draft] int32,
    draft_lens [batch] int32 or None, uniforms [batch, max_draft], noise [batch, vocab] float32;
    num_accepted [batch] and out_tokens [batch, max_draft + 1] int32 are written."""
    import torch
    where = "gemma_attn_draft_verify"
    dt = target_probs.dtype
    if target_probs.dim() != 3 or target_probs.shape[1] < 1 or dt not in (torch.float32, torch.bfloat16):
        _refuse(where, "target_probs is [batch, max_draft + 1, vocab], float32 or bfloat16")
    b, n1, v = target_probs.shape
    dev, i32, f32 = target_probs.device, torch.int32, torch.float32
    _call(_lib.gemma_attn_draft_verify, where, dev, stream, _tensor(target_probs, where, "target_probs", dt),
          _tensor(draft_probs, where, "draft_probs", dt, (b, n1 - 1, v), dev),
          PROBS_BF16 if dt == torch.bfloat16 else PROBS_F32,
          _tensor(draft_tokens, where, "draft_tokens", i32, (b, n1 - 1), dev),
          _tensor(draft_lens, where, "draft_lens", i32, (b,), dev),
          _tensor(uniforms, where, "uniforms", f32, (b, n1 - 1), dev), _tensor(noise, where, "noise", f32, (b, v), dev),
          b, n1 - 1, v, _tensor(num_accepted, where, "num_accepted", i32, (b,), dev),
          _tensor(out_tokens, where, "out_tokens", i32, (b, n1), dev))


def gemma_attn_check(stream=None) -> None:
    _check(_lib.gemma_attn_check(_stream(stream)), "gemma_attn_check")


def gemma_attn_selftest_umma(mode: int, a, b, p, d, stream=None) -> None:
    _check(_lib.gemma_attn_selftest_umma(mode, _ptr(a), _ptr(b), _ptr(p), _ptr(d), _stream(stream)),
           "gemma_attn_selftest_umma")


def gemma_attn_selftest_timeout(gave_up, stream=None) -> None:
    _check(_lib.gemma_attn_selftest_timeout(_ptr(gave_up), _stream(stream)), "gemma_attn_selftest_timeout")


def raw_call(name: str, *args) -> int:
    """Call an entry point with raw ctypes arguments and return its status (for contract tests)."""
    return int(getattr(_lib, name)(*args))
