"""Python face of the 8-bit cache (include/lix_kv8.h): filling it, attention over it, the weight its tokens got,
and cutting it to the heaviest.

As in ops.py, the functions check and marshal arguments and call the C ABI; the
arithmetic runs in the HIP kernels.  They are for serving and record no
gradient: an input that asks for one is refused.
"""

from typing import NamedTuple

import torch

from . import _lib
from .ops import _need, _ptr, _stream

_DTYPES = {torch.bfloat16: _lib.LIX_BF16, torch.float16: _lib.LIX_FP16}
_E4M3, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32


class KV8Cache(NamedTuple):
    """A paged cache in 8 bits: keys and values as e4m3 codes [num_pages, kv_heads, page, head_dim]
    (float8_e4m3fn) and one fp32 scale per page and head [num_pages, kv_heads]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv8_cache(num_pages, kv_heads, page, head_dim, device="cuda"):
    """An empty KV8Cache: zero codes, scales of one."""
    codes = lambda: torch.zeros(num_pages, kv_heads, page, head_dim, dtype=torch.uint8,   # noqa: E731
                                device=device).view(torch.float8_e4m3fn)
    scales = lambda: torch.ones(num_pages, kv_heads, dtype=torch.float32, device=device)   # noqa: E731
    return KV8Cache(codes(), codes(), scales(), scales())


def _is(x, dtype, ndim, dev):
    return (isinstance(x, torch.Tensor) and x.dtype is dtype and x.ndim == ndim and x.get_device() == dev
            and x.is_contiguous())


def _cache(cache, table, lens):
    """Checks a cache and its tables; the shape of the codes.  One pass of cheap tests first: the calls of a
    decoding step last about as long on the host as on the GPU."""
    k, v, ks, vs = cache
    try:
        dev, shape = k.get_device(), k.shape
        ok = (dev >= 0 and k.dtype is _E4M3 and v.dtype is _E4M3 and ks.dtype is _F32 and vs.dtype is _F32
              and table.dtype is _I32 and lens.dtype is _I32 and v.shape == shape and k.is_contiguous()
              and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous() and table.is_contiguous()
              and lens.is_contiguous() and v.get_device() == dev and ks.get_device() == dev
              and vs.get_device() == dev and table.get_device() == dev and lens.get_device() == dev
              and ks.shape == shape[:2] and vs.shape == shape[:2] and len(shape) == 4 and table.ndim == 2
              and lens.ndim == 1 and lens.shape[0] == table.shape[0])
    except AttributeError:
        ok = False
    if ok:
        return shape
    _need(k, "cache.k", _E4M3, 4)
    _need(v, "cache.v", _E4M3, 4)
    _need(ks, "cache.k_scale", _F32, 2)
    _need(vs, "cache.v_scale", _F32, 2)
    _need(table, "block_table", _I32, 2)
    _need(lens, "kv_lens", _I32, 1)
    if v.shape != k.shape or ks.shape != k.shape[:2] or vs.shape != k.shape[:2]:
        raise ValueError("the cache must hold k and v [num_pages, kv_heads, page, head_dim] and scales "
                         "[num_pages, kv_heads]")
    if lens.shape[0] != table.shape[0]:
        raise ValueError("block_table and kv_lens must have one row per sequence")
    raise ValueError("the cache, block_table and kv_lens must be on the same device")


def _rows(x, name, batch, like):
    if (isinstance(x, torch.Tensor) and x.dtype in _DTYPES and x.ndim == 4 and x.shape[0] == batch
            and x.get_device() == like.get_device() and not (x.requires_grad and torch.is_grad_enabled())):
        strides = x.stride()
        if strides[3] == 1:
            return strides
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    if x.ndim != 4:
        raise ValueError(f"{name} must have 4 dimensions, got shape {tuple(x.shape)}")
    if x.shape[0] != batch:
        raise ValueError(f"{name} must have one row per sequence of block_table ({batch}), got {x.shape[0]}")
    if x.device != like.device:
        raise ValueError(f"{name} must be on the cache's device")
    raise ValueError(f"{name} asks for a gradient, which the 8-bit cache does not record")


def _per_sequence(x, name, lens):
    if x is None:
        return None
    if not _is(x, torch.int32, 1, lens.get_device()) or x.shape[0] != lens.shape[0]:
        _need(x, name, torch.int32, 1)
        raise ValueError(f"{name} must have one entry per sequence, on the cache's device")
    return x.data_ptr()


def kv8_append(cache, k, v, block_table, kv_lens, new_lens=None):
    """lix_kv8_append: k, v [B, S, kv_heads, head_dim] (bf16 or fp16, any strides that are multiples of 8 with the
    last dimension contiguous) become tokens kv_lens[b] .. kv_lens[b] + new_lens[b] - 1 (new_lens None: S of
    each) of the sequences of block_table [B, max_pages], quantised into the cache in place.  kv_lens is not
    changed.  Returns the cache."""
    pages, heads, page, dim = _cache(cache, block_table, kv_lens)
    B, mp = block_table.shape
    sk, sv = _rows(k, "k", B, cache.k), _rows(v, "v", B, cache.k)
    if v.shape != k.shape or v.dtype != k.dtype or k.shape[2] != heads or k.shape[3] != dim:
        raise ValueError(f"k and v must be [{B}, S, {heads}, {dim}] of one dtype")
    st = _lib.load().lix_kv8_append(
        k.data_ptr(), sk[0], sk[1], sk[2], v.data_ptr(), sv[0], sv[1], sv[2], _DTYPES[k.dtype], B, k.shape[1], heads, dim, cache.k.data_ptr(), cache.v.data_ptr(),
        cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), pages, page, block_table.data_ptr(), mp,
        kv_lens.data_ptr(), _per_sequence(new_lens, "new_lens", kv_lens), _stream(k.device))
    _lib.check(st, "lix_kv8_append")
    return cache


def _query(q, cache, table, lens, q_start, q_lens, scale):
    pages, heads, page, dim = _cache(cache, table, lens)
    strides = _rows(q, "q", table.shape[0], cache.k)
    if q.shape[2] % heads or q.shape[3] != dim:
        raise ValueError(f"q must be [B, S, heads, {dim}] with heads a multiple of {heads}, got {tuple(q.shape)}")
    return (pages, heads, page, dim, strides, _per_sequence(q_start, "q_start", lens),
            _per_sequence(q_lens, "q_lens", lens), float(dim ** -0.5 if scale is None else scale))


def kv8_attention(q, cache, block_table, kv_lens, q_start=None, q_lens=None, compress_ratio=1, scale=None,
                  topk_indices=None, workspace=None):
    """lix_kv8_attention: q [B, S, heads, head_dim] (bf16 or fp16) attends over the cached tokens of its sequence.

    q_start None: every query sees all kv_lens[b] tokens; else query t, at position q_start[b] + t, sees tokens
    [0, min(kv_lens[b], (q_start[b] + t + 1) // compress_ratio)).  q_lens [B] int32: queries behind it are
    padding.  topk_indices int32 [B, S, topk] (as select_topk returns them): only those tokens, shared by the
    heads.  scale: of the scores, head_dim ** -0.5 if None.  workspace: an optional uint8 GPU tensor of
    kv8_attention_workspace_bytes.  Returns (out like q, lse fp32 [B, S, heads]); a query that sees nothing has
    out 0 and lse -inf."""
    pages, heads, page, dim, sq, start, lens, scale = _query(q, cache, block_table, kv_lens, q_start, q_lens, scale)
    B, S, Hq, _ = q.shape
    mp = block_table.shape[1]
    topk = 0
    if topk_indices is not None:
        _need(topk_indices, "topk_indices", torch.int32, 3)
        if topk_indices.shape[0] != B or topk_indices.shape[1] != S or topk_indices.device != q.device:
            raise ValueError("topk_indices must be [B, S, topk] on the device of q")
        topk = topk_indices.shape[2]
    lib = _lib.load()
    if workspace is None:
        need = lib.lix_kv8_attention_workspace_bytes(B, S, Hq, heads, dim, page, mp, topk)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, "workspace", torch.uint8, 1)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty((B, S, Hq), dtype=torch.float32, device=q.device)
    st = lib.lix_kv8_attention(
        q.data_ptr(), sq[0], sq[1], sq[2], _DTYPES[q.dtype], B, S, Hq, heads, dim,
        cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), pages, page,
        block_table.data_ptr(), mp, kv_lens.data_ptr(), start, lens, int(compress_ratio), scale, _ptr(topk_indices),
        topk, out.data_ptr(), lse.data_ptr(), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(q.device))
    _lib.check(st, "lix_kv8_attention")
    return out, lse


def kv8_attention_workspace_bytes(batch, queries, heads, kv_heads, head_dim, page, max_pages, topk=0):
    """lix_kv8_attention_workspace_bytes: the workspace kv8_attention takes for these sizes (topk 0: no
    topk_indices); 0 where it needs none, -1 for sizes it does not take."""
    return int(_lib.load().lix_kv8_attention_workspace_bytes(int(batch), int(queries), int(heads), int(kv_heads),
                                                             int(head_dim), int(page), int(max_pages), int(topk)))


def kv8_token_weights(q, cache, block_table, kv_lens, lse, q_start=None, q_lens=None, compress_ratio=1, scale=None,
                      out=None, accumulate=False):
    """lix_kv8_token_weights: the attention weight each cached token got from the queries, summed over queries and
    the heads of its key head.  Arguments as for kv8_attention; lse is what it returned.  Returns fp32
    [B, kv_heads, max_pages * page]; out (of at least that width) is written for s < kv_lens[b], or added to with
    accumulate=True, and keeps its other entries."""
    pages, heads, page, dim, sq, start, lens, scale = _query(q, cache, block_table, kv_lens, q_start, q_lens, scale)
    B, S, Hq, _ = q.shape
    mp = block_table.shape[1]
    _need(lse, "lse", torch.float32, 3)
    if tuple(lse.shape) != (B, S, Hq) or lse.device != q.device:
        raise ValueError(f"lse must be [{B}, {S}, {Hq}] on the device of q")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.zeros((B, heads, mp * page), dtype=torch.float32, device=q.device)
    else:
        _need(out, "out", torch.float32, 3)
        if out.shape[0] != B or out.shape[1] != heads or out.device != q.device:
            raise ValueError(f"out must be [{B}, {heads}, width] on the device of q")
    lib = _lib.load()
    need = lib.lix_kv8_token_weights_workspace_bytes(B, S, Hq, heads, dim, page, mp)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
    st = lib.lix_kv8_token_weights(
        q.data_ptr(), sq[0], sq[1], sq[2], _DTYPES[q.dtype], B, S, Hq, heads, dim,
        cache.k.data_ptr(), cache.k_scale.data_ptr(), pages, page, block_table.data_ptr(), mp, kv_lens.data_ptr(),
        start, lens, int(compress_ratio), scale, lse.data_ptr(), out.data_ptr(), out.shape[2], int(bool(accumulate)),
        _ptr(ws), max(need, 0), _stream(q.device))
    _lib.check(st, "lix_kv8_token_weights")
    return out


def kv8_evict(cache, block_table, kv_lens, weights, new_block_table, keep, recent=0, sinks=0):
    """lix_kv8_evict: of each sequence with more than `keep` tokens, for each key head, keeps the first `sinks`, the
    last `recent` and the heaviest others by weights fp32 [B, kv_heads, width >= max_pages * page] (equal weights:
    the lower token first), of the others all, and writes them in ascending order to the pages of new_block_table
    [B, >= keep / page], which no sequence may be using.  Returns (new_lens int32 [B], kept int32
    [B, kv_heads, keep], their weights fp32 [B, kv_heads, keep]); -1 and 0 behind the last kept token."""
    pages, heads, page, dim = _cache(cache, block_table, kv_lens)
    B, mp = block_table.shape
    keep, recent, sinks = int(keep), int(recent), int(sinks)
    _need(weights, "weights", torch.float32, 3)
    _need(new_block_table, "new_block_table", torch.int32, 2)
    if weights.shape[0] != B or weights.shape[1] != heads or weights.device != cache.k.device:
        raise ValueError(f"weights must be [{B}, {heads}, width] on the cache's device")
    if new_block_table.shape[0] != B or new_block_table.device != cache.k.device:
        raise ValueError("new_block_table must have one row per sequence, on the cache's device")
    lib = _lib.load()
    need = lib.lix_kv8_evict_workspace_bytes(B, heads, page, mp, weights.shape[2], keep, recent, sinks)
    if need < 0:
        raise _lib.LixError(_lib.LIX_ERR_SHAPE, "lix_kv8_evict_workspace_bytes")
    dev = cache.k.device
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    new_lens = torch.empty(B, dtype=torch.int32, device=dev)
    kept = torch.empty((B, heads, keep), dtype=torch.int32, device=dev)
    new_weights = torch.empty((B, heads, keep), dtype=torch.float32, device=dev)
    st = lib.lix_kv8_evict(
        cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), pages, page, B,
        heads, dim, block_table.data_ptr(), mp, kv_lens.data_ptr(), weights.data_ptr(), weights.shape[2],
        new_block_table.data_ptr(), new_block_table.shape[1], keep, recent, sinks, new_lens.data_ptr(),
        kept.data_ptr(), new_weights.data_ptr(), _ptr(ws), need, _stream(dev))
    _lib.check(st, "lix_kv8_evict")
    return new_lens, kept, new_weights
