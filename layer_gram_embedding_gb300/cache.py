"""Binding of the entry points for caches in 8 bits and for pages (argument
marshalling only).

Keys and values may be kept as 8-bit floats with a scale for each block of
tokens and head: half the bytes of the cache of tree.py, for contexts twice as
long in the same memory.  The three operators that touch it there stand here in
that form (ple_qk_norm_rope_fp8, ple_tree_attention_fp8, ple_tree_commit_fp8).
ple_plan_pages and ple_copy_pages keep the pages of either kind of cache:
requests that fork, end or begin, and pools that shrink.

A cache in 8 bits is torch.float8_e4m3fn, shaped and strided as in tree.py but
for strides and head_dim that are multiples of 16.  Its scales are
torch.bfloat16, [pages, kv_heads, page_size / block] (several layers:
[layers, pages, ...]), block being 16, 32, 64 or 128: any strides with the last
dimension contiguous, the same for keys and values.  What a slot stands for is
element * scale, so cache.to(torch.bfloat16).unflatten(-2, (-1, block)) times
scale[..., None, None] is the cache in 16 bits, exactly where scales are powers
of two.  A new cache's scales may hold anything finite and positive, as
torch.ones does.

Checks, streams, workspaces and autograd are as in tree.py.
"""

from __future__ import annotations

import struct

import torch

from .binding import _lend, lib
from .tree import (_ELEMENTS, _IDS, _call, _caches, _device, _element, _empty, _heads, _i32, _i64,
                   _overlap, _table, _vector)

# the argument structs of include/ple.h, field by field
_NORM_ROPE8 = struct.Struct("@PPPqqqqqqPPPPPqqPqqPPqqqqPPPqiiiiiiiiiff0qPPqqqi0q")
_ATTENTION8 = struct.Struct("@PqqPPqqqqPPPPPPPqqiiiiiiiif0qPPqqqi0q")
_COMMIT8 = struct.Struct("@PPPPPPPPPPPqqqqqqiiiiiiiiii0qPPqqqi0q")
_PLAN = struct.Struct("@PPPPPPPPPqiiiiii0q")
_COPY = struct.Struct("@PPPqqqqPPqqqi0qqiiiiii0q")

_fp8, _bf16 = torch.float8_e4m3fn, torch.bfloat16
_BLOCKS = (16, 32, 64, 128)


def _caches8(k, v, k_scale, v_scale, dims: int, where: str) -> int:
    """Checks caches in 8 bits and their scales; the tokens of a block."""
    _caches(k, v, _fp8, dims, where)
    for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
        if s.dtype != _bf16:
            raise TypeError(f"{where}: {name} must be {_bf16}, got {s.dtype}")
    blocks = k_scale.shape[-1] if k_scale.dim() else 0
    page_size = k.shape[-2]
    if k_scale.dim() != dims - 1 or k_scale.shape[:-1] != k.shape[:-2] or \
            v_scale.shape != k_scale.shape or v_scale.stride() != k_scale.stride() or \
            (blocks > 1 and k_scale.stride(-1) != 1):
        raise ValueError(f"{where}: the scales must be {'[layers, ' if dims == 5 else '['}pages, "
                         "kv_heads, page_size / block] with one shape and the same strides, the "
                         "last dimension contiguous")
    block = page_size // blocks if blocks else 0
    if block * blocks != page_size or block not in _BLOCKS:
        raise ValueError(f"{where}: {blocks} scales a page of {page_size} slots: a block must "
                         f"have one of {_BLOCKS} tokens")
    return block


def ple_qk_norm_rope_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         positions: torch.Tensor | None, rope: torch.Tensor | None,
                         q_weight: torch.Tensor | None, k_weight: torch.Tensor | None,
                         k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, page_table: torch.Tensor, ctx_lens: torch.Tensor,
                         cu_seqlens: torch.Tensor, eps: float = 1e-6, interleaved: bool = False,
                         rope_scale: float = 1.0, q_out: torch.Tensor | None = None, stream=None):
    """ple_qk_norm_rope with the append to a cache in 8 bits, in one launch;
    returns q_out.

    Norms, rotation, slots and q, k, v as there (k_out is not offered: keys go
    to the cache).  Every block that new tokens go to gets, for the keys and the
    values of each head, the least power of two as its scale under which they
    fit; where it holds tokens already its scale never falls, and where that
    grows their elements are rounded anew.  Infinities and NaN become NaN and
    have no part in the scale."""
    where = "ple_qk_norm_rope_fp8"
    dev = q.get_device()
    dtype = q.dtype
    element = _ELEMENTS.get(dtype)
    if element is None or q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4 or \
            k_scale.dim() != 3:
        _device(where, q, k, k_cache, k_scale)
        _element(q, "q", where)
        raise ValueError(f"{where}: q must be [T, q_heads, head_dim], k [T, kv_heads, head_dim], "
                         "the caches [pages, kv_heads, page_size, head_dim] and the scales "
                         "[pages, kv_heads, blocks]")
    T, Hq, D = q_shape = q.shape
    k_shape = k.shape
    Hk = k_shape[1]
    R = 0 if rope is None else 2 * rope.shape[0]
    B = ctx_lens.shape[0] if ctx_lens.dim() == 1 else -1
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    strides, shape = k_cache.stride(), k_cache.shape
    scale_strides, scale_shape = k_scale.stride(), k_scale.shape
    table_shape = page_table.shape
    blocks = scale_shape[2]
    block = shape[2] // blocks if blocks else 0
    # the step of a serving loop: norms, a rotation, new queries
    if not (q_out is None and rope is not None and positions is not None and q_weight is not None
            and k_weight is not None and dev >= 0 and B >= 0
            and k.dtype is dtype and v.dtype is dtype and q_weight.dtype is dtype
            and k_weight.dtype is dtype and k_cache.dtype is _fp8 and v_cache.dtype is _fp8
            and k_scale.dtype is _bf16 and v_scale.dtype is _bf16
            and positions.dtype is _i32 and rope.dtype is _i64 and page_table.dtype is _i32
            and ctx_lens.dtype is _i32 and cu_seqlens.dtype is _i32
            and k.get_device() == dev and v.get_device() == dev and q_weight.get_device() == dev
            and k_weight.get_device() == dev and k_cache.get_device() == dev
            and v_cache.get_device() == dev and k_scale.get_device() == dev
            and v_scale.get_device() == dev and positions.get_device() == dev
            and rope.get_device() == dev and page_table.get_device() == dev
            and ctx_lens.get_device() == dev and cu_seqlens.get_device() == dev
            and k_shape[0] == T and k_shape[2] == D and v.shape == k_shape
            and qs[2] == 1 and ks[2] == 1 and vs[2] == 1
            and q_weight.shape == (D,) and k_weight.shape == (D,) and positions.shape == (T,)
            and rope.dim() == 1 and v_cache.shape == shape and v_cache.stride() == strides
            and strides[3] == 1 and shape[1] == Hk and shape[3] == D
            and scale_shape[:2] == shape[:2] and v_scale.shape == scale_shape
            and v_scale.stride() == scale_strides and scale_strides[2] == 1
            and block * blocks == shape[2] and block in _BLOCKS
            and cu_seqlens.shape == (B + 1,) and len(table_shape) == 2 and table_shape[0] == B
            and q_weight.is_contiguous() and k_weight.is_contiguous()
            and positions.is_contiguous() and rope.is_contiguous() and page_table.is_contiguous()
            and ctx_lens.is_contiguous() and cu_seqlens.is_contiguous()):
        dev = _device(where, q, k, v, positions, rope, q_weight, k_weight, k_cache, v_cache,
                      k_scale, v_scale, page_table, ctx_lens, cu_seqlens, q_out)
        _heads(q, dtype, T, None, D, "q", where)
        _heads(k, dtype, T, None, D, "k", where)
        _heads(v, dtype, T, Hk, D, "v", where)
        if rope is not None:
            _vector(rope, _i64, rope.shape[0], "rope", where)
            if positions is None:
                raise ValueError(f"{where}: a rotation needs positions")
        if positions is not None:
            _vector(positions, _i32, T, "positions", where)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _vector(w, dtype, D, name, where)
        block = _caches8(k_cache, v_cache, k_scale, v_scale, 4, where)
        if shape[1] != Hk or shape[3] != D:
            raise ValueError(f"{where}: the caches must be [pages, {Hk}, page_size, {D}]")
        _vector(ctx_lens, _i32, B, "ctx_lens", where)
        _vector(cu_seqlens, _i32, B + 1, "cu_seqlens", where)
        _table(page_table, _i32, B, "page_table", where)
        if q_out is not None:
            _heads(q_out, dtype, T, Hq, D, "q_out", where)
    if q_out is None:
        q_out = _empty(q_shape, dtype=dtype, device=q.device)
        _lend(stream, dev, q_out)
    os = q_out.stride()
    args = _NORM_ROPE8.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
        0 if positions is None else positions.data_ptr(), rope.data_ptr() if R else 0,
        0 if q_weight is None else q_weight.data_ptr(),
        0 if k_weight is None else k_weight.data_ptr(), q_out.data_ptr(), os[0], os[1], 0, 0, 0,
        k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], strides[2], shape[0],
        page_table.data_ptr(), ctx_lens.data_ptr(), cu_seqlens.data_ptr(), T, B, table_shape[1],
        shape[2], element, Hq, Hk, D, R, 1 if interleaved else 0, rope_scale, eps,
        k_scale.data_ptr(), v_scale.data_ptr(), 0, scale_strides[0], scale_strides[1], block)
    _call(where, lib().ple_qk_norm_rope_fp8, dev, stream, args)
    return q_out


# bytes by (num_tokens, q_heads, kv_heads, head_dim, device index)
_workspace_sizes: dict = {}


def _workspace_size(*sizes) -> int:
    """The bytes of a call's own workspace.  A query that failed is no answer:
    it is not kept, and the call itself says what is wrong."""
    size = _workspace_sizes.get(sizes)
    if size is None:
        with torch.cuda.device(sizes[4]):
            size = lib().ple_tree_attention_fp8_workspace(*sizes[:4])
        if size < 0:
            return 0
        if len(_workspace_sizes) >= 4096:
            _workspace_sizes.clear()
        _workspace_sizes[sizes] = size
    return size


def ple_tree_attention_fp8_workspace(num_tokens: int, q_heads: int, kv_heads: int, head_dim: int,
                                     device=None) -> torch.Tensor:
    """A uint8 workspace for ple_tree_attention_fp8 calls of these sizes (or
    fewer tokens) on one stream; need not be cleared."""
    with torch.cuda.device(torch.device("cuda" if device is None else device)):
        n = lib().ple_tree_attention_fp8_workspace(int(num_tokens), int(q_heads), int(kv_heads),
                                                   int(head_dim))
        if n < 0:
            raise ValueError("ple_tree_attention_fp8_workspace: sizes out of range")
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def ple_tree_attention_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           k_scale: torch.Tensor, v_scale: torch.Tensor,
                           page_table: torch.Tensor, ctx_lens: torch.Tensor,
                           cu_seqlens: torch.Tensor, tree_mask: torch.Tensor,
                           scale: float | None = None, out: torch.Tensor | None = None,
                           lse: torch.Tensor | None = None, return_lse: bool = False,
                           workspace: torch.Tensor | None = None, stream=None):
    """ple_tree_attention over a cache in 8 bits.

    q [T, q_heads, D] in bfloat16 or float16; the other arguments and the
    results as there, workspace being ple_tree_attention_fp8_workspace's.  Keys
    and values enter as element times scale; nothing else is rounded to 8 bits."""
    where = "ple_tree_attention_fp8"
    dev = q.get_device()
    dtype = q.dtype
    element = _ELEMENTS.get(dtype)
    if element is None or q.dim() != 3 or k_cache.dim() != 4 or k_scale.dim() != 3:
        _device(where, q, k_cache, v_cache, k_scale, v_scale)
        _element(q, "q", where)
        raise ValueError(f"{where}: q must be [T, q_heads, head_dim], the caches [pages, "
                         "kv_heads, page_size, head_dim] and the scales [pages, kv_heads, blocks]")
    T, Hq, D = q.shape
    cache_shape = k_cache.shape
    pages, Hk, page_size, cache_dim = cache_shape
    qs, strides = q.stride(), k_cache.stride()
    scale_strides, scale_shape = k_scale.stride(), k_scale.shape
    blocks = scale_shape[2]
    block = page_size // blocks if blocks else 0
    B = ctx_lens.shape[0] if ctx_lens.dim() == 1 else -1
    table_shape, mask_shape = page_table.shape, tree_mask.shape
    if not (out is None and lse is None and workspace is None and dev >= 0 and B >= 0
            and k_cache.dtype is _fp8 and v_cache.dtype is _fp8 and k_scale.dtype is _bf16
            and v_scale.dtype is _bf16 and page_table.dtype is _i32 and ctx_lens.dtype is _i32
            and cu_seqlens.dtype is _i32 and tree_mask.dtype is _i64
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and k_scale.get_device() == dev and v_scale.get_device() == dev
            and page_table.get_device() == dev and ctx_lens.get_device() == dev
            and cu_seqlens.get_device() == dev and tree_mask.get_device() == dev
            and qs[2] == 1 and v_cache.shape == cache_shape and v_cache.stride() == strides
            and strides[3] == 1 and cache_dim == D and Hk >= 1 and Hq % Hk == 0
            and scale_shape[:2] == cache_shape[:2] and v_scale.shape == scale_shape
            and v_scale.stride() == scale_strides and scale_strides[2] == 1
            and block * blocks == page_size and block in _BLOCKS
            and cu_seqlens.shape == (B + 1,) and len(table_shape) == 2 and table_shape[0] == B
            and len(mask_shape) == 2 and mask_shape[0] == T and page_table.is_contiguous()
            and ctx_lens.is_contiguous() and cu_seqlens.is_contiguous()
            and tree_mask.is_contiguous()):
        dev = _device(where, q, k_cache, v_cache, k_scale, v_scale, page_table, ctx_lens,
                      cu_seqlens, tree_mask, out, lse, workspace)
        _heads(q, dtype, T, Hq, D, "q", where)
        block = _caches8(k_cache, v_cache, k_scale, v_scale, 4, where)
        if cache_dim != D or Hk < 1 or Hq % Hk:
            raise ValueError(f"{where}: the caches' heads must divide q's and have their width")
        _vector(ctx_lens, _i32, B, "ctx_lens", where)
        _vector(cu_seqlens, _i32, B + 1, "cu_seqlens", where)
        _table(page_table, _i32, B, "page_table", where)
        _table(tree_mask, _i64, T, "tree_mask", where)
        if out is not None and (out.dtype != dtype or out.shape != q.shape
                                or not out.is_contiguous()):
            raise ValueError(f"{where}: out must be contiguous, of q's shape and dtype")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, Hq)
                                or not lse.is_contiguous()):
            raise ValueError(f"{where}: lse must be a contiguous float32 [T, q_heads]")
        if workspace is not None and (workspace.dtype != torch.uint8 or workspace.dim() != 1
                                      or not workspace.is_contiguous()):
            raise ValueError(f"{where}: workspace must be a contiguous uint8 tensor")
    device = q.device
    made = []
    if out is None:
        out = _empty((T, Hq, D), dtype=dtype, device=device)
        made.append(out)
    if lse is None and return_lse:
        lse = _empty((T, Hq), dtype=torch.float32, device=device)
        made.append(lse)
    if workspace is None:
        workspace = _empty(_workspace_size(T, Hq, Hk, D, dev), dtype=torch.uint8, device=device)
        made.append(workspace)
    _lend(stream, dev, *made)
    args = _ATTENTION8.pack(
        q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), strides[0],
        strides[1], strides[2], pages, page_table.data_ptr(), ctx_lens.data_ptr(),
        cu_seqlens.data_ptr(), tree_mask.data_ptr(), out.data_ptr(),
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.shape[0], T, B,
        table_shape[1], page_size, element, Hq, Hk, D, mask_shape[1],
        D ** -0.5 if scale is None else scale, k_scale.data_ptr(), v_scale.data_ptr(), 0,
        scale_strides[0], scale_strides[1], block)
    _call(where, lib().ple_tree_attention_fp8, dev, stream, args)
    return (out, lse) if return_lse else out


def ple_tree_commit_fp8(input_ids: torch.Tensor, path: torch.Tensor, accepted: torch.Tensor,
                        cu_seqlens: torch.Tensor, ngram_context: torch.Tensor | None,
                        ctx_lens: torch.Tensor, page_table: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                        next_context: torch.Tensor | None = None,
                        next_ctx_lens: torch.Tensor | None = None, stream=None):
    """(next_context, next_ctx_lens): ple_tree_commit in a cache in 8 bits.

    Arguments and results as there; caches and scales of all layers
    ([layers, pages, ...]) or of one.  A block that kept tokens move to takes the
    largest of the scales that they had."""
    where = "ple_tree_commit_fp8"
    dev = input_ids.get_device()
    if k_cache.dim() == 4 and v_cache.dim() == 4 and k_scale.dim() == 3 and v_scale.dim() == 3:
        k_cache, v_cache = k_cache.unsqueeze(0), v_cache.unsqueeze(0)
        k_scale, v_scale = k_scale.unsqueeze(0), v_scale.unsqueeze(0)
    kind = input_ids.dtype
    ids = _IDS.get(kind)
    if k_cache.dim() != 5 or k_scale.dim() != 4:
        _device(where, input_ids, k_cache, k_scale)
        raise ValueError(f"{where}: the caches must be [layers, pages, kv_heads, page_size, "
                         "head_dim] and the scales [layers, pages, kv_heads, blocks], or one "
                         "layer's")
    strides, cache_shape = k_cache.stride(), k_cache.shape
    scale_strides, scale_shape = k_scale.stride(), k_scale.shape
    blocks = scale_shape[3]
    block = cache_shape[3] // blocks if blocks else 0
    T, B = input_ids.shape[0], ctx_lens.shape[0]
    path_shape, table_shape = path.shape, page_table.shape
    if not (ids is not None and next_context is None and next_ctx_lens is None
            and ngram_context is not None and dev >= 0
            and k_cache.dtype is _fp8 and v_cache.dtype is _fp8 and k_scale.dtype is _bf16
            and v_scale.dtype is _bf16 and path.dtype is _i32 and accepted.dtype is _i32
            and cu_seqlens.dtype is _i32 and ctx_lens.dtype is _i32
            and page_table.dtype is _i32 and ngram_context.dtype is kind
            and path.get_device() == dev and accepted.get_device() == dev
            and cu_seqlens.get_device() == dev and ngram_context.get_device() == dev
            and ctx_lens.get_device() == dev and page_table.get_device() == dev
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and k_scale.get_device() == dev and v_scale.get_device() == dev
            and input_ids.dim() == 1 and ctx_lens.dim() == 1 and accepted.shape == (B,)
            and cu_seqlens.shape == (B + 1,) and len(path_shape) == 2 and path_shape[0] == B
            and len(table_shape) == 2 and table_shape[0] == B and ngram_context.dim() == 2
            and ngram_context.shape[0] == B and v_cache.shape == cache_shape
            and v_cache.stride() == strides and strides[4] == 1
            and scale_shape[:3] == cache_shape[:3] and v_scale.shape == scale_shape
            and v_scale.stride() == scale_strides and scale_strides[3] == 1
            and block * blocks == cache_shape[3] and block in _BLOCKS
            and input_ids.is_contiguous() and path.is_contiguous()
            and accepted.is_contiguous() and cu_seqlens.is_contiguous()
            and ngram_context.is_contiguous() and ctx_lens.is_contiguous()
            and page_table.is_contiguous()):
        dev = _device(where, input_ids, path, accepted, cu_seqlens, ngram_context, ctx_lens,
                      page_table, k_cache, v_cache, k_scale, v_scale, next_context,
                      next_ctx_lens)
        block = _caches8(k_cache, v_cache, k_scale, v_scale, 5, where)
        if ids is None:
            raise TypeError(f"{where}: input_ids must be int32 or int64")
        _vector(input_ids, kind, T, "input_ids", where)
        _vector(ctx_lens, _i32, B, "ctx_lens", where)
        _vector(accepted, _i32, B, "accepted", where)
        _vector(cu_seqlens, _i32, B + 1, "cu_seqlens", where)
        _table(path, _i32, B, "path", where)
        _table(page_table, _i32, B, "page_table", where)
        if ngram_context is not None:
            _table(ngram_context, kind, B, "ngram_context", where)
            if next_context is not None:
                _table(next_context, kind, B, "next_context", where)
                if next_context.shape != ngram_context.shape:
                    raise ValueError(f"{where}: next_context must have ngram_context's shape")
        elif next_context is not None:
            raise ValueError(f"{where}: next_context needs ngram_context")
        if next_ctx_lens is not None:
            _vector(next_ctx_lens, _i32, B, "next_ctx_lens", where)
        for name, t in (("next_context", next_context), ("next_ctx_lens", next_ctx_lens)):
            for other, u in (("input_ids", input_ids), ("path", path), ("accepted", accepted),
                             ("cu_seqlens", cu_seqlens), ("ngram_context", ngram_context),
                             ("ctx_lens", ctx_lens), ("page_table", page_table),
                             ("next_ctx_lens", next_ctx_lens)):
                if t is not None and u is not None and name != other and _overlap(t, u):
                    raise ValueError(f"{where}: {name} must not overlap {other}")
    C = 0 if ngram_context is None else ngram_context.shape[1]
    made = []
    if next_context is None and ngram_context is not None:
        next_context = _empty((B, C), dtype=kind, device=input_ids.device)
        made.append(next_context)
    if next_ctx_lens is None:
        next_ctx_lens = _empty(B, dtype=_i32, device=input_ids.device)
        made.append(next_ctx_lens)
    _lend(stream, dev, *made)
    L, pages, Hk, page_size, D = cache_shape
    args = _COMMIT8.pack(
        input_ids.data_ptr(), path.data_ptr() if path_shape[1] else 0, accepted.data_ptr(),
        cu_seqlens.data_ptr(), 0 if C == 0 else ngram_context.data_ptr(),
        0 if C == 0 else next_context.data_ptr(), ctx_lens.data_ptr(), next_ctx_lens.data_ptr(),
        page_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1],
        strides[2], strides[3], pages, T, B, path_shape[1], ids, C, L, table_shape[1], page_size,
        Hk, D, 0, k_scale.data_ptr(), v_scale.data_ptr(), scale_strides[0], scale_strides[1],
        scale_strides[2], block)
    _call(where, lib().ple_tree_commit_fp8, dev, stream, args)
    return next_context, next_ctx_lens


def ple_plan_pages(page_table: torch.Tensor, ctx_lens: torch.Tensor, source: torch.Tensor,
                   want: torch.Tensor, num_pages: int, page_size: int, limit: int | None = None,
                   stream=None):
    """(next_table, next_ctx_lens, copies, counts): the next step's pages.

    page_table [B, max_pages], ctx_lens [B]: the present requests.  source,
    want [N]: for each row of the next batch the request that it goes on with
    (several rows may take the same one: it forks; -1 begins an empty one; a
    request that no row takes has ended), and how many tokens will be appended
    to it.  All int32.

    Rows share the pages of their common past; the page that a row's new tokens
    start in, if others hold it too, is doubled, and what new tokens need besides
    are free pages, the lowest first.  With limit, pages from that number on move
    below it, so that the cache's end can be given back.  next_table [N, max_pages]
    has -1 where a row has no page.  copies [N + num_pages - limit, 2] lists
    (from, to) for ple_copy_pages, which has to run before the next append, and
    (-1, -1) behind them.  counts [3]: copies, pages in use, pages that were
    missing; if any were, the plan is not to be used: the old tables stand."""
    where = "ple_plan_pages"
    dev = page_table.get_device()
    P, page_size = int(num_pages), int(page_size)
    L = P if limit is None else int(limit)
    B = ctx_lens.shape[0] if ctx_lens.dim() == 1 else -1
    N = source.shape[0] if source.dim() == 1 else -1
    table_shape = page_table.shape
    if not (dev >= 0 and page_table.dtype is _i32 and ctx_lens.dtype is _i32
            and source.dtype is _i32 and want.dtype is _i32 and ctx_lens.get_device() == dev
            and source.get_device() == dev and want.get_device() == dev and B >= 0 and N >= 1
            and len(table_shape) == 2 and table_shape[0] == B and want.shape == (N,)
            and 0 <= L <= P and page_table.is_contiguous() and ctx_lens.is_contiguous()
            and source.is_contiguous() and want.is_contiguous()):
        dev = _device(where, page_table, ctx_lens, source, want)
        _vector(ctx_lens, _i32, B, "ctx_lens", where)
        _table(page_table, _i32, B, "page_table", where)
        _vector(source, _i32, N, "source", where)
        _vector(want, _i32, N, "want", where)
        if N < 1:
            raise ValueError(f"{where}: the next batch must have a row")
        if not 0 <= L <= P:
            raise ValueError(f"{where}: limit must be from 0 to num_pages")
    if not 0 < page_size < 2 ** 31:
        raise ValueError(f"{where}: page_size must be positive, below 2^31")
    device, M = page_table.device, table_shape[1]
    if N * M > 2 ** 31 - 1 - P:
        raise ValueError(f"{where}: num_rows * max_pages + num_pages must stay below 2^31")
    size = lib().ple_plan_pages_workspace(N, P) // 4 if 0 < P < 2 ** 31 else 0
    # one piece of memory for tables, lengths, copies and counts; the call's own is another, so
    # that it is not kept as long as they are
    lens_at = (N * M + 3) // 4 * 4
    copies_at = lens_at + (N + 3) // 4 * 4
    counts_at = copies_at + (2 * (N + P - L) + 3) // 4 * 4
    memory = _empty(counts_at + 4, dtype=_i32, device=device)
    workspace = _empty(max(size, 0), dtype=_i32, device=device)
    _lend(stream, dev, memory, workspace)
    next_table = memory.as_strided((N, M), (M, 1))
    next_ctx_lens = memory.as_strided((N,), (1,), lens_at)
    copies = memory.as_strided((N + P - L, 2), (2, 1), copies_at)
    counts = memory.as_strided((3,), (1,), counts_at)
    args = _PLAN.pack(
        page_table.data_ptr(), ctx_lens.data_ptr(), source.data_ptr(), want.data_ptr(),
        next_table.data_ptr(), next_ctx_lens.data_ptr(), copies.data_ptr(), counts.data_ptr(),
        workspace.data_ptr(), 4 * max(size, 0), B, N, M, page_size, P, L)
    _call(where, lib().ple_plan_pages, dev, stream, args)
    return next_table, next_ctx_lens, copies, counts


def ple_copy_pages(copies: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                   stream=None) -> None:
    """Copies pages in place in the caches of all layers ([layers, pages,
    kv_heads, page_size, head_dim]) or of one (without the first dimension).

    copies [n, 2] int32: (from, to), as of ple_plan_pages; entries with a number
    that is no page are passed over.  No page may be both copied from and copied
    to, or copied to twice.  Caches of bfloat16, float16 or, with their scales,
    float8_e4m3fn."""
    where = "ple_copy_pages"
    if k_cache.dim() == 4 and v_cache.dim() == 4:
        k_cache, v_cache = k_cache.unsqueeze(0), v_cache.unsqueeze(0)
        if k_scale is not None and v_scale is not None:
            k_scale, v_scale = k_scale.unsqueeze(0), v_scale.unsqueeze(0)
    dev = _device(where, copies, k_cache, v_cache, k_scale, v_scale)
    block, scale_strides = 0, (0, 0, 0)
    if k_scale is not None or v_scale is not None:
        if k_scale is None or v_scale is None:
            raise ValueError(f"{where}: pass both scales or neither")
        block = _caches8(k_cache, v_cache, k_scale, v_scale, 5, where)
        scale_strides = k_scale.stride()
    else:
        if k_cache.dtype == _fp8:
            raise ValueError(f"{where}: a cache in 8 bits needs its scales")
        _element(k_cache, "the caches", where)
        _caches(k_cache, v_cache, k_cache.dtype, 5, where)
    if copies.dtype != _i32:
        raise TypeError(f"{where}: copies must be {_i32}, got {copies.dtype}")
    if copies.dim() != 2 or copies.shape[1] != 2 or not copies.is_contiguous():
        raise ValueError(f"{where}: copies must be contiguous, [n, 2]; got {tuple(copies.shape)}")
    strides = k_cache.stride()
    layers, pages, Hk, page_size, D = k_cache.shape
    args = _COPY.pack(
        copies.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1],
        strides[2], strides[3], k_scale.data_ptr() if block else 0,
        v_scale.data_ptr() if block else 0, scale_strides[0], scale_strides[1], scale_strides[2],
        block, pages, copies.shape[0], layers, Hk, page_size, D, k_cache.element_size())
    _call(where, lib().ple_copy_pages, dev, stream, args)
