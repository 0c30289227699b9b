"""Binding of the tree-verification entry points (argument marshalling only).

A request drafts a tree of tokens behind its cached ones and verifies all of
them in one pass of the model.  These functions are what the pass needs
besides its matrix products: positions and ancestor masks
(ple_build_tree_index), row ids along the branches (ple_tree_row_ids), norms,
rotation and cache append (ple_prepare_rope, ple_qk_norm_rope), attention over
the paged cache (ple_tree_attention) and the commit of the accepted branches
(ple_tree_commit).

As in binding.py every function checks and converts its arguments and calls
the C ABI entry point of its name; tensors that are not all on one CUDA device
are refused with ValueError, and there is no CPU path.  A verification step
makes most of these calls once per layer, and a small one lasts a few
microseconds on the device, so each function first tests its arguments in one
expression; only when that fails do the checks that name the culprit run.

`stream` defaults to the device's current stream.  Outputs and workspaces that
a call is not given come from torch's allocator, from the current stream's
memory: on another stream such a call first makes that stream wait for the
current one.  A caller that orders the streams itself passes them all.

These operators serve and are no part of autograd's graph: outputs never require
gradients, whatever the inputs do, and what a call writes into caches and given
outputs does not move their version counters.

Caches are [pages, kv_heads, page_size, head_dim] views (for the commit of
several layers [layers, pages, kv_heads, page_size, head_dim]): any strides
that are multiples of 8 elements with the last dimension contiguous, the same
ones for keys and values.
"""

from __future__ import annotations

import struct

import torch

from .binding import (PLE_BF16, PLE_F16, PLE_HEAD_BYTES, PLE_I32, PLE_I64, PLE_OK,
                      PLE_ROPE_BASE, PLE_ROPE_LINEAR, PLE_ROPE_PARTS, PLE_ROPE_PLAIN, _check, _lend,
                      lib)

ROPE_SCALINGS = {"plain": PLE_ROPE_PLAIN, "linear": PLE_ROPE_LINEAR, "base": PLE_ROPE_BASE,
                 "parts": PLE_ROPE_PARTS}
_ELEMENTS = {torch.bfloat16: PLE_BF16, torch.float16: PLE_F16}
_IDS = {torch.int32: PLE_I32, torch.int64: PLE_I64}

# the argument structs of include/ple.h, field by field
_NORM_ROPE = struct.Struct("@PPPqqqqqqPPPPPqqPqqPPqqqqPPPqiiiiiiiiiff")
_ATTENTION = struct.Struct("@PqqPPqqqqPPPPPPPqqiiiiiiiif")
_COMMIT = struct.Struct("@PPPPPPPPPPPqqqqqqiiiiiiiiii")


def _device(where: str, *tensors) -> int:
    """The index of the one CUDA device that every given tensor is on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            dev = -1
    if dev < 0:
        raise ValueError(f"{where}: every tensor must be on one CUDA device (got "
                         f"{sorted({str(t.device) for t in tensors if t is not None})})")
    return dev


_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty
_i32, _i64 = torch.int32, torch.int64


def _call(where: str, fn, dev: int, stream, *args):
    """Call a library function on the tensors' device and the given (or the
    device's current) stream."""
    handle = _current_stream(dev) if stream is None else stream.cuda_stream
    if _current_device() == dev:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != PLE_OK:
        _check(status, where)


def _vector(t: torch.Tensor, dtype, n: int, name: str, where: str):
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous, [{n}]; got {tuple(t.shape)}")


def _table(t: torch.Tensor, dtype, rows: int, name: str, where: str):
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != rows or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous with {rows} rows; got "
                         f"{tuple(t.shape)}")


def _heads(t: torch.Tensor, dtype, T: int, heads, dim, name: str, where: str):
    """Head rows [T, heads, dim] with the last dimension contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != T or (heads is not None and t.shape[1] != heads) or \
            t.shape[2] != dim:
        raise ValueError(f"{where}: {name} must be [{T}, {'heads' if heads is None else heads}, "
                         f"{dim}]; got {tuple(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{where}: {name}'s last dimension must be contiguous")


def _caches(k: torch.Tensor, v: torch.Tensor, dtype, dims: int, where: str):
    """The two caches' common strides."""
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError(f"{where}: the caches must be {dtype}, got {k.dtype} and {v.dtype}")
    strides = k.stride()
    if k.dim() != dims or k.shape != v.shape or strides != v.stride() or strides[-1] != 1:
        raise ValueError(f"{where}: the caches must be {'[layers, ' if dims == 5 else '['}pages, "
                         "kv_heads, page_size, head_dim] with one shape and the same strides, the "
                         "last dimension contiguous")
    return strides


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two contiguous tensors share a byte."""
    x, y = a.data_ptr(), b.data_ptr()
    n, m = a.numel() * a.element_size(), b.numel() * b.element_size()
    return n > 0 and m > 0 and x < y + m and y < x + n


def _element(t: torch.Tensor, name: str, where: str) -> int:
    code = _ELEMENTS.get(t.dtype)
    if code is None:
        raise TypeError(f"{where}: {name} must be bfloat16 or float16, got {t.dtype}")
    return code


def ple_build_tree_index(parent: torch.Tensor, cu_seqlens: torch.Tensor, ctx_lens: torch.Tensor,
                         mask_words: int, positions: torch.Tensor | None = None,
                         tree_mask: torch.Tensor | None = None, stream=None):
    """(positions [T] int32, tree_mask [T, mask_words] int64) of drafted trees.

    parent [T] int32: the place within its own request of each node's parent,
    or -1; parents come before children.  cu_seqlens [B + 1], ctx_lens [B]:
    int32.  A position is the request's cached length plus the node's depth;
    bit j of a mask (64 to a word) is set for the node itself and its
    ancestors.  mask_words words hold trees of up to 64 * mask_words nodes."""
    where = "ple_build_tree_index"
    dev = parent.get_device()
    T, B, W = parent.shape[0], ctx_lens.shape[0], int(mask_words)
    if not (positions is None and tree_mask is None and dev >= 0
            and parent.dtype is _i32 and cu_seqlens.dtype is _i32 and ctx_lens.dtype is _i32
            and cu_seqlens.get_device() == dev and ctx_lens.get_device() == dev
            and parent.dim() == 1 and ctx_lens.dim() == 1 and cu_seqlens.shape == (B + 1,)
            and parent.is_contiguous() and cu_seqlens.is_contiguous()
            and ctx_lens.is_contiguous()):
        dev = _device(where, parent, cu_seqlens, ctx_lens, positions, tree_mask)
        _vector(parent, _i32, T, "parent", where)
        _vector(cu_seqlens, _i32, B + 1, "cu_seqlens", where)
        _vector(ctx_lens, _i32, B, "ctx_lens", where)
        if positions is not None:
            _vector(positions, _i32, T, "positions", where)
        if tree_mask is not None:
            _table(tree_mask, _i64, T, "tree_mask", where)
            if tree_mask.shape[1] != W:
                raise ValueError(f"{where}: tree_mask must be [T, mask_words]")
    made = []
    if positions is None:
        positions = _empty(T, dtype=_i32, device=parent.device)
        made.append(positions)
    if tree_mask is None:
        tree_mask = _empty((T, max(W, 0)), dtype=_i64, device=parent.device)
        made.append(tree_mask)
    _lend(stream, dev, *made)
    _call(where, lib().ple_build_tree_index, dev, stream, parent.data_ptr(),
          cu_seqlens.data_ptr(), ctx_lens.data_ptr(), B, T, W, positions.data_ptr(),
          tree_mask.data_ptr())
    return positions, tree_mask


def ple_tree_row_ids(input_ids: torch.Tensor, parent: torch.Tensor, cu_seqlens: torch.Tensor,
                     ngram_context: torch.Tensor, layer_multipliers: torch.Tensor,
                     vocab_sizes: torch.Tensor, offsets: torch.Tensor, ngram_size: int,
                     heads_per_ngram: int, boundary_id: int, out: torch.Tensor | None = None,
                     stream=None, out_dtype=torch.int64,
                     heads: torch.Tensor | None = None) -> torch.Tensor:
    """Row ids [L, T, H] of drafted trees (one launch for every layer).

    ple_row_ids with each window taken along the node's branch: the ids of its
    ancestors, then the carried context.  parent [T] and cu_seqlens [B + 1]:
    int32, as for ple_build_tree_index; the other arguments as ple_row_ids."""
    where = "ple_tree_row_ids"
    dev = input_ids.get_device()
    kind = input_ids.dtype
    ids, out_code = _IDS.get(kind), _IDS.get(out_dtype)
    N, T = int(ngram_size), input_ids.shape[0]
    M = layer_multipliers.reshape(1, -1) if layer_multipliers.dim() == 1 else layer_multipliers
    vocab = vocab_sizes.reshape(1, -1) if vocab_sizes.dim() == 1 else vocab_sizes
    off = offsets.reshape(1, -1) if offsets.dim() == 1 else offsets
    shape = vocab.shape
    B, C = ngram_context.shape if ngram_context.dim() == 2 else (-1, -1)
    if not (out is None and heads is None and dev >= 0 and ids is not None
            and out_code is not None and ngram_context.dtype is kind and parent.dtype is _i32
            and cu_seqlens.dtype is _i32 and M.dtype is _i64 and vocab.dtype is _i64
            and off.dtype is _i64 and parent.get_device() == dev
            and cu_seqlens.get_device() == dev and ngram_context.get_device() == dev
            and M.get_device() == dev and vocab.get_device() == dev and off.get_device() == dev
            and B >= 0 and cu_seqlens.shape == (B + 1,) and input_ids.dim() == 1
            and parent.shape == (T,) and len(shape) == 2 and off.shape == shape
            and M.shape == (shape[0], N) and input_ids.is_contiguous() and parent.is_contiguous()
            and cu_seqlens.is_contiguous() and ngram_context.is_contiguous()
            and M.is_contiguous() and vocab.is_contiguous() and off.is_contiguous()):
        dev = _device(where, input_ids, parent, cu_seqlens, ngram_context, layer_multipliers,
                      vocab_sizes, offsets, out, heads)
        if ids is None or ngram_context.dtype != kind:
            raise TypeError(f"{where}: input_ids and ngram_context must share int32 or int64")
        _vector(input_ids, kind, T, "input_ids", where)
        _vector(parent, _i32, T, "parent", where)
        _table(ngram_context, kind, B, "ngram_context", where)
        _vector(cu_seqlens, _i32, B + 1, "cu_seqlens", where)
        _table(vocab, _i64, shape[0], "vocab_sizes", where)
        _table(M, _i64, shape[0], "layer_multipliers", where)
        _table(off, _i64, shape[0], "offsets", where)
        if M.shape[1] != N or off.shape[1] != shape[1]:
            raise ValueError(f"{where}: layer_multipliers must be [L, ngram_size], offsets must "
                             "have the shape of vocab_sizes")
        if out_code is None:
            raise TypeError(f"{where}: out_dtype must be torch.int64 or torch.int32")
        if out is not None and (out.dtype != out_dtype or not out.is_contiguous()
                                or out.shape != (shape[0], T, shape[1])):
            raise ValueError(f"{where}: out must be a contiguous {out_dtype} [L, T, H]")
        if heads is not None and (heads.dtype != torch.uint8 or not heads.is_contiguous()
                                  or heads.shape != (shape[0], shape[1], PLE_HEAD_BYTES)):
            raise ValueError(f"{where}: heads must be ple_prepare_heads' [L, H, "
                             f"{PLE_HEAD_BYTES}]")
    L, H = shape
    if out is None:
        out = _empty((L, T, H), dtype=out_dtype, device=input_ids.device)
        _lend(stream, dev, out)
    _call(where, lib().ple_tree_row_ids, dev, stream, input_ids.data_ptr(), ids, T,
          parent.data_ptr(), cu_seqlens.data_ptr(), ngram_context.data_ptr(), B, C, M.data_ptr(),
          vocab.data_ptr(), off.data_ptr(), H, N, int(heads_per_ngram), L, int(boundary_id),
          out.data_ptr(), out_code, None if heads is None else heads.data_ptr())
    return out


def ple_prepare_rope(rotary_dim: int, base: float = 10000.0, scaling: str = "plain",
                     factor: float = 1.0, trained_positions: float = 0.0,
                     beta_fast: float = 32.0, beta_slow: float = 1.0,
                     out: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """[rotary_dim / 2] int64: the rotation of each pair per position, in 2^-64
    turns, set up once and passed to ple_qk_norm_rope call after call.

    Pair i turns by base^(-2i / rotary_dim) radians a position.  For contexts
    beyond the trained ones: scaling "linear" divides every angle by factor,
    "base" raises the base so that the slowest pair slows by factor, "parts"
    keeps the pairs that turn more than beta_fast times over
    trained_positions, divides those that turn less than beta_slow times, and
    mixes between (then 0.1 * ln(factor) + 1 is the usual rope_scale).

    The mix goes linearly over turns (Peng et al. 2023).  A checkpoint whose
    code ramps linearly over the pairs' indices instead has other angles, and
    like any other frequencies w [rotary_dim / 2] below pi radians a position they
    make a table of their own: (w.double() / (2 * pi) * 2.0 ** 64).long()."""
    where = "ple_prepare_rope"
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"{where}: scaling must be one of {sorted(ROPE_SCALINGS)}")
    R = int(rotary_dim)
    if out is None:
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise ValueError(f"{where}: the rotation is kept on a CUDA device, got {device}")
        out = torch.empty(max(R // 2, 0), dtype=torch.int64, device=device)
        _lend(stream, device, out)
    dev = _device(where, out)
    _vector(out, torch.int64, R // 2, "out", where)
    _call(where, lib().ple_prepare_rope, dev, stream, R, float(base), ROPE_SCALINGS[scaling],
          float(factor), float(trained_positions), float(beta_fast), float(beta_slow),
          out.data_ptr())
    return out


def ple_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor | None,
                     positions: torch.Tensor | None, rope: torch.Tensor | None,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                     k_cache: torch.Tensor | None = None, v_cache: torch.Tensor | None = None,
                     page_table: torch.Tensor | None = None,
                     ctx_lens: torch.Tensor | None = None,
                     cu_seqlens: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, rope_scale: float = 1.0,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     stream=None):
    """Norms of queries and keys per head, their rotation, and the append of
    keys and values to the paged cache, in one launch.

    q [T, q_heads, D], k and v [T, kv_heads, D]: bfloat16 or float16, views of
    one product allowed (strides multiples of 8 elements, the last dimension
    contiguous).  q_weight / k_weight [D]: the norms' weights; None leaves the
    rows without a norm.  rope: ple_prepare_rope's, rotating the first
    2 * len(rope) elements at `positions` [T] int32 (pairs half of them apart,
    or side by side when interleaved); None rotates nothing.

    With a cache: node j of request r is written to cached token
    ctx_lens[r] + j through page_table [B, max_pages], and q_out is returned.
    Without one v is not read and (q_out, k_out) is returned.  q_out and k_out
    may be q and k themselves."""
    where = "ple_qk_norm_rope"
    dev = q.get_device()
    dtype = q.dtype
    element = _ELEMENTS.get(dtype)
    if element is None or q.dim() != 3 or k.dim() != 3:
        _device(where, q, k)
        _element(q, "q", where)
        raise ValueError(f"{where}: q must be [T, q_heads, head_dim] and k [T, kv_heads, head_dim]")
    T, Hq, D = q_shape = q.shape
    k_shape = k.shape
    Hk = k_shape[1]
    R = 0 if rope is None else 2 * rope.shape[0]
    qs, ks = q.stride(), k.stride()
    cached = k_cache is not None
    # the step of a serving loop: norms, a rotation and a cache, new queries
    quick = (cached and q_out is None and k_out is None and rope is not None
             and positions is not None and q_weight is not None and k_weight is not None
             and v is not None and v_cache is not None and page_table is not None
             and ctx_lens is not None and cu_seqlens is not None and dev >= 0
             and k.dtype is dtype and v.dtype is dtype and q_weight.dtype is dtype
             and k_weight.dtype is dtype and k_cache.dtype is dtype and v_cache.dtype is dtype
             and positions.dtype is _i32 and rope.dtype is _i64 and page_table.dtype is _i32
             and ctx_lens.dtype is _i32 and cu_seqlens.dtype is _i32
             and k.get_device() == dev and v.get_device() == dev
             and q_weight.get_device() == dev and k_weight.get_device() == dev
             and k_cache.get_device() == dev and v_cache.get_device() == dev
             and positions.get_device() == dev and rope.get_device() == dev
             and page_table.get_device() == dev and ctx_lens.get_device() == dev
             and cu_seqlens.get_device() == dev)
    if quick:
        B = ctx_lens.shape[0]
        v_strides, cache_strides, cache_shape = v.stride(), k_cache.stride(), k_cache.shape
        table_shape = page_table.shape
        quick = (k_shape[0] == T and k_shape[2] == D and v.shape == k_shape
                 and qs[2] == 1 and ks[2] == 1 and v_strides[2] == 1
                 and q_weight.shape == (D,) and k_weight.shape == (D,)
                 and positions.shape == (T,) and rope.dim() == 1
                 and len(cache_shape) == 4 and v_cache.shape == cache_shape
                 and v_cache.stride() == cache_strides and cache_strides[3] == 1
                 and cache_shape[1] == Hk and cache_shape[3] == D and ctx_lens.dim() == 1
                 and cu_seqlens.shape == (B + 1,) and len(table_shape) == 2
                 and table_shape[0] == B and q_weight.is_contiguous()
                 and k_weight.is_contiguous() and positions.is_contiguous()
                 and rope.is_contiguous() and page_table.is_contiguous()
                 and ctx_lens.is_contiguous() and cu_seqlens.is_contiguous())
    if quick:
        q_out = _empty(q_shape, dtype=dtype, device=q.device)
        _lend(stream, dev, q_out)
        args = _NORM_ROPE.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], v_strides[0],
            v_strides[1], positions.data_ptr(), rope.data_ptr(), q_weight.data_ptr(),
            k_weight.data_ptr(), q_out.data_ptr(), Hq * D, D, 0, 0, 0, k_cache.data_ptr(),
            v_cache.data_ptr(), cache_strides[0], cache_strides[1], cache_strides[2],
            cache_shape[0], page_table.data_ptr(), ctx_lens.data_ptr(), cu_seqlens.data_ptr(), T,
            B, table_shape[1], cache_shape[2], element, Hq, Hk, D, R, 1 if interleaved else 0,
            rope_scale, eps)
        _call(where, lib().ple_qk_norm_rope, dev, stream, args)
        return q_out

    dev = _device(where, q, k, v, positions, rope, q_weight, k_weight, k_cache, v_cache,
                  page_table, ctx_lens, cu_seqlens, q_out, k_out)
    _heads(q, dtype, T, None, D, "q", where)
    _heads(k, dtype, T, None, D, "k", where)
    if rope is not None:
        _vector(rope, _i64, rope.shape[0], "rope", where)
        if positions is None:
            raise ValueError(f"{where}: a rotation needs positions")
        _vector(positions, _i32, T, "positions", where)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _vector(w, dtype, D, name, where)
    made = []
    if q_out is None:
        q_out = _empty((T, Hq, D), dtype=dtype, device=q.device)
        made.append(q_out)
    else:
        _heads(q_out, dtype, T, Hq, D, "q_out", where)
    pages = B = 0
    cache_strides = (0, 0, 0, 0)
    page_size = max_pages = 1
    v_strides = k_out_strides = (0, 0, 0)
    if cached:
        if v is None or v_cache is None or page_table is None or ctx_lens is None or \
                cu_seqlens is None:
            raise ValueError(f"{where}: a cache needs v, v_cache, page_table, ctx_lens and "
                             "cu_seqlens")
        if k_out is not None:
            raise ValueError(f"{where}: pass a cache or k_out, not both")
        _heads(v, dtype, T, Hk, D, "v", where)
        v_strides = v.stride()
        cache_strides = _caches(k_cache, v_cache, dtype, 4, where)
        pages, page_size, B = k_cache.shape[0], k_cache.shape[2], ctx_lens.shape[0]
        if k_cache.shape[1] != Hk or k_cache.shape[3] != D:
            raise ValueError(f"{where}: the caches must be [pages, {Hk}, page_size, {D}]")
        _vector(ctx_lens, _i32, B, "ctx_lens", where)
        _vector(cu_seqlens, _i32, B + 1, "cu_seqlens", where)
        _table(page_table, _i32, B, "page_table", where)
        max_pages = page_table.shape[1]
    else:
        if v_cache is not None:
            raise ValueError(f"{where}: pass both caches or neither")
        if k_out is None:
            k_out = _empty((T, Hk, D), dtype=dtype, device=q.device)
            made.append(k_out)
        else:
            _heads(k_out, dtype, T, Hk, D, "k_out", where)
        k_out_strides = k_out.stride()
    _lend(stream, dev, *made)
    os = q_out.stride()
    args = _NORM_ROPE.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr() if cached else 0, qs[0], qs[1], ks[0], ks[1],
        v_strides[0], v_strides[1], 0 if positions is None else positions.data_ptr(),
        rope.data_ptr() if R else 0, 0 if q_weight is None else q_weight.data_ptr(),
        0 if k_weight is None else k_weight.data_ptr(), q_out.data_ptr(), os[0], os[1],
        0 if cached else k_out.data_ptr(), k_out_strides[0], k_out_strides[1],
        k_cache.data_ptr() if cached else 0, v_cache.data_ptr() if cached else 0,
        cache_strides[0], cache_strides[1], cache_strides[2], pages,
        page_table.data_ptr() if cached else 0, ctx_lens.data_ptr() if cached else 0,
        cu_seqlens.data_ptr() if cached else 0, T, B, max_pages, page_size, element, Hq, Hk, D, R,
        1 if interleaved else 0, rope_scale, eps)
    _call(where, lib().ple_qk_norm_rope, dev, stream, args)
    return q_out if cached else (q_out, k_out)


# bytes by (num_tokens, q_heads, kv_heads, head_dim, device index)
_workspace_sizes: dict = {}


def _workspace_size(*sizes) -> int:
    """The bytes of a call's own workspace.  A query that failed is no answer:
    it is not kept, and the call itself says what is wrong."""
    size = _workspace_sizes.get(sizes)
    if size is None:
        with torch.cuda.device(sizes[4]):
            size = lib().ple_tree_attention_workspace(*sizes[:4])
        if size < 0:
            return 0
        if len(_workspace_sizes) >= 4096:
            _workspace_sizes.clear()
        _workspace_sizes[sizes] = size
    return size


def ple_tree_attention_workspace(num_tokens: int, q_heads: int, kv_heads: int, head_dim: int,
                                 device=None) -> torch.Tensor:
    """A uint8 workspace for ple_tree_attention calls of these sizes (or fewer
    tokens) on one stream; need not be cleared."""
    with torch.cuda.device(torch.device("cuda" if device is None else device)):
        n = lib().ple_tree_attention_workspace(int(num_tokens), int(q_heads), int(kv_heads),
                                               int(head_dim))
        if n < 0:
            raise ValueError("ple_tree_attention_workspace: sizes out of range")
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def ple_tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       page_table: torch.Tensor, ctx_lens: torch.Tensor,
                       cu_seqlens: torch.Tensor, tree_mask: torch.Tensor,
                       scale: float | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, return_lse: bool = False,
                       workspace: torch.Tensor | None = None, stream=None):
    """Attention of drafted nodes over the paged cache and their own branch.

    q [T, q_heads, D]; caches [pages, kv_heads, page_size, D] with the nodes'
    keys and values already appended (ple_qk_norm_rope); tree_mask [T, words]
    int64 (ple_build_tree_index, or any mask of the same form).  A node sees
    its request's first ctx_lens[r] cached tokens and the nodes of its mask; a
    node that sees nothing gets zeros and lse -inf.  scale: 1 / sqrt(D) when
    None.  Returns out [T, q_heads, D], or (out, lse [T, q_heads] float32) with
    return_lse.  workspace: ple_tree_attention_workspace's, taken from torch's
    allocator in each call when None."""
    where = "ple_tree_attention"
    dev = q.get_device()
    dtype = q.dtype
    element = _ELEMENTS.get(dtype)
    if element is None or q.dim() != 3 or k_cache.dim() != 4:
        _device(where, q, k_cache, v_cache)
        _element(q, "q", where)
        raise ValueError(f"{where}: q must be [T, q_heads, head_dim] and the caches [pages, "
                         "kv_heads, page_size, head_dim]")
    T, Hq, D = q.shape
    cache_shape = k_cache.shape
    pages, Hk, page_size, cache_dim = cache_shape
    qs, strides = q.stride(), k_cache.stride()
    B = ctx_lens.shape[0]
    table_shape, mask_shape = page_table.shape, tree_mask.shape
    if not (out is None and lse is None and workspace is None and dev >= 0
            and k_cache.dtype is dtype and v_cache.dtype is dtype and page_table.dtype is _i32
            and ctx_lens.dtype is _i32 and cu_seqlens.dtype is _i32 and tree_mask.dtype is _i64
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and page_table.get_device() == dev and ctx_lens.get_device() == dev
            and cu_seqlens.get_device() == dev and tree_mask.get_device() == dev
            and qs[2] == 1 and v_cache.shape == cache_shape and v_cache.stride() == strides
            and strides[3] == 1 and cache_dim == D and Hk >= 1 and Hq % Hk == 0
            and ctx_lens.dim() == 1 and cu_seqlens.shape == (B + 1,)
            and len(table_shape) == 2 and table_shape[0] == B and len(mask_shape) == 2
            and mask_shape[0] == T and page_table.is_contiguous() and ctx_lens.is_contiguous()
            and cu_seqlens.is_contiguous() and tree_mask.is_contiguous()):
        dev = _device(where, q, k_cache, v_cache, page_table, ctx_lens, cu_seqlens, tree_mask, out,
                      lse, workspace)
        _heads(q, dtype, T, Hq, D, "q", where)
        _caches(k_cache, v_cache, dtype, 4, where)
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
    args = _ATTENTION.pack(
        q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), strides[0],
        strides[1], strides[2], pages, page_table.data_ptr(), ctx_lens.data_ptr(),
        cu_seqlens.data_ptr(), tree_mask.data_ptr(), out.data_ptr(),
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.shape[0], T, B,
        table_shape[1], page_size, element, Hq, Hk, D, mask_shape[1],
        D ** -0.5 if scale is None else scale)
    _call(where, lib().ple_tree_attention, dev, stream, args)
    return (out, lse) if return_lse else out


def ple_tree_commit(input_ids: torch.Tensor, path: torch.Tensor, accepted: torch.Tensor,
                    cu_seqlens: torch.Tensor, ngram_context: torch.Tensor | None,
                    ctx_lens: torch.Tensor, page_table: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, next_context: torch.Tensor | None = None,
                    next_ctx_lens: torch.Tensor | None = None, stream=None):
    """(next_context, next_ctx_lens): keep the accepted branches.

    path [B, P] int32: the kept nodes of each request, ascending (P may be 0);
    accepted [B] int32: how many of them.  Their keys and values move together behind the
    request's cached tokens, in every layer of the caches ([layers, pages,
    kv_heads, page_size, head_dim], or one layer's four dimensions), in place;
    next_ctx_lens [B] is the cached length after that, and next_context
    [B, ngram_size - 1] what the next step passes as its ngram_context (None
    when ngram_context is None).  Where given, the two must not overlap each
    other or an argument that is read, ctx_lens and ngram_context among them:
    a captured step copies them back behind the call."""
    where = "ple_tree_commit"
    dev = input_ids.get_device()
    if k_cache.dim() == 4 and v_cache.dim() == 4:
        k_cache, v_cache = k_cache.unsqueeze(0), v_cache.unsqueeze(0)
    dtype, kind = k_cache.dtype, input_ids.dtype
    element, ids = _ELEMENTS.get(dtype), _IDS.get(kind)
    strides, cache_shape = k_cache.stride(), k_cache.shape
    T, B = input_ids.shape[0], ctx_lens.shape[0]
    path_shape, table_shape = path.shape, page_table.shape
    if not (element is not None and ids is not None and next_context is None
            and next_ctx_lens is None and ngram_context is not None and dev >= 0
            and v_cache.dtype is dtype and path.dtype is _i32 and accepted.dtype is _i32
            and cu_seqlens.dtype is _i32 and ctx_lens.dtype is _i32
            and page_table.dtype is _i32 and ngram_context.dtype is kind
            and path.get_device() == dev and accepted.get_device() == dev
            and cu_seqlens.get_device() == dev and ngram_context.get_device() == dev
            and ctx_lens.get_device() == dev and page_table.get_device() == dev
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and input_ids.dim() == 1 and ctx_lens.dim() == 1 and accepted.shape == (B,)
            and cu_seqlens.shape == (B + 1,) and len(path_shape) == 2 and path_shape[0] == B
            and len(table_shape) == 2 and table_shape[0] == B and ngram_context.dim() == 2
            and ngram_context.shape[0] == B and len(cache_shape) == 5
            and v_cache.shape == cache_shape and v_cache.stride() == strides
            and strides[4] == 1 and input_ids.is_contiguous() and path.is_contiguous()
            and accepted.is_contiguous() and cu_seqlens.is_contiguous()
            and ngram_context.is_contiguous() and ctx_lens.is_contiguous()
            and page_table.is_contiguous()):
        dev = _device(where, input_ids, path, accepted, cu_seqlens, ngram_context, ctx_lens,
                      page_table, k_cache, v_cache, next_context, next_ctx_lens)
        _element(k_cache, "the caches", where)
        _caches(k_cache, v_cache, dtype, 5, where)
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
    args = _COMMIT.pack(
        input_ids.data_ptr(), path.data_ptr() if path_shape[1] else 0, accepted.data_ptr(),
        cu_seqlens.data_ptr(), 0 if C == 0 else ngram_context.data_ptr(),
        0 if C == 0 else next_context.data_ptr(), ctx_lens.data_ptr(), next_ctx_lens.data_ptr(), page_table.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), strides[0], strides[1], strides[2], strides[3], pages, T, B,
        path_shape[1], ids, C, L, table_shape[1], page_size, Hk, D, element)
    _call(where, lib().ple_tree_commit, dev, stream, args)
    return next_context, next_ctx_lens
