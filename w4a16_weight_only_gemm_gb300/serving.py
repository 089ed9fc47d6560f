"""Serving operators for torch tensors: the paged key-value cache between the
quantized linear layers, rotary positions, the attention of new tokens over the
cache, the care of its pages, the adjustment of logits and the scores of sampled
tokens.

As in ``ops``, each function checks shapes and dtypes, allocates outputs with
torch, and calls the library on the current CUDA stream (or on ``stream``).
Page, row and token numbers are device data: the kernels check their range.
"""
from __future__ import annotations

import functools
import struct

import torch

from . import _native
from .ops import _call, _device_of, _raw_stream, _stream_ptr
from .rotary import Rotary

MAX_TOP = 32
MAX_BIASES = 1024

_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_CACHE_SHAPE = struct.Struct("11q").pack
_QUERY_SHAPE = struct.Struct("5qd").pack
_BOOKS_SHAPE = struct.Struct("6q").pack
_POOL_SHAPE = struct.Struct("4q").pack
_HEADS_SHAPE = struct.Struct("8q").pack
_ADJUST_TENSORS = struct.Struct("11Q").pack
_ADJUST_SHAPE = struct.Struct("11q3d").pack

# A decode step makes these calls once a layer, and their kernels take a few
# microseconds: each check below is one pass over plain attributes, and what
# was wrong is looked for only when something was.


@functools.lru_cache(maxsize=1)
def _one_device() -> bool:
    return torch.cuda.device_count() == 1


def _run(dev: int, stream, name: str, *args) -> None:
    """Calls the library's entry point on device `dev` and the given or current stream."""
    fn = getattr(_native.lib(), name)
    if (stream is None and _raw_stream is not None
            and (_one_device() or dev == torch.cuda.current_device())):
        rc = fn(*args, _raw_stream(dev))
    else:
        device = torch.device("cuda", dev)
        rc = _call(device, fn, *args, _stream_ptr(stream, device))
    if rc:
        _native.check(rc, name)


def _empty(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A new tensor on `like`'s device whose memory belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _device(stream, **named) -> int:
    """The index of the one CUDA device of the named tensors (None passed over)."""
    _device_of(stream, *named.items())
    for name, t in named.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    raise AssertionError("unreachable")


def _ints(t: torch.Tensor, name: str, shape: tuple) -> None:
    """Refuses what is not a dense int32 tensor of `shape` (None: any size)."""
    if t.dtype is not torch.int32:
        raise ValueError(f"{name} must be an int32 tensor, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be dense in its last dimension")


def _row(t: torch.Tensor, n: int, name: str) -> None:
    """Refuses what is not a dense int32 tensor [n]."""
    if t.dtype is not torch.int32 or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        _ints(t, name, (n,))


def _heads(t: torch.Tensor, name: str, dtype, shape: tuple) -> tuple:
    """The strides of a [rows, heads, head_dim] tensor, dense in its last dimension."""
    strides = t.stride()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if strides[2] != 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return strides


def _cache_shape(k_pool: torch.Tensor, v_pool: torch.Tensor, tables: torch.Tensor) -> bytes:
    """The cache's geometry, packed for the library."""
    shape, strides, dtype = k_pool.shape, k_pool.stride(), k_pool.dtype
    if len(shape) != 4 or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must be [pages, page_size, kv_heads, head_dim], "
                         f"got {list(shape)} and {list(v_pool.shape)}")
    if v_pool.dtype is not dtype or dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("k_pool and v_pool must be both float16 or both bfloat16, got "
                         f"{dtype} and {v_pool.dtype}")
    if v_pool.stride() != strides or strides[3] != 1:
        raise ValueError("k_pool and v_pool must have the same strides, dense in their last "
                         "dimension")
    rows = tables.stride()
    if tables.dtype is not torch.int32 or len(rows) != 2 or rows[1] != 1:
        _ints(tables, "tables", (None, None))
    return _CACHE_SHAPE(*shape, _TYPES[dtype], strides[0], strides[1], strides[2], *tables.shape,
                        rows[0])


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                 tables: torch.Tensor, starts: torch.Tensor, offsets: torch.Tensor | None = None,
                 stream=None) -> None:
    """Writes new tokens' keys and values [tokens, kv_heads, head_dim] into the
    pages of k_pool / v_pool [pages, page_size, kv_heads, head_dim] (any
    strides, fp16 or bf16).

    Row b of `tables` (int32 [rows, width]) lists its pages; its tokens
    offsets[b] .. offsets[b+1] - 1 (int32 [rows + 1]; one token a row when None)
    go to positions starts[b], starts[b] + 1, ...  Tokens without a valid page
    are left out."""
    cache = _cache_shape(k_pool, v_pool, tables)
    rows, tokens, dtype = tables.shape[0], k.shape[0], k_pool.dtype
    heads = (tokens, k_pool.shape[2], k_pool.shape[3])
    ks, vs = _heads(k, "k", dtype, heads), _heads(v, "v", dtype, heads)
    _row(starts, rows, "starts")
    dev = k.get_device()
    if (dev < 0 or v.get_device() != dev or k_pool.get_device() != dev
            or v_pool.get_device() != dev or tables.get_device() != dev
            or starts.get_device() != dev or offsets is not None and offsets.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, k=k, v=v, k_pool=k_pool, v_pool=v_pool, tables=tables, starts=starts,
                offsets=offsets)
    if offsets is not None:
        _row(offsets, rows + 1, "offsets")
        offsets = offsets.data_ptr()
    if not rows:
        return
    _run(dev, stream, "w4a16_paged_append", k.data_ptr(), v.data_ptr(), k_pool.data_ptr(),
         v_pool.data_ptr(), tables.data_ptr(), starts.data_ptr(), offsets, cache, tokens, ks[0],
         ks[1], vs[0], vs[1])


@functools.lru_cache(maxsize=1024)
def _attention_workspace(cache: bytes, q_heads: int, dev: int) -> int:
    with torch.cuda.device(dev):
        n = _native.lib().w4a16_paged_attention_workspace(cache, q_heads)
    if n < 0:
        _native.check(2, "w4a16_paged_attention_workspace")
    return n


def paged_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                    tables: torch.Tensor, lengths: torch.Tensor, scale: float | None = None,
                    out: torch.Tensor | None = None, return_lse: bool = False, stream=None):
    """Attention of one new token a row, q [rows, q_heads, head_dim], over the
    first lengths[b] (int32 [rows]) positions of its pages; see paged_append for
    the cache.  q_heads is a multiple of kv_heads; scale defaults to
    head_dim ** -0.5.  Returns [rows, q_heads, head_dim] (zeros for a row of
    length 0), and with return_lse also the logarithm of each head's sum of
    exponentials, fp32 [rows, q_heads] (-inf for a row of length 0)."""
    cache = _cache_shape(k_pool, v_pool, tables)
    shape, dtype, strides = q.shape, k_pool.dtype, q.stride()
    rows, dim = tables.shape[0], k_pool.shape[3]
    if (len(shape) != 3 or shape[0] != rows or shape[2] != dim or strides[2] != 1
            or q.dtype is not dtype):
        _heads(q, "q", dtype, (rows, shape[1] if len(shape) == 3 else "q_heads", dim))
    q_heads = shape[1]
    if lengths.dtype is not torch.int32 or lengths.shape != (rows,) or lengths.stride(0) != 1:
        _row(lengths, rows, "lengths")
    dev = q.get_device()
    if (dev < 0 or k_pool.get_device() != dev or v_pool.get_device() != dev
            or tables.get_device() != dev or lengths.get_device() != dev
            or out is not None and out.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, q=q, k_pool=k_pool, v_pool=v_pool, tables=tables, lengths=lengths, out=out)
    if out is None:
        out = _empty(q, shape, dtype, stream)
        row, head = q_heads * dim, dim
    else:
        row, head, _ = _heads(out, "out", dtype, shape)
    lse = _empty(q, (rows, q_heads), torch.float32, stream) if return_lse else None
    if rows:
        size = _attention_workspace(cache, q_heads, dev)
        workspace = _empty(q, size, torch.uint8, stream) if size else out  # 0: not looked at
        _run(dev, stream, "w4a16_paged_attention", q.data_ptr(), k_pool.data_ptr(),
             v_pool.data_ptr(), tables.data_ptr(), lengths.data_ptr(), out.data_ptr(),
             lse.data_ptr() if return_lse else None, workspace.data_ptr(), cache,
             _QUERY_SHAPE(q_heads, strides[0], strides[1], row, head,
                          dim ** -0.5 if scale is None else scale))
    return (out, lse) if return_lse else out


def rotate(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Heads x [tokens, heads, head_dim] (fp16, bf16 or fp32, any strides) rotated to
    their tokens' positions (int32 [tokens], of either sign); `out` may be x, and else
    overlaps none of it.  A rotation to -positions is the gradient; it undoes the rotation
    but for the square of its magnitude."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 3 or dtype not in _TYPES or not 1 <= rotary.dim <= shape[2]:
        raise ValueError("x must be a float16, bfloat16 or float32 tensor [tokens, heads, "
                         f"head_dim >= {rotary.dim}], got {dtype} {list(shape)}")
    row, head, _ = _heads(x, "x", dtype, shape)
    tokens, heads, dim = shape
    _row(positions, tokens, "positions")
    dev = x.get_device()
    on, turns = rotary._held()
    if (dev < 0 or positions.get_device() != dev or on != dev
            or out is not None and out.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, x=x, positions=positions, rotary=rotary.turns, out=out)
    if out is None:
        out = _empty(x, shape, dtype, stream)
        to_row, to_head = heads * dim, dim
    else:
        to_row, to_head, _ = _heads(out, "out", dtype, shape)
    if tokens and heads:
        _run(dev, stream, "w4a16_rotate", x.data_ptr(), positions.data_ptr(),
             turns, out.data_ptr(), rotary._shape,
             _HEADS_SHAPE(tokens, heads, dim, _TYPES[dtype], row, head, to_row, to_head))
    return out


def paged_append_rotary(k: torch.Tensor, v: torch.Tensor, k_pool: torch.Tensor,
                        v_pool: torch.Tensor, tables: torch.Tensor, starts: torch.Tensor,
                        rotary: Rotary, offsets: torch.Tensor | None = None,
                        q: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        stream=None):
    """paged_append with the keys rotated to their positions in the cache, and with
    queries of the same tokens, q [tokens, q_heads, head_dim], rotated to theirs: returns
    those (a new tensor, or `out`, which may be q and else overlaps no input), or None
    without q.  The queries of a token that no row claims become zeros."""
    cache = _cache_shape(k_pool, v_pool, tables)
    rows, tokens, dtype = tables.shape[0], k.shape[0], k_pool.dtype
    _, _, kv_heads, dim = k_pool.shape
    if rotary.dim > dim:
        raise ValueError(f"the rotation has {rotary.dim} dimensions, a head {dim}")
    heads = (tokens, kv_heads, dim)
    ks, vs = _heads(k, "k", dtype, heads), _heads(v, "v", dtype, heads)
    _row(starts, rows, "starts")
    dev = k.get_device()
    on, turns = rotary._held()
    same = (dev >= 0 and v.get_device() == dev and k_pool.get_device() == dev
            and v_pool.get_device() == dev and tables.get_device() == dev
            and starts.get_device() == dev and on == dev
            and (stream is None or stream.device.index == dev))
    at = None
    if offsets is not None:
        _row(offsets, rows + 1, "offsets")
        same, at = same and offsets.get_device() == dev, offsets.data_ptr()
    elif tokens != rows:
        raise ValueError(f"without offsets there must be one token a row, got {tokens} for {rows}")
    if q is None:
        if out is not None:
            raise ValueError("out without q")
    else:
        q_heads = q.shape[1] if q.dim() == 3 else "q_heads"
        qs = _heads(q, "q", dtype, (tokens, q_heads, dim))
        same = same and q.get_device() == dev and (out is None or out.get_device() == dev)
    if not same:
        _device(stream, k=k, v=v, k_pool=k_pool, v_pool=v_pool, tables=tables, starts=starts,
                rotary=rotary.turns, offsets=offsets, q=q, out=out)
    q_at = out_at = None
    if q is None:
        queries = _HEADS_SHAPE(tokens, 0, dim, 0, 0, 0, 0, 0)
    else:
        if out is None:
            out = _empty(q, (tokens, q_heads, dim), dtype, stream)
            row, head = q_heads * dim, dim
        else:
            row, head, _ = _heads(out, "out", dtype, (tokens, q_heads, dim))
        queries = _HEADS_SHAPE(tokens, q_heads, dim, _TYPES[dtype], qs[0], qs[1], row, head)
        if q_heads:
            q_at, out_at = q.data_ptr(), out.data_ptr()
    if rows and tokens:
        _run(dev, stream, "w4a16_paged_append_rotary", k.data_ptr(), v.data_ptr(), turns,
             k_pool.data_ptr(), v_pool.data_ptr(), tables.data_ptr(), starts.data_ptr(), at, q_at,
             out_at, cache, rotary._shape, queries, ks[0], ks[1], vs[0], vs[1])
    elif q is not None and tokens:
        _fill(out, stream, 0.0)
    return out


@functools.lru_cache(maxsize=1024)
def _chunk_workspace(cache: bytes, q_heads: int, tokens: int, dev: int) -> int:
    with torch.cuda.device(dev):
        n = _native.lib().w4a16_paged_chunk_workspace(cache, q_heads, tokens)
    if n < 0:
        _native.check(2, "w4a16_paged_chunk_workspace")
    return n


def paged_chunk_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                          tables: torch.Tensor, lengths: torch.Tensor, offsets: torch.Tensor,
                          scale: float | None = None, out: torch.Tensor | None = None,
                          return_lse: bool = False, stream=None):
    """Attention of each row's last tokens over its pages, whose keys and values the cache
    holds already; see paged_append for the cache.  Row b's tokens offsets[b] ..
    offsets[b+1] - 1 (int32 [rows + 1]) of q [tokens, q_heads, head_dim] are the last of
    its lengths[b] positions (int32 [rows]), and each sees the positions up to its own.
    q_heads is a multiple of kv_heads; scale defaults to head_dim ** -0.5.  Returns
    [tokens, q_heads, head_dim] (or `out`, which overlaps no input), zeros for tokens of no
    row or of a position below 0, and with return_lse also the logarithm of each head's sum
    of exponentials, fp32 [tokens, q_heads] (-inf for such tokens).  Weights enter the
    product with the values in the cache's type (paged_attention, for one new token a row,
    keeps twice their bits)."""
    cache = _cache_shape(k_pool, v_pool, tables)
    shape, dtype = q.shape, k_pool.dtype
    rows, dim = tables.shape[0], k_pool.shape[3]
    tokens, q_heads = (shape[0], shape[1]) if len(shape) == 3 else ("tokens", "q_heads")
    row, head, _ = _heads(q, "q", dtype, (tokens, q_heads, dim))
    _row(lengths, rows, "lengths")
    _row(offsets, rows + 1, "offsets")
    dev = q.get_device()
    if (dev < 0 or k_pool.get_device() != dev or v_pool.get_device() != dev
            or tables.get_device() != dev or lengths.get_device() != dev
            or offsets.get_device() != dev or out is not None and out.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, q=q, k_pool=k_pool, v_pool=v_pool, tables=tables, lengths=lengths,
                offsets=offsets, out=out)
    if out is None:
        out = _empty(q, shape, dtype, stream)
        to_row, to_head = q_heads * dim, dim
    else:
        to_row, to_head, _ = _heads(out, "out", dtype, shape)
    lse = _empty(q, (tokens, q_heads), torch.float32, stream) if return_lse else None
    if rows and tokens:
        size = _chunk_workspace(cache, q_heads, tokens, dev)
        workspace = _empty(q, size, torch.uint8, stream) if size else out  # 0: not looked at
        _run(dev, stream, "w4a16_paged_chunk_attention", q.data_ptr(), k_pool.data_ptr(),
             v_pool.data_ptr(), tables.data_ptr(), lengths.data_ptr(), offsets.data_ptr(),
             out.data_ptr(), lse.data_ptr() if return_lse else None, workspace.data_ptr(), cache,
             _QUERY_SHAPE(q_heads, row, head, to_row, to_head,
                          dim ** -0.5 if scale is None else scale), tokens)
    elif tokens:
        _fill(out, stream, 0.0)
        if return_lse:
            _fill(lse, stream, -float("inf"))
    return (out, lse) if return_lse else out


def _fill(t: torch.Tensor, stream, value: float) -> None:
    """Fills what no row of an empty batch claims."""
    with torch.cuda.stream(stream):
        t.fill_(value)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """torch.empty_like on a stream (dense in its last dimension as t is)."""
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _books(refs, tables, lengths, out, page_size: int, stream, names: tuple, *others):
    """The books' device, their addresses, their outputs (new ones, or `out`), the outputs'
    addresses and the packed shape; `others` (of those names) share the device.  lengths may be
    None: neither read nor written."""
    pages, (rows, width), strides, dev = refs.shape[0], tables.shape, tables.stride(), refs.get_device()
    if refs.dtype is not torch.int32 or refs.stride() != (1,):
        _row(refs, pages, "refs")
    if tables.dtype is not torch.int32 or strides[1] != 1:
        _ints(tables, "tables", (None, None))
    same = dev >= 0 and tables.get_device() == dev and (stream is None or stream.device.index == dev)
    ins = (refs, tables)
    if lengths is not None:
        _row(lengths, rows, "lengths")
        same = same and lengths.get_device() == dev
        ins = (refs, tables, lengths)
    for t in others:
        same = same and t.get_device() == dev
    if out is None:
        outs = ins
        if same:
            outs = tuple(map(torch.empty_like, ins)) if stream is None \
                else tuple(_like(t, stream) for t in ins)
    else:
        outs = tuple(out)
        if len(outs) != len(ins):
            raise ValueError(f"out must be {len(ins)} tensors")
        for t, o in zip(ins, outs):
            _ints(o, "out", tuple(t.shape))
            if o.data_ptr() == t.data_ptr() and o.stride() != t.stride():
                raise ValueError("an out tensor that is its input must have its strides")
            same = same and o.get_device() == dev
    row = outs[1].stride(0) if rows > 1 else width
    if not same:
        _device(stream, refs=refs, tables=tables, lengths=lengths, **dict(zip(names, others)),
                **{f"out[{i}]": o for i, o in enumerate(outs)})
    return (dev, [t.data_ptr() for t in ins], outs, [t.data_ptr() for t in outs],
            _BOOKS_SHAPE(pages, rows, width, strides[0], row, page_size))


def _pool_shape(pool: torch.Tensor, pages: int | None) -> bytes:
    """`pool` [planes, pages, ...] with dense pages, packed for the library."""
    shape, strides, size = pool.shape, pool.stride(), pool.element_size()
    if len(shape) < 3:
        raise ValueError(f"pool must be [planes, pages, ...], got {list(shape)}")
    if pages is not None and shape[1] != pages:
        raise ValueError(f"pool has {shape[1]} pages, the books {pages}")
    page = size
    if shape[1] > 1 and pool.is_contiguous():
        page *= strides[1]
    else:
        for i in range(len(shape) - 1, 1, -1):
            if strides[i] * size != page and shape[i] > 1:
                raise ValueError("pool must be dense within a page")
            page *= shape[i]
    return _POOL_SHAPE(shape[0], strides[0] * size, strides[1] * size, page)


@functools.lru_cache(maxsize=1024)
def _pages_workspace(name: str, *shape) -> int:
    n = getattr(_native.lib(), name)(*shape)
    if n < 0:
        _native.check(2, name)
    return n


def pages_free(refs: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
               rows: torch.Tensor, out=None, stream=None):
    """Gives back the pages of the listed rows (int32): one holder fewer in
    refs [pages], page numbers -1 in tables [rows, width], length 0.  Returns
    (refs, tables, lengths), new tensors or `out` (which may be the inputs)."""
    count = rows.shape[0]
    _row(rows, count, "rows")
    dev, ins, outs, to, shape = _books(refs, tables, lengths, out, 1, stream, ("rows",), rows)
    _run(dev, stream, "w4a16_pages_free", *ins, rows.data_ptr(), count, *to, shape)
    return outs


def pages_extend(refs: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
                 rows: torch.Tensor, counts: torch.Tensor, page_size: int, out=None, stream=None):
    """Makes rows[i] longer by counts[i] positions and gives it the lowest free
    pages it then needs, in the order of the list.  Returns (refs, tables,
    lengths, done); done[i] = 0 where the row is left as it was: too few free
    pages, a row too long, out of range or listed before."""
    count = rows.shape[0]
    _row(rows, count, "rows")
    _row(counts, count, "counts")
    dev, ins, outs, to, shape = _books(refs, tables, lengths, out, page_size, stream,
                                       ("rows", "counts"), rows, counts)
    done = _empty(refs, count, torch.int32, stream)
    space = _empty(refs, _pages_workspace("w4a16_pages_workspace", shape, count), torch.uint8,
                   stream)
    _run(dev, stream, "w4a16_pages_extend", *ins, rows.data_ptr(), counts.data_ptr(), count, *to,
         done.data_ptr(), space.data_ptr(), shape)
    return *outs, done


def pages_fork(pool: torch.Tensor, refs: torch.Tensor, tables: torch.Tensor,
               lengths: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
               page_size: int, out=None, stream=None):
    """Makes the empty row children[i] a copy of row parents[i]: full pages are
    shared, a partly filled last page is copied in every plane of pool
    [planes, pages, ...] to the lowest free page.  Returns (refs, tables,
    lengths, done); done[i] = 0 where the child is left as it was: too few free
    pages, a child not empty, a row out of range or a child listed before."""
    planes, count = _pool_shape(pool, refs.shape[0]), parents.shape[0]
    _row(parents, count, "parents")
    _row(children, count, "children")
    dev, ins, outs, to, shape = _books(refs, tables, lengths, out, page_size, stream,
                                       ("pool", "parents", "children"), pool, parents, children)
    done = _empty(refs, count, torch.int32, stream)
    apart = out is None or not any(i == o for i, o in zip(ins, to))
    size = _pages_workspace("w4a16_pages_fork_workspace", shape, planes, count, apart)
    space = _empty(refs, size, torch.uint8, stream) if size else pool  # 0: not looked at
    _run(dev, stream, "w4a16_pages_fork", pool.data_ptr(), *ins, parents.data_ptr(),
         children.data_ptr(), count, *to, done.data_ptr(), space.data_ptr(), shape, planes)
    return *outs, done


def pages_compact(pool: torch.Tensor, refs: torch.Tensor, tables: torch.Tensor, out=None,
                  stream=None):
    """Moves the n held pages to the numbers below n: those at n and above go,
    in ascending order, to the free ones below, in every plane of pool
    [planes, pages, ...].  Returns (refs, tables, used) with used = [n]."""
    planes = _pool_shape(pool, refs.shape[0])
    dev, ins, outs, to, shape = _books(refs, tables, None, out, 1, stream, ("pool",), pool)
    used = _empty(refs, 1, torch.int32, stream)
    apart = out is None or not any(i == o for i, o in zip(ins, to))
    size = _pages_workspace("w4a16_pages_compact_workspace", shape, planes, apart)
    space = _empty(refs, size, torch.uint8, stream) if size else pool  # 0: not looked at
    _run(dev, stream, "w4a16_pages_compact", pool.data_ptr(), *ins, *to, used.data_ptr(),
         space.data_ptr(), shape, planes)
    return *outs, used


def pages_copy(pool: torch.Tensor, sources: torch.Tensor, targets: torch.Tensor,
               stream=None) -> None:
    """Copies page sources[i] to page targets[i] (int32) in every plane of pool
    [planes, pages, ...]; pairs out of range are passed over."""
    planes, count, dev = _pool_shape(pool, None), sources.shape[0], pool.get_device()
    _row(sources, count, "sources")
    _row(targets, count, "targets")
    if (dev < 0 or sources.get_device() != dev or targets.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, pool=pool, sources=sources, targets=targets)
    _run(dev, stream, "w4a16_pages_copy", pool.data_ptr(), sources.data_ptr(), targets.data_ptr(),
         count, pool.shape[1], planes)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, stream=None):
    """Scores of the given tokens (int64 or int32 [rows]) under logits [rows,
    vocabulary] (fp16, bf16 or fp32, dense in the last dimension): returns
    (logprobs, entropies, top_ids, top_logprobs), fp32 [rows] twice, int32 and
    fp32 [rows, top]; the `top` (at most 32) largest logits come first, of equal
    ones the lowest index.  -inf masks a logit; a token outside the vocabulary
    has the log probability NaN."""
    strides, kind = logits.stride(), _TYPES.get(logits.dtype)
    if kind is None or len(strides) != 2:
        raise ValueError("logits must be a float16, bfloat16 or float32 tensor "
                         f"[rows, vocabulary], got {logits.dtype} {list(logits.shape)}")
    rows, vocabulary = logits.shape
    if strides[1] != 1 and vocabulary > 1:
        raise ValueError("logits must be dense in their last dimension")
    wide = tokens.dtype is torch.int64
    if (not wide and tokens.dtype is not torch.int32 or tokens.shape != (rows,)
            or not tokens.is_contiguous()):
        raise ValueError(f"tokens must be a dense int64 or int32 tensor [{rows}]")
    if not 0 <= top <= MAX_TOP or top > vocabulary:
        raise ValueError(f"top must be 0 .. {min(MAX_TOP, vocabulary)}, got {top}")
    dev = logits.get_device()
    if (dev < 0 or tokens.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, logits=logits, tokens=tokens)
    logprobs = _empty(logits, rows, torch.float32, stream)
    entropies = _empty(logits, rows, torch.float32, stream)
    ids = _empty(logits, (rows, top), torch.int32, stream)
    likeliest = _empty(logits, (rows, top), torch.float32, stream)
    if rows:
        _run(dev, stream, "w4a16_token_logprobs", logits.data_ptr(), tokens.data_ptr(),
             logprobs.data_ptr(), entropies.data_ptr(), ids.data_ptr(), likeliest.data_ptr(), rows,
             vocabulary, strides[0], kind, wide, top)
    return logprobs, entropies, ids, likeliest


def _penalty(value: torch.Tensor, rows: int, name: str) -> int:
    """The address of a penalty that is one of every row."""
    if value.dtype is not torch.float32 or value.shape != (rows,) or not value.is_contiguous():
        raise ValueError(f"{name} must be a number or a dense float32 tensor [{rows}], got "
                         f"{value.dtype} {list(value.shape)}")
    return value.data_ptr()


def _rows_of(t: torch.Tensor, rows: int, name: str, *dtypes) -> tuple:
    """The width and row stride of what is [rows, any], dense in its last dimension, of one of the
    types."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a {' or '.join(map(str, dtypes))} tensor [{rows}, any], "
                         f"got {t.dtype} {list(shape)}")
    strides = t.stride()
    if strides[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return shape[1], strides[0]


def adjust_logits(logits: torch.Tensor, tokens: torch.Tensor | None = None,
                  lengths: torch.Tensor | None = None, prompts: torch.Tensor | None = None,
                  repetition=1.0, presence=0.0, frequency=0.0,
                  bias_ids: torch.Tensor | None = None, biases: torch.Tensor | None = None,
                  mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Penalties, biases and masks on logits [rows, vocabulary] (fp16, bf16 or fp32, dense in
    the last dimension), in this order; returns a new tensor, or `out`, which may be logits and
    else overlaps none of them.

    tokens (int32 or int64 [rows, width]) lists what each row has said: its first lengths[r]
    (int32 [rows]; all when None), of which the first prompts[r] (int32 [rows]; none when None)
    are the prompt's.  A logit x of a token said at all becomes x / repetition where x > 0 and
    x * repetition elsewhere; frequency times its count in the generation is taken off, and
    presence once if it is there.  The three are numbers or fp32 tensors [rows].  Then
    biases[r, i] (fp32 [rows, n], n at most 1024) is added to the logit bias_ids[r, i] (int32),
    and where bit j % 32 of mask[r, j / 32] (int32 [rows, ceil(vocabulary / 32)]) is 0 logit j
    becomes -inf.  Tokens outside the vocabulary are passed over."""
    dtype, shape, strides = logits.dtype, logits.shape, logits.stride()
    kind = _TYPES.get(dtype)
    if kind is None or len(shape) != 2:
        raise ValueError("logits must be a float16, bfloat16 or float32 tensor "
                         f"[rows, vocabulary], got {dtype} {list(shape)}")
    rows, vocabulary = shape
    if strides[1] != 1 and vocabulary > 1:
        raise ValueError("logits must be dense in their last dimension")
    dev = logits.get_device()
    same = dev >= 0 and (stream is None or stream.device.index == dev)
    width = token_stride = wide = said = known = prompted = 0
    if tokens is not None:
        width, token_stride = _rows_of(tokens, rows, "tokens", torch.int32, torch.int64)
        wide, said = tokens.dtype is torch.int64, tokens.data_ptr()
        same = same and tokens.get_device() == dev
        if lengths is not None:
            _row(lengths, rows, "lengths")
            known, same = lengths.data_ptr(), same and lengths.get_device() == dev
        if prompts is not None:
            _row(prompts, rows, "prompts")
            prompted, same = prompts.data_ptr(), same and prompts.get_device() == dev
    elif lengths is not None or prompts is not None:
        raise ValueError("lengths or prompts without tokens")
    penalties = {"repetition": repetition, "presence": presence, "frequency": frequency}
    each = [0, 0, 0]                            # addresses of those that rows have of their own
    if isinstance(repetition, torch.Tensor):
        same = same and repetition.get_device() == dev
        each[0], repetition = _penalty(repetition, rows, "repetition"), 1.0
    elif not repetition > 0:
        raise ValueError(f"repetition must be above 0, got {repetition}")
    if isinstance(presence, torch.Tensor):
        same = same and presence.get_device() == dev
        each[1], presence = _penalty(presence, rows, "presence"), 0.0
    if isinstance(frequency, torch.Tensor):
        same = same and frequency.get_device() == dev
        each[2], frequency = _penalty(frequency, rows, "frequency"), 0.0
    count = bias_stride = ids = values = 0
    if bias_ids is not None and biases is not None:
        count, bias_stride = _rows_of(biases, rows, "biases", torch.float32)
        if _rows_of(bias_ids, rows, "bias_ids", torch.int32) != (count, bias_stride) and (
                bias_ids.shape[1] != count or rows > 1):
            raise ValueError("bias_ids and biases must have the same shape and strides")
        if count > MAX_BIASES:
            raise ValueError(f"at most {MAX_BIASES} biases a row, got {count}")
        same = same and bias_ids.get_device() == dev and biases.get_device() == dev
        if count:
            ids, values = bias_ids.data_ptr(), biases.data_ptr()
    elif bias_ids is not None or biases is not None:
        raise ValueError("bias_ids and biases go together")
    mask_stride = bits = 0
    if mask is not None:
        words, mask_stride = _rows_of(mask, rows, "mask", torch.int32)
        if words != -(-vocabulary // 32):
            raise ValueError(f"mask must have {-(-vocabulary // 32)} words a row, got {words}")
        bits, same = mask.data_ptr(), same and mask.get_device() == dev
    if out is not None:
        if out.dtype is not dtype or out.shape != shape or vocabulary > 1 and out.stride(1) != 1:
            raise ValueError(f"out must be {dtype} {list(shape)}, dense in its last dimension, got "
                             f"{out.dtype} {list(out.shape)}")
        same = same and out.get_device() == dev
    if not same:
        given = {"tokens": tokens, "lengths": lengths, "prompts": prompts, "bias_ids": bias_ids,
                 "biases": biases, "mask": mask, "out": out,
                 **{n: t for n, t in penalties.items() if isinstance(t, torch.Tensor)}}
        _device(stream, logits=logits, **given)
    if out is None:
        out = _empty(logits, shape, dtype, stream)
        out_stride = vocabulary
    else:
        out_stride = out.stride(0)
    if rows and vocabulary:
        _run(dev, stream, "w4a16_adjust_logits",
             _ADJUST_TENSORS(logits.data_ptr(), said, known, prompted, *each, ids, values, bits,
                             out.data_ptr()),
             _ADJUST_SHAPE(rows, vocabulary, kind, strides[0], out_stride, wide, width,
                           token_stride, count, bias_stride, mask_stride, repetition, presence,
                           frequency))
    return out


def _listed(tables: torch.Tensor, lengths: torch.Tensor | None, rows: torch.Tensor, stream):
    """The listed rows' tables and lengths (None for None), taken on the stream the call runs on;
    a row out of range has no pages and length 0."""
    (n, width), count, dev = tables.shape, rows.shape[0], tables.get_device()
    if rows.dtype is torch.int64:
        with torch.cuda.stream(stream):
            rows = rows.clamp(-1, n).int()
    _row(rows, count, "rows")
    _ints(tables, "tables", (n, width))
    if lengths is not None:
        _row(lengths, n, "lengths")
    if (dev < 0 or rows.get_device() != dev or lengths is not None and lengths.get_device() != dev
            or stream is not None and stream.device.index != dev):
        _device(stream, tables=tables, lengths=lengths, rows=rows)
    new_tables = _empty(tables, (count, width), torch.int32, stream)
    new_lengths = None if lengths is None else _empty(tables, count, torch.int32, stream)
    _run(dev, stream, "w4a16_pages_rows", tables.data_ptr(),
         None if lengths is None else lengths.data_ptr(), rows.data_ptr(), count,
         new_tables.data_ptr(), None if lengths is None else new_lengths.data_ptr(),
         _BOOKS_SHAPE(1, n, width, tables.stride(0), width, 1))
    return new_tables, new_lengths


class PagedCache:
    """The keys and values of a decoder's layers for `rows` sequences, in pages
    that sequences take, share and give back.

    pool [2 * layers, pages, page_size, kv_heads, head_dim] holds layer l's keys
    in plane 2l and its values in plane 2l + 1; one page number means the same
    page of every plane.  refs, tables and lengths are the books the pages_*
    functions keep, updated in place, so the methods may be captured in a CUDA
    graph.  A listed row that is out of range is passed over by every method: its
    tokens go nowhere, its attention is that of a row of length 0."""

    def __init__(self, layers: int, rows: int, pages: int, kv_heads: int, head_dim: int,
                 page_size: int = 16, max_length: int | None = None,
                 dtype: torch.dtype = torch.float16, device="cuda"):
        width = pages if max_length is None else -(-max_length // page_size)
        self.page_size = page_size
        self.pool = torch.empty((2 * layers, pages, page_size, kv_heads, head_dim), dtype=dtype,
                                device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.tables = torch.full((rows, width), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(rows, dtype=torch.int32, device=device)

    def _all(self):
        return self.refs, self.tables, self.lengths

    def keys(self, layer: int) -> torch.Tensor:
        """A layer's key pool [pages, page_size, kv_heads, head_dim]."""
        return self.pool[2 * layer]

    def values(self, layer: int) -> torch.Tensor:
        """A layer's value pool [pages, page_size, kv_heads, head_dim]."""
        return self.pool[2 * layer + 1]

    def extend(self, rows: torch.Tensor, counts: torch.Tensor, stream=None) -> torch.Tensor:
        """Room for counts[i] more positions in rows[i]; returns done (pages_extend)."""
        return pages_extend(*self._all(), rows, counts, self.page_size, out=self._all(),
                            stream=stream)[3]

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
               offsets: torch.Tensor | None = None, rows: torch.Tensor | None = None,
               stream=None) -> None:
        """New tokens of every row (or of the listed ones) of one layer (paged_append)."""
        tables = self.tables if rows is None else _listed(self.tables, None, rows, stream)[0]
        paged_append(k, v, self.keys(layer), self.values(layer), tables, starts, offsets,
                     stream=stream)

    def append_rotary(self, layer: int, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                      rotary: Rotary, offsets: torch.Tensor | None = None,
                      q: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None):
        """New tokens of every row (or of the listed ones) of one layer, keys rotated to their
        positions; returns the rotated queries (paged_append_rotary)."""
        tables = self.tables if rows is None else _listed(self.tables, None, rows, stream)[0]
        return paged_append_rotary(k, v, self.keys(layer), self.values(layer), tables, starts,
                                   rotary, offsets, q=q, out=out, stream=stream)

    def attend(self, layer: int, q: torch.Tensor, rows: torch.Tensor | None = None,
               scale: float | None = None, out: torch.Tensor | None = None, stream=None):
        """Attention of one new token of every row (or of the listed ones) (paged_attention)."""
        tables, lengths = self.tables, self.lengths
        if rows is not None:
            tables, lengths = _listed(tables, lengths, rows, stream)
        return paged_attention(q, self.keys(layer), self.values(layer), tables, lengths,
                               scale=scale, out=out, stream=stream)

    def attend_chunks(self, layer: int, q: torch.Tensor, offsets: torch.Tensor,
                      rows: torch.Tensor | None = None, scale: float | None = None,
                      out: torch.Tensor | None = None, stream=None):
        """Attention of the last tokens of every row (or of the listed ones)
        (paged_chunk_attention)."""
        tables, lengths = self.tables, self.lengths
        if rows is not None:
            tables, lengths = _listed(tables, lengths, rows, stream)
        return paged_chunk_attention(q, self.keys(layer), self.values(layer), tables, lengths,
                                     offsets, scale=scale, out=out, stream=stream)

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream=None) -> torch.Tensor:
        """Row children[i] becomes a copy of row parents[i]; returns done (pages_fork)."""
        return pages_fork(self.pool, *self._all(), parents, children, self.page_size,
                          out=self._all(), stream=stream)[3]

    def free(self, rows: torch.Tensor, stream=None) -> None:
        """Gives the listed rows' pages back (pages_free)."""
        pages_free(*self._all(), rows, out=self._all(), stream=stream)

    def compact(self, stream=None) -> torch.Tensor:
        """Draws the held pages together; returns their number, int32 [1] (pages_compact)."""
        return pages_compact(self.pool, self.refs, self.tables, out=(self.refs, self.tables),
                             stream=stream)[2]
