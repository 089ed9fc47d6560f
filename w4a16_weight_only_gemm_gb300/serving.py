"""Serving operators for torch tensors: the paged key-value cache between the
quantized linear layers, the attention of a new token over it, the care of its
pages, and the scores of sampled tokens.

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

MAX_TOP = 32

_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_CACHE_SHAPE = struct.Struct("11q").pack
_QUERY_SHAPE = struct.Struct("5qd").pack
_BOOKS_SHAPE = struct.Struct("6q").pack
_POOL_SHAPE = struct.Struct("4q").pack

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

    def attend(self, layer: int, q: torch.Tensor, rows: torch.Tensor | None = None,
               scale: float | None = None, out: torch.Tensor | None = None, stream=None):
        """Attention of one new token of every row (or of the listed ones) (paged_attention)."""
        tables, lengths = self.tables, self.lengths
        if rows is not None:
            tables, lengths = _listed(tables, lengths, rows, stream)
        return paged_attention(q, self.keys(layer), self.values(layer), tables, lengths,
                               scale=scale, out=out, stream=stream)

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
