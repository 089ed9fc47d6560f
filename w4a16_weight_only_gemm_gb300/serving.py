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
from .ops import _call, _device_of, _stream_ptr

MAX_TOP = 32

_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_CACHE_SHAPE = struct.Struct("11q")
_QUERY_SHAPE = struct.Struct("5qd")
_BOOKS_SHAPE = struct.Struct("6q")
_POOL_SHAPE = struct.Struct("4q")


def _empty(shape, dtype, dev, stream) -> torch.Tensor:
    """A new tensor whose memory belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _ints(t: torch.Tensor, name: str, shape: tuple) -> None:
    """A dense int32 CUDA tensor of `shape` (None: any size)."""
    if t.dtype != torch.int32 or not t.is_cuda:
        raise ValueError(f"{name} must be an int32 CUDA tensor, got {t.dtype} on {t.device}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be dense in its last dimension")


def _stride(t: torch.Tensor, dim: int) -> int:
    return t.stride(dim) if t.shape[dim] > 1 else 0


def _heads(t: torch.Tensor, name: str, dtype, shape: tuple) -> None:
    """A CUDA tensor [rows, heads, head_dim], dense in its last dimension."""
    if t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be dense in its last dimension")


def _cache_shape(k_pool: torch.Tensor, v_pool: torch.Tensor, tables: torch.Tensor) -> bytes:
    """The cache's geometry, packed for the library."""
    shape, strides = k_pool.shape, k_pool.stride()
    if len(shape) != 4 or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must be [pages, page_size, kv_heads, head_dim], "
                         f"got {list(shape)} and {list(v_pool.shape)}")
    if k_pool.dtype not in (torch.float16, torch.bfloat16) or v_pool.dtype != k_pool.dtype:
        raise ValueError("k_pool and v_pool must be both float16 or both bfloat16, got "
                         f"{k_pool.dtype} and {v_pool.dtype}")
    if not k_pool.is_cuda or v_pool.stride() != strides or strides[3] != 1:
        raise ValueError("k_pool and v_pool must be CUDA tensors of the same strides, dense in "
                         "their last dimension")
    _ints(tables, "tables", (None, None))
    return _CACHE_SHAPE.pack(*shape, _TYPES[k_pool.dtype], _stride(k_pool, 0), _stride(k_pool, 1),
                             _stride(k_pool, 2), *tables.shape, _stride(tables, 0))


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
    rows, tokens = tables.shape[0], k.shape[0]
    heads = (tokens, k_pool.shape[2], k_pool.shape[3])
    _heads(k, "k", k_pool.dtype, heads)
    _heads(v, "v", k_pool.dtype, heads)
    _ints(starts, "starts", (rows,))
    if offsets is not None:
        _ints(offsets, "offsets", (rows + 1,))
    dev = _device_of(stream, ("k", k), ("v", v), ("k_pool", k_pool), ("v_pool", v_pool),
                     ("tables", tables), ("starts", starts), ("offsets", offsets))
    if not rows:
        return
    rc = _call(dev, _native.lib().w4a16_paged_append, k.data_ptr(), v.data_ptr(),
               k_pool.data_ptr(), v_pool.data_ptr(), tables.data_ptr(), starts.data_ptr(),
               offsets.data_ptr() if offsets is not None else None, cache, tokens, _stride(k, 0),
               _stride(k, 1), _stride(v, 0), _stride(v, 1), _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_paged_append")


@functools.lru_cache(maxsize=1024)
def _attention_workspace(cache: bytes, q_heads: int, device: int | None) -> int:
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
    if q.dim() != 3:
        raise ValueError(f"q must be [rows, q_heads, head_dim], got {list(q.shape)}")
    rows, q_heads, dim = tables.shape[0], q.shape[1], k_pool.shape[3]
    _heads(q, "q", k_pool.dtype, (rows, q_heads, dim))
    _ints(lengths, "lengths", (rows,))
    dev = _device_of(stream, ("q", q), ("k_pool", k_pool), ("v_pool", v_pool), ("tables", tables),
                     ("lengths", lengths), ("out", out))
    if out is None:
        out = _empty((rows, q_heads, dim), q.dtype, dev, stream)
    else:
        _heads(out, "out", q.dtype, (rows, q_heads, dim))
    lse = _empty((rows, q_heads), torch.float32, dev, stream) if return_lse else None
    if not rows:
        return (out, lse) if return_lse else out
    size = _call(dev, _attention_workspace, cache, q_heads, dev.index)
    workspace = _empty(size, torch.uint8, dev, stream)
    query = _QUERY_SHAPE.pack(q_heads, _stride(q, 0), _stride(q, 1), _stride(out, 0),
                              _stride(out, 1), dim ** -0.5 if scale is None else scale)
    rc = _call(dev, _native.lib().w4a16_paged_attention, q.data_ptr(), k_pool.data_ptr(),
               v_pool.data_ptr(), tables.data_ptr(), lengths.data_ptr(), out.data_ptr(),
               lse.data_ptr() if return_lse else None, workspace.data_ptr(), cache, query,
               _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_paged_attention")
    return (out, lse) if return_lse else out


def _books(refs, tables, lengths, out, page_size: int, stream):
    """The checked books, their outputs (new ones, or `out`) and the packed shape."""
    _ints(refs, "refs", (None,))
    _ints(tables, "tables", (None, None))
    if lengths is not None:
        _ints(lengths, "lengths", (tables.shape[0],))
    ins = (refs, tables) if lengths is None else (refs, tables, lengths)
    if out is None:
        outs = tuple(_empty(t.shape, torch.int32, refs.device, stream) for t in ins)
    else:
        outs = tuple(out)
        if len(outs) != len(ins):
            raise ValueError(f"out must be {len(ins)} tensors")
        for t, o in zip(ins, outs):
            _ints(o, "out", tuple(t.shape))
            if o.data_ptr() == t.data_ptr() and o.stride() != t.stride():
                raise ValueError("an out tensor that is its input must have its strides")
    rows, width = tables.shape
    shape = _BOOKS_SHAPE.pack(refs.shape[0], rows, width, _stride(tables, 0),
                              outs[1].stride(0) if rows > 1 else width, page_size)
    return ins, outs, shape


def _pool_shape(pool: torch.Tensor, pages: int | None) -> bytes:
    """`pool` [planes, pages, ...] with dense pages, packed for the library."""
    if not pool.is_cuda or pool.dim() < 3:
        raise ValueError("pool must be a CUDA tensor [planes, pages, ...]")
    if pages is not None and pool.shape[1] != pages:
        raise ValueError(f"pool has {pool.shape[1]} pages, the books {pages}")
    if not pool[0, 0].is_contiguous():
        raise ValueError("pool must be dense within a page")
    size = pool.element_size()
    return _POOL_SHAPE.pack(pool.shape[0], _stride(pool, 0) * size, _stride(pool, 1) * size,
                            pool[0, 0].numel() * size)


def _space(books: bytes, count: int, dev, stream) -> torch.Tensor:
    n = _native.lib().w4a16_pages_workspace(books, count)
    if n < 0:
        _native.check(2, "w4a16_pages_workspace")
    return _empty(n, torch.uint8, dev, stream)


def pages_free(refs: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
               rows: torch.Tensor, out=None, stream=None):
    """Gives back the pages of the listed rows (int32): one holder fewer in
    refs [pages], page numbers -1 in tables [rows, width], length 0.  Returns
    (refs, tables, lengths), new tensors or `out` (which may be the inputs)."""
    ins, outs, shape = _books(refs, tables, lengths, out, 1, stream)
    _ints(rows, "rows", (None,))
    dev = _device_of(stream, ("refs", refs), ("tables", tables), ("lengths", lengths),
                     ("rows", rows), *(("out", o) for o in outs))
    rc = _call(dev, _native.lib().w4a16_pages_free, *(t.data_ptr() for t in ins), rows.data_ptr(),
               rows.shape[0], *(t.data_ptr() for t in outs), shape, _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_pages_free")
    return outs


def pages_extend(refs: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
                 rows: torch.Tensor, counts: torch.Tensor, page_size: int, out=None, stream=None):
    """Makes rows[i] longer by counts[i] positions and gives it the lowest free
    pages it then needs, in the order of the list.  Returns (refs, tables,
    lengths, done); done[i] = 0 where the row is left as it was: too few free
    pages, a row too long, out of range or listed before."""
    ins, outs, shape = _books(refs, tables, lengths, out, page_size, stream)
    _ints(rows, "rows", (None,))
    _ints(counts, "counts", (rows.shape[0],))
    dev = _device_of(stream, ("refs", refs), ("tables", tables), ("lengths", lengths),
                     ("rows", rows), ("counts", counts), *(("out", o) for o in outs))
    done = _empty(rows.shape, torch.int32, dev, stream)
    space = _space(shape, rows.shape[0], dev, stream)
    rc = _call(dev, _native.lib().w4a16_pages_extend, *(t.data_ptr() for t in ins),
               rows.data_ptr(), counts.data_ptr(), rows.shape[0], *(t.data_ptr() for t in outs),
               done.data_ptr(), space.data_ptr(), shape, _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_pages_extend")
    return *outs, done


def pages_fork(pool: torch.Tensor, refs: torch.Tensor, tables: torch.Tensor,
               lengths: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
               page_size: int, out=None, stream=None):
    """Makes the empty row children[i] a copy of row parents[i]: full pages are
    shared, a partly filled last page is copied in every plane of pool
    [planes, pages, ...] to the lowest free page.  Returns (refs, tables,
    lengths, done); done[i] = 0 where the child is left as it was: too few free
    pages, a child not empty, a row out of range or a child listed before."""
    ins, outs, shape = _books(refs, tables, lengths, out, page_size, stream)
    planes = _pool_shape(pool, refs.shape[0])
    _ints(parents, "parents", (None,))
    _ints(children, "children", (parents.shape[0],))
    dev = _device_of(stream, ("pool", pool), ("refs", refs), ("tables", tables),
                     ("lengths", lengths), ("parents", parents), ("children", children),
                     *(("out", o) for o in outs))
    done = _empty(parents.shape, torch.int32, dev, stream)
    space = _space(shape, parents.shape[0], dev, stream)
    rc = _call(dev, _native.lib().w4a16_pages_fork, pool.data_ptr(),
               *(t.data_ptr() for t in ins), parents.data_ptr(), children.data_ptr(),
               parents.shape[0], *(t.data_ptr() for t in outs), done.data_ptr(), space.data_ptr(),
               shape, planes, _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_pages_fork")
    return *outs, done


def pages_compact(pool: torch.Tensor, refs: torch.Tensor, tables: torch.Tensor, out=None,
                  stream=None):
    """Moves the n held pages to the numbers below n: those at n and above go,
    in ascending order, to the free ones below, in every plane of pool
    [planes, pages, ...].  Returns (refs, tables, used) with used = [n]."""
    ins, outs, shape = _books(refs, tables, None, out, 1, stream)
    planes = _pool_shape(pool, refs.shape[0])
    dev = _device_of(stream, ("pool", pool), ("refs", refs), ("tables", tables),
                     *(("out", o) for o in outs))
    used = _empty((1,), torch.int32, dev, stream)
    space = _space(shape, 0, dev, stream)
    rc = _call(dev, _native.lib().w4a16_pages_compact, pool.data_ptr(),
               *(t.data_ptr() for t in ins), *(t.data_ptr() for t in outs), used.data_ptr(),
               space.data_ptr(), shape, planes, _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_pages_compact")
    return *outs, used


def pages_copy(pool: torch.Tensor, sources: torch.Tensor, targets: torch.Tensor,
               stream=None) -> None:
    """Copies page sources[i] to page targets[i] (int32) in every plane of pool
    [planes, pages, ...]; pairs out of range are passed over."""
    planes = _pool_shape(pool, None)
    _ints(sources, "sources", (None,))
    _ints(targets, "targets", (sources.shape[0],))
    dev = _device_of(stream, ("pool", pool), ("sources", sources), ("targets", targets))
    rc = _call(dev, _native.lib().w4a16_pages_copy, pool.data_ptr(), sources.data_ptr(),
               targets.data_ptr(), sources.shape[0], pool.shape[1], planes,
               _stream_ptr(stream, dev))
    if rc:
        _native.check(rc, "w4a16_pages_copy")


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, stream=None):
    """Scores of the given tokens (int64 or int32 [rows]) under logits [rows,
    vocabulary] (fp16, bf16 or fp32, dense in the last dimension): returns
    (logprobs, entropies, top_ids, top_logprobs), fp32 [rows] twice, int32 and
    fp32 [rows, top]; the `top` (at most 32) largest logits come first, of equal
    ones the lowest index.  -inf masks a logit; a token outside the vocabulary
    has the log probability NaN."""
    if logits.dim() != 2 or logits.dtype not in _TYPES or not logits.is_cuda:
        raise ValueError("logits must be a float16, bfloat16 or float32 CUDA tensor "
                         f"[rows, vocabulary], got {logits.dtype} {list(logits.shape)}")
    rows, vocabulary = logits.shape
    if vocabulary > 1 and logits.stride(1) != 1:
        raise ValueError("logits must be dense in their last dimension")
    if tokens.dtype not in (torch.int64, torch.int32) or tokens.shape != (rows,) \
            or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a dense int64 or int32 tensor [{rows}]")
    if not 0 <= top <= min(MAX_TOP, vocabulary):
        raise ValueError(f"top must be 0 .. {min(MAX_TOP, vocabulary)}, got {top}")
    dev = _device_of(stream, ("logits", logits), ("tokens", tokens))
    logprobs = _empty(rows, torch.float32, dev, stream)
    entropies = _empty(rows, torch.float32, dev, stream)
    ids = _empty((rows, top), torch.int32, dev, stream)
    likeliest = _empty((rows, top), torch.float32, dev, stream)
    if rows:
        rc = _call(dev, _native.lib().w4a16_token_logprobs, logits.data_ptr(), tokens.data_ptr(),
                   logprobs.data_ptr(), entropies.data_ptr(), ids.data_ptr(),
                   likeliest.data_ptr(), rows, vocabulary, _stride(logits, 0),
                   _TYPES[logits.dtype], tokens.dtype == torch.int64, top,
                   _stream_ptr(stream, dev))
        if rc:
            _native.check(rc, "w4a16_token_logprobs")
    return logprobs, entropies, ids, likeliest


class PagedCache:
    """The keys and values of a decoder's layers for `rows` sequences, in pages
    that sequences take, share and give back.

    pool [2 * layers, pages, page_size, kv_heads, head_dim] holds layer l's keys
    in plane 2l and its values in plane 2l + 1; one page number means the same
    page of every plane.  refs, tables and lengths are the books the pages_*
    functions keep, updated in place, so the methods may be captured in a CUDA
    graph."""

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

    def extend(self, rows: torch.Tensor, counts: torch.Tensor, stream=None) -> torch.Tensor:
        """Room for counts[i] more positions in rows[i]; returns done (pages_extend)."""
        return pages_extend(*self._all(), rows, counts, self.page_size, out=self._all(),
                            stream=stream)[3]

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
               offsets: torch.Tensor | None = None, rows: torch.Tensor | None = None,
               stream=None) -> None:
        """New tokens of every row (or of the listed ones) of one layer (paged_append)."""
        tables = self.tables if rows is None else self.tables.index_select(0, rows)
        paged_append(k, v, self.pool[2 * layer], self.pool[2 * layer + 1], tables, starts, offsets,
                     stream=stream)

    def attend(self, layer: int, q: torch.Tensor, rows: torch.Tensor | None = None,
               scale: float | None = None, out: torch.Tensor | None = None, stream=None):
        """Attention of one new token of every row (or of the listed ones) (paged_attention)."""
        tables, lengths = self.tables, self.lengths
        if rows is not None:
            tables, lengths = tables.index_select(0, rows), lengths.index_select(0, rows)
        return paged_attention(q, self.pool[2 * layer], self.pool[2 * layer + 1], tables, lengths,
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
