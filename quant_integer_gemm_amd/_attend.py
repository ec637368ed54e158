"""ctypes binding of the attention operators, the 4-bit cache and its pages.

As in _int8: sizes, strides, types and devices are checked before a pointer
reaches the library; all tensors of a call must be on one GPU, and it runs on
that GPU's current stream (or ``stream``).  Lengths, starts and tables stay on the
GPU: nothing in these calls visits the host, so a decoding step with them can
be captured into a graph.
"""
from __future__ import annotations

import struct

from . import _int8 as _i
from ._int8 import _device_of, _is, _matrix, _new, _type
from ._lib import QigError, load

# The library's calls by number, their arguments packed into one block of 8-byte words
# (qig_attend_packed): ctypes takes 5 us to convert 25 arguments and 1 us for a block.
_OPS = {name: (n, struct.Struct(layout)) for n, (name, layout) in enumerate((
    ("attend_prompt", "=19qd4q"), ("write_kv4", "=20q"), ("read_kv4", "=20q"), ("attend_kv4", "=18qd5q"),
    ("copy_pages", "=7q"), ("free_pages", "=9q"), ("take_pages", "=10q"), ("fork_pages", "=16q"),
    ("compact_pages", "=12q")))}


def _start():
    global _i32, _u8, _packed
    if _i.torch is None:
        _i._start()
    _i32, _u8, _packed = _i.torch.int32, _i.torch.uint8, load().qig_attend_packed
    return _i.torch


_packed = None


def _call(what, names, tensors, stream, *args):
    """The library's call `what` with these arguments, on the GPU of the tensors."""
    op, layout = _OPS[what]
    dev, here, handle = _device_of(names, tensors, stream)
    if here:
        rc = _packed(op, layout.pack(*args), handle)
    else:
        with _i.torch.cuda.device(dev):
            rc = _packed(op, layout.pack(*args), handle)
    if rc:
        _i._check(rc, what)


def _heads(t, name, heads=None, d=None):
    """(tokens, heads, d, token stride, head stride) of a 3-D tensor with unit
    stride in its last dimension."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1 and t.numel() > 0):
        raise QigError(f"{name} must be [tokens][heads][d] with unit stride in the last dimension")
    n, h, c = shape
    if heads is not None and h != heads:
        raise QigError(f"{name} has {h} heads, not {heads}")
    if d is not None and c != d:
        raise QigError(f"{name} has heads of {c}, not {d}")
    return n, h, c, stride[0], stride[1]


def _result(y, name, dtype, nt, heads, d, device, stream):
    """(y, its type's code, token stride, head stride); a given y's rows may not
    overlap."""
    if y is None:
        return _new((nt, heads, d), dtype, device, stream), _type(dtype, name), heads * d, d
    if dtype is not None and y.dtype != dtype:
        raise QigError(f"{name} is {y.dtype}, dtype asks for {dtype}")
    code = _type(y.dtype, name)
    n, _, _, token, head = _heads(y, name, heads, d)
    if n != nt:
        raise QigError(f"{name} holds {n} tokens, not {nt}")
    if not ((head >= d or heads <= 1) and (token >= (heads - 1) * head + d or nt <= 1)
            or (token >= d or nt <= 1) and (head >= (nt - 1) * token + d or heads <= 1)):
        raise QigError(f"{name}'s rows overlap: strides {y.stride()} for {list(y.shape)}")
    return y, code, token, head


def _ints(t, n, name):
    """A contiguous int32 vector of n."""
    if t.dtype is _i32 and t.shape == (n,) and t.is_contiguous():
        return
    _is(t, _i32, name)
    raise QigError(f"{name} must be contiguous with {n} elements, not {list(t.shape)}")


def _length(t, name):
    if len(t.shape) != 1:
        raise QigError(f"{name} must be a vector")
    return t.shape[0]


def _table(tables):
    """(rows, entries a row, row stride)."""
    if tables.dtype is not _i32:
        _is(tables, _i32, "tables")
    return _matrix(tables, "tables")


def attend_prompt(q, k, v, starts, k_starts=None, causal=True, scale=None, y=None, dtype=None, stream=None):
    """y[nt][hq][d]: attention of the queries q[nt][hq][d] of packed sequences
    over their keys and values k, v[nk][hkv][d] (fp32, bf16 or fp16, all of one
    type; hq / hkv query heads in a row share a key head).  Sequence s has the
    rows starts[s] .. starts[s + 1] of q and those of k_starts (starts where it is
    None) of k and v; both int32 on the GPU.  causal: a query sees the keys up to
    its own position, the last query being at the last key's; else all of them.
    scale: 1 / sqrt(d) where it is None.  y is of q's type, or of ``dtype`` or the
    given y's type; rows outside of every sequence are not written, queries that
    see no key get zeros."""
    if _packed is None:
        _start()
    qt = _type(q.dtype, "q")
    _is(k, q.dtype, "k")
    _is(v, q.dtype, "v")
    nt, hq, d, qn, qh = _heads(q, "q")
    nk, hkv, _, kn, kh = _heads(k, "k", None, d)
    nv, _, _, vn, vh = _heads(v, "v", hkv, d)
    if nv != nk:
        raise QigError(f"v has {nv} tokens, k has {nk}")
    n = _length(starts, "starts")
    if n < 1:
        raise QigError("starts must hold one more than the sequences")
    _ints(starts, n, "starts")
    if k_starts is None:
        k_starts = starts
    elif k_starts is not starts:
        _ints(k_starts, n, "k_starts")
    if scale is not None and not scale > 0:
        raise QigError(f"scale must be above 0, not {scale}")
    if dtype is None and y is None:
        dtype = q.dtype
    y, yt, yn, yh = _result(y, "y", dtype, nt, hq, d, q.device, stream)
    _call("attend_prompt", ("q", "k", "v", "starts", "k_starts", "y"), (q, k, v, starts, k_starts, y), stream,
          q.data_ptr(), qn, qh, k.data_ptr(), kn, kh, v.data_ptr(), vn, vh, qt, nt, nk, hq, hkv, d,
          starts.data_ptr(), k_starts.data_ptr(), n - 1, 1 if causal else 0, 0.0 if scale is None else scale,
          y.data_ptr(), yn, yh, yt)
    return y


# --- the 4-bit cache -------------------------------------------------------------

def kv4_page_bytes(page: int, heads: int, d: int) -> int:
    """Bytes of a page: 1.25 d a token and head, keys and values together."""
    return int(load().kv4_page_bytes(page, heads, d))


def new_kv4(npages, heads, d, page=64, device="cuda"):
    """Pages for a 4-bit cache, uint8 [npages][heads][1.25 * page * d].  page: tokens
    of a page, a multiple of 32; d: 64, 128 or 256.  Several layers may share a
    pool: any tensor [npages][layers][heads][1.25 * page * d], of which the calls
    take pages[:, layer] and the pages' operators the whole."""
    torch = _start()
    n = kv4_page_bytes(page, heads, d)
    if n == 0 or npages < 0:
        raise QigError(f"no cache of {npages} pages of {page} tokens with {heads} heads of {d}")
    return torch.empty((npages, heads, n // heads), dtype=torch.uint8, device=device)


def _cache(pages, tables, lengths, starts, nt, d):
    """The cache's arguments of a call, from heads of d on."""
    if pages.dtype is not _u8:
        _is(pages, _u8, "pages")
    shape, stride = pages.shape, pages.stride()
    if len(shape) != 3:
        raise QigError("pages must be [pages][heads][bytes], each page contiguous")
    npages, heads, nbytes = shape
    if (stride[2] != 1 or (heads > 1 and stride[1] != nbytes)) and pages.numel() > 0:
        raise QigError("pages must be [pages][heads][bytes], each page contiguous")
    page, rest = divmod(nbytes * 4, 5 * d) if d > 0 else (0, 1)
    if rest or page % 32 or page == 0:
        raise QigError(f"pages of {nbytes} bytes a head hold no whole blocks of 32 tokens with heads of {d}")
    nseq, width, ld = _table(tables)
    _ints(lengths, nseq, "lengths")
    if starts is None:
        if nt != nseq:
            raise QigError(f"{nt} tokens for {nseq} sequences: starts says which are whose")
        at = 0
    else:
        _ints(starts, nseq + 1, "starts")
        at = starts.data_ptr()
    return (heads, d, pages.data_ptr(), npages, stride[0] if npages > 1 else heads * nbytes, page, tables.data_ptr(), ld,
            width, lengths.data_ptr(), at, nseq)


_ROWS = ("k", "v", "pages", "tables", "lengths", "starts")


def write_kv4(k, v, pages, tables, lengths, starts=None, stream=None):
    """Put keys and values k, v[nt][heads][d] (fp32, bf16 or fp16) into the cache
    as the last tokens of their sequences.  tables[nseq][width] (int32) lists each
    sequence's pages, lengths[nseq] (int32) its tokens with the new ones; sequence
    s's are the rows starts[s] .. starts[s + 1], or without starts row s alone.
    Tokens whose place the table does not have are left out."""
    if _packed is None:
        _start()
    code = _type(k.dtype, "k")
    _is(v, k.dtype, "v")
    nt, heads, d, kn, kh = _heads(k, "k")
    nv, _, _, vn, vh = _heads(v, "v", heads, d)
    if nv != nt:
        raise QigError(f"v has {nv} tokens, k has {nt}")
    cache = _cache(pages, tables, lengths, starts, nt, d)
    if cache[0] != heads:
        raise QigError(f"k has {heads} heads, pages have {cache[0]}")
    _call("write_kv4", _ROWS, (k, v, pages, tables, lengths, starts), stream,
          k.data_ptr(), kn, kh, v.data_ptr(), vn, vh, code, nt, *cache)


def read_kv4(pages, tables, lengths, d, starts=None, nt=None, k=None, v=None, dtype=None, stream=None):
    """(k, v): the last tokens of each sequence back as the values that the cache
    stands for, [nt][heads][d]; arguments as write_kv4.  nt: the rows, where
    starts is given and k is not.  fp32, or of ``dtype`` or the given tensors' type.
    Rows that stand nowhere in the cache are zeros, those outside of every
    sequence are not written."""
    if _packed is None:
        _start()
    if nt is None:
        if k is not None or v is not None:
            nt = (v if k is None else k).shape[0]
        elif starts is None:
            nt = tables.shape[0]
        else:
            raise QigError("nt is needed with starts: the rows of k and v")
    cache = _cache(pages, tables, lengths, starts, nt, d)
    heads = cache[0]
    if dtype is None:
        dtype = _i.torch.float32 if k is None and v is None else (v if k is None else k).dtype
    k, code, kn, kh = _result(k, "k", dtype, nt, heads, d, pages.device, stream)
    v, _, vn, vh = _result(v, "v", dtype, nt, heads, d, pages.device, stream)
    _call("read_kv4", _ROWS, (k, v, pages, tables, lengths, starts), stream,
          k.data_ptr(), kn, kh, v.data_ptr(), vn, vh, code, nt, *cache)
    return k, v


def attend_kv4(q, pages, tables, lengths, starts=None, scale=None, y=None, dtype=None, ws=None, stream=None):
    """y[nt][hq][d]: attention of the sequences' last tokens, q[nt][hq][d] (fp32,
    bf16 or fp16), over all their tokens in the cache; arguments as write_kv4.
    The last query of a sequence sees all lengths[s] tokens, each one before it one
    less.  Pages that the table does not have are left out; queries that see
    nothing get zeros.  scale: 1 / sqrt(d) where it is None.  y is of q's type, or of
    ``dtype`` or the given y's.  ws: None, or a workspace (qig.workspace()), which
    lets long sequences be split over the whole GPU; where all are shorter than a
    thousand tokens or so the call is faster without."""
    if _packed is None:
        _start()
    code = _type(q.dtype, "q")
    nt, hq, d, qn, qh = _heads(q, "q")
    cache = _cache(pages, tables, lengths, starts, nt, d)
    if scale is not None and not scale > 0:
        raise QigError(f"scale must be above 0, not {scale}")
    if dtype is None and y is None:
        dtype = q.dtype
    y, yt, yn, yh = _result(y, "y", dtype, nt, hq, d, q.device, stream)
    if ws is not None and (ws.numel() * (1 if ws.dtype is _u8 else ws.element_size()) < _i._ws_bytes
                           or not ws.is_contiguous()):
        raise QigError(f"ws holds {ws.numel() * ws.element_size()} bytes, the call needs {_i._ws_bytes}, contiguous")
    _call("attend_kv4", ("q", "pages", "tables", "lengths", "starts", "y", "ws"),
          (q, pages, tables, lengths, starts, y, ws), stream, q.data_ptr(), qn, qh, code, nt, hq, *cache,
          0.0 if scale is None else scale, y.data_ptr(), yn, yh, yt, 0 if ws is None else ws.data_ptr())
    return y


# --- pages -----------------------------------------------------------------------

def _whole_pages(pages):
    """(pages, bytes of one, bytes from one to the next): any tensor whose first
    dimension counts pages, each of them contiguous."""
    shape, stride = pages.shape, pages.stride()
    if len(shape) < 2:
        raise QigError("pages must have a dimension of pages and others in each page")
    n = 1
    for i in range(len(shape) - 1, 0, -1):
        if stride[i] != n and shape[i] != 1 and pages.numel() > 0:
            raise QigError("each page must be contiguous")
        n *= shape[i]
    e = pages.element_size()
    return shape[0], n * e, stride[0] * e if shape[0] > 1 else n * e


def _refs(refs):
    if refs.dtype is not _i32:
        _is(refs, _i32, "refs")
    if len(refs.shape) != 1 or not refs.is_contiguous():
        raise QigError("refs must be a contiguous vector, a count a page")
    return refs.shape[0]


def _count_and_scratch(given, name, npages, rows, device, stream):
    """The int32 [1] that a call returns and its scratch memory: one new tensor, of
    which the count is the first word (the scratch stands 8 bytes on)."""
    n = (npages + 63) // 64 * 8 + rows * 4 + 8
    if not 0 < npages <= 1 << 20:
        raise QigError(f"no pool of {npages} pages")
    scratch = _new(((n + 3) // 4,), _i32, device, stream)
    if given is None:
        given = scratch[:1]
    else:
        _ints(given, 1, name)
    return given, scratch


def copy_pages(pages, src, dst, stream=None):
    """pages[dst[i]] = pages[src[i]] for every i (int32 vectors on the GPU); a pair
    with an index outside of the pages is left out.  No page may be named twice in
    dst, or in both src and dst other than in one pair.  pages: any tensor whose first
    dimension counts pages, each contiguous and of a multiple of 16 bytes."""
    if _packed is None:
        _start()
    npages, nbytes, step = _whole_pages(pages)
    n = _length(src, "src")
    _ints(src, n, "src")
    _ints(dst, n, "dst")
    _call("copy_pages", ("pages", "src", "dst"), (pages, src, dst), stream,
          pages.data_ptr(), npages, nbytes, step, src.data_ptr(), dst.data_ptr(), n)


def take_pages(tables, lengths, refs, page, missing=None, stream=None):
    """Give every sequence the pages that its length needs: each entry below
    ceil(lengths[s] / page) of tables[s] that holds none gets a free one (refs 0,
    then 1), the lowest first, in the order of the table.  Returns int32 [1]: how many
    found none and stay -1.  What a length has beyond the table's width is not
    counted: the caller keeps lengths within width * page."""
    if _packed is None:
        _start()
    rows, width, ld = _table(tables)
    _ints(lengths, rows, "lengths")
    npages = _refs(refs)
    missing, scratch = _count_and_scratch(missing, "missing", npages, rows, refs.device, stream)
    _call("take_pages", ("tables", "lengths", "refs", "missing"), (tables, lengths, refs, missing), stream,
          tables.data_ptr(), rows, ld, width, lengths.data_ptr(), refs.data_ptr(), npages, page, missing.data_ptr(),
          scratch.data_ptr() + 8)
    return missing


def free_pages(tables, lengths, refs, rows, stream=None):
    """The table's rows named by rows (int32 vector) give up their pages: refs of
    each is one less, their entries are -1 and their lengths 0.  Rows named twice
    do so once; those that the table does not have are left out."""
    if _packed is None:
        _start()
    height, width, ld = _table(tables)
    _ints(lengths, height, "lengths")
    npages, n = _refs(refs), _length(rows, "rows")
    _ints(rows, n, "rows")
    _call("free_pages", ("tables", "lengths", "refs", "rows"), (tables, lengths, refs, rows), stream,
          tables.data_ptr(), height, ld, width, lengths.data_ptr(), refs.data_ptr(), npages, rows.data_ptr(), n)


def fork_pages(pages, tables, lengths, refs, parents, children, page, missing=None, stream=None):
    """Row children[i] of the table becomes a copy of row parents[i] (int32 vectors):
    it gives up what it held, shares the parent's full pages, and has its last page,
    where that is not full, copied to a free one (the lowest, in the order of the
    pairs).  A pair counts where both rows are the table's, no later pair has the
    same child and no pair has its parent as child.  Returns int32 [1]: how many
    copies found no free page (the child's entry is then -1)."""
    if _packed is None:
        _start()
    npages, nbytes, step = _whole_pages(pages)
    rows, width, ld = _table(tables)
    _ints(lengths, rows, "lengths")
    if _refs(refs) != npages:
        raise QigError(f"refs counts {refs.shape[0]} pages, pages has {npages}")
    n = _length(parents, "parents")
    _ints(parents, n, "parents")
    _ints(children, n, "children")
    missing, scratch = _count_and_scratch(missing, "missing", npages, n, refs.device, stream)
    _call("fork_pages", ("pages", "tables", "lengths", "refs", "parents", "children", "missing"),
          (pages, tables, lengths, refs, parents, children, missing), stream,
          pages.data_ptr(), nbytes, step, tables.data_ptr(), rows, ld, width, lengths.data_ptr(), refs.data_ptr(),
          npages, page, parents.data_ptr(), children.data_ptr(), n, missing.data_ptr(), scratch.data_ptr() + 8)
    return missing


def compact_pages(pages, tables, refs, used=None, to=None, stream=None):
    """Move the pages in use (refs above 0) to the front of the pool: with U of them,
    the k-th in use from page U on goes to the k-th free page below U, and refs and
    the tables' entries follow.  Returns int32 [1]: U.  to: None, or an int32 vector
    that receives each page's place after it, for pages that are known elsewhere."""
    if _packed is None:
        _start()
    npages, nbytes, step = _whole_pages(pages)
    rows, width, ld = _table(tables)
    if _refs(refs) != npages:
        raise QigError(f"refs counts {refs.shape[0]} pages, pages has {npages}")
    if to is not None:
        _ints(to, npages, "to")
    used, scratch = _count_and_scratch(used, "used", npages, 0, refs.device, stream)
    _call("compact_pages", ("pages", "tables", "refs", "used", "to"), (pages, tables, refs, used, to), stream,
          pages.data_ptr(), nbytes, step, tables.data_ptr(), rows, ld, width, refs.data_ptr(), npages, used.data_ptr(),
          0 if to is None else to.data_ptr(), scratch.data_ptr() + 8)
    return used
