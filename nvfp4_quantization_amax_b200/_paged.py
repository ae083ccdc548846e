"""The paged packed cache: append, page bounds, page selection and the
attention of one new token.  Argument marshalling only.

The cache of K (and of V) is a pair (codes, scales) of contiguous uint8 CUDA
tensors: what quantize_cache_packed returns for values [pages, kv_heads,
page_size, head_dim].  It stays where it is: these calls never copy it.
"""
import math

import torch

from ._abi import _DTYPES, _FORMATS, _check, _device_word, _out, _result, _to_device, lib

_U8, _I32 = torch.uint8, torch.int32
# The raw handle of a device's current stream, without a Stream object (a step
# of serving makes several of these calls, and its host time is theirs).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
        lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ints(t, shape, dev, name):
    """An int32 tensor of a call (page table, lengths, offs, a page list)."""
    if t.dtype is not _I32:
        raise TypeError("%s must be int32, not %s" % (name, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, list(shape), list(t.shape)))
    if t.device != dev:
        t, _ = _to_device(t, dev, False)
    return t if t.is_contiguous() else t.contiguous()


def _cache(cache, format, block_size, name):
    """(codes, scales, codes' shape) of a cache."""
    codes, scales = cache
    shape, sshape = codes.shape, scales.shape
    if (codes.dtype is not _U8 or scales.dtype is not _U8 or len(shape) != 4 or len(sshape) != 4
            or not codes.is_cuda or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError("%s: codes and scales must be contiguous uint8 CUDA tensors of 4 "
                         "dimensions" % name)
    if (sshape[:3] != shape[:3]
            or sshape[3] * block_size != (shape[3] if format == "fp8" else 2 * shape[3])):
        raise ValueError("%s: scales must have shape [pages, kv_heads, page_size, head_dim / "
                         "block_size]" % name)
    if scales.device != codes.device:
        raise ValueError("%s: codes and scales must share a device" % name)
    return codes, scales, shape


def _second(cache, format, block_size, name, first):
    """V's (codes, scales): as K's in shape and device."""
    codes, scales, shape = _cache(cache, format, block_size, name)
    if shape != first.shape or codes.device != first.device:
        raise ValueError("%s must have K's shape and device" % name)
    return codes, scales


def _format(format, block_size, what):
    if format not in _FORMATS:
        raise ValueError("%s: format must be one of %s" % (what, sorted(_FORMATS)))
    if block_size < 1:
        raise ValueError("%s: block_size must be >= 1" % what)
    return _FORMATS[format]


def _table(page_table, what):
    if page_table.dim() != 2:
        raise ValueError("%s: page_table must be [sequences, max_pages]" % what)
    return page_table.shape


def _rows(t, dev, waits=True):
    """(device tensor, elements between its rows, was on the host) of a tensor
    [rows, heads, channels] whose rows must be dense, the rows themselves at
    any distance.  waits: whether the call waits for its results where this
    one is on the host."""
    host = False
    if t.device != dev:
        t, host = _to_device(t, dev, waits)
    n, heads, dim = t.shape
    row = heads * dim
    if not t.is_contiguous():
        apart, head, one = t.stride()
        if one == 1 and head == dim and apart >= row:
            return t, apart, host
        t = t.contiguous()
    return t, row, host


def _run(dev, what, fn, *args):
    """Call the library on dev's current stream, with dev current."""
    index = dev.index
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        _check(rc, what)


def _word(t, dev):
    """The optional status word."""
    return None if t is None else _device_word(t, _I32, 1, dev, "status")


def _scratch(t, need, dev):
    """The optional workspace, or a new one (kept alive by the caller until the
    call is made; the allocator hands its memory on in stream order)."""
    if t is None:
        return torch.empty(need, dtype=_U8, device=dev)
    _device_word(t, _U8, need, dev, "workspace")
    return t


def append_cache_paged(k, v, offs, page_table, lengths, k_cache, v_cache, format, block_size,
                       values=False, status=None):
    """Quantize new K and V rows into their pages.

    k, v: bf16/f16/f32 [rows, kv_heads, head_dim] (rows may be strided slices
    of a projection's output); offs int32 [sequences]: cumulative new rows,
    as in the grouped GEMM; page_table int32 [sequences, max_pages]; lengths
    int32 [sequences]: tokens with the new ones counted, so that a sequence's
    last new row goes to position lengths - 1.  Rows behind offs[-1] are
    padding.  k_cache, v_cache: (codes, scales), written in place; v and
    v_cache may both be None.  values=True returns (k, v) as the cache holds
    them (what quantize_cache gives; the padding's rows are not written), else
    None.  status: optional device int32 [1]: a bad offs, page, length or row
    is reported there, and its rows are left out.
    """
    what = "append_cache_paged"
    fmt = _format(format, block_size, what)
    if (v is None) != (v_cache is None):
        raise ValueError("%s: v and v_cache belong together" % what)
    kc, ks, (P, H, S, D) = _cache(k_cache, format, block_size, "k_cache")
    D = D if fmt == 0 else 2 * D
    dev = kc.device
    vc = vs = None
    if v is not None:
        vc, vs = _second(v_cache, format, block_size, "v_cache", kc)
        if v.dtype != k.dtype or v.shape != k.shape:
            raise ValueError("%s: k and v must have one dtype and shape" % what)
    if k.dtype not in _DTYPES:
        raise TypeError("%s: unsupported dtype %s" % (what, k.dtype))
    if k.dim() != 3 or k.shape[1] != H or k.shape[2] != D:
        raise ValueError("%s: k must be [rows, %d, %d]" % (what, H, D))
    n, M = _table(page_table, what)
    page_table = _ints(page_table, (n, M), dev, "page_table")
    lengths = _ints(lengths, (n,), dev, "lengths")
    offs = _ints(offs, (n,), dev, "offs")
    k, k_stride, host = _rows(k, dev, values)
    v_stride = 0
    if v is not None:
        v, v_stride, _ = _rows(v, dev, values and host)
    T = k.shape[0]
    k_out = v_out = None
    if values:
        k_out = torch.empty((T, H, D), dtype=k.dtype, device=dev)
        v_out = torch.empty((T, H, D), dtype=k.dtype, device=dev) if v is not None else None
    ptr = [None if x is None else x.data_ptr() for x in (v, vc, vs, k_out, v_out)]
    _run(dev, what, lib().append_cache_paged, k.data_ptr(), ptr[0], _DTYPES[k.dtype], T, H, D,
         k_stride, v_stride, offs.data_ptr(), page_table.data_ptr(), lengths.data_ptr(), n, M, fmt,
         block_size, P, S, kc.data_ptr(), ks.data_ptr(), ptr[1], ptr[2], ptr[3], ptr[4],
         _word(status, dev))
    if not values:
        return None
    return _result(k_out, None, host), None if v is None else _result(v_out, None, host)


def bound_cache_pages(k_cache, page_table, lengths, format, block_size, bounds=None,
                      new_tokens=None, status=None):
    """Channelwise least and largest key of the pages, over their valid tokens.

    Writes bounds bf16 [pages, kv_heads, 2, head_dim] (a new tensor of zeros
    where none is given) for the pages that hold each sequence's last
    new_tokens tokens (None: for all of its pages), and returns it.
    """
    what = "bound_cache_pages"
    fmt = _format(format, block_size, what)
    kc, ks, (P, H, S, D) = _cache(k_cache, format, block_size, "k_cache")
    D = D if fmt == 0 else 2 * D
    dev = kc.device
    n, M = _table(page_table, what)
    page_table = _ints(page_table, (n, M), dev, "page_table")
    lengths = _ints(lengths, (n,), dev, "lengths")
    if bounds is None:
        bounds = torch.zeros((P, H, 2, D), dtype=torch.bfloat16, device=dev)
    if not bounds.is_cuda:
        raise ValueError("%s: bounds must be a CUDA tensor" % what)
    bounds, _ = _out(bounds, (P, H, 2, D), torch.bfloat16, dev, "bounds")
    _run(dev, what, lib().bound_cache_pages, kc.data_ptr(), ks.data_ptr(), H, D, fmt, block_size,
         P, S, page_table.data_ptr(), lengths.data_ptr(), n, M,
         M * S if new_tokens is None else int(new_tokens), bounds.data_ptr(), _word(status, dev))
    return bounds


def _queries(q, dev, H, D, what):
    if q.dtype not in _DTYPES:
        raise TypeError("%s: unsupported dtype %s" % (what, q.dtype))
    if q.dim() != 3 or q.shape[2] != D or q.shape[1] < 1 or q.shape[1] % H != 0:
        raise ValueError("%s: q must be [sequences, a multiple of %d, %d]" % (what, H, D))
    return _rows(q, dev)


def select_cache_pages(q, bounds, page_table, lengths, page_size, top, keep_first=0, keep_last=1,
                       out=None, workspace=None, status=None):
    """Pages that each sequence's new token attends to.

    q [sequences, q_heads, head_dim]; bounds as bound_cache_pages writes them.
    Returns int32 [sequences, kv_heads, top]: positions in the page table,
    ascending, -1 behind the last: the sequence's first keep_first and last
    keep_last pages, and those with the largest bound of the head group's
    summed logits (in 64 bits; equal ones from the front).
    workspace: optional device uint8 scratch of 8 bytes per sequence, kv head
    and table entry.
    """
    what = "select_cache_pages"
    if not bounds.is_cuda or bounds.dtype != torch.bfloat16 or not bounds.is_contiguous():
        raise ValueError("%s: bounds must be a contiguous bf16 CUDA tensor" % what)
    if bounds.dim() != 4 or bounds.shape[2] != 2:
        raise ValueError("%s: bounds must be [pages, kv_heads, 2, head_dim]" % what)
    P, H, _, D = bounds.shape
    dev = bounds.device
    q, q_stride, host = _queries(q, dev, H, D, what)
    n, M = q.shape[0], _table(page_table, what)[1]
    page_table = _ints(page_table, (n, M), dev, "page_table")
    lengths = _ints(lengths, (n,), dev, "lengths")
    top = int(top)
    if top < 0:
        raise ValueError("%s: top must not be negative" % what)
    out, target = _out(out, (n, H, top), _I32, dev, "out")
    ws = _scratch(workspace, 8 * n * H * M, dev)
    _run(dev, what, lib().select_cache_pages, q.data_ptr(), _DTYPES[q.dtype], n, q.shape[1], H, D,
         q_stride, bounds.data_ptr(), P, int(page_size), page_table.data_ptr(),
         lengths.data_ptr(), M, top, int(keep_first), int(keep_last), out.data_ptr(),
         ws.data_ptr(), _word(status, dev))
    return _result(out, target, host)


_attend_need = {}  # workspace bytes by heads, head size and device


def attend_cache_paged(q, k_cache, v_cache, page_table, lengths, format, block_size, scale=None,
                       window=None, pages=None, return_lse=False, out=None, workspace=None,
                       status=None):
    """Attention of one new token per sequence over a paged packed cache.

    q [sequences, q_heads, head_dim], bf16/f16/f32; q head j reads kv head
    j // (q_heads // kv_heads).  scale: of the logits, 1/sqrt(head_dim) where
    None.  window: the sequence's last tokens that are seen (None: all).
    pages: int32 [sequences, kv_heads, n]: only these pages (positions in the
    page table, as select_cache_pages gives them; negative ones are passed
    over, a page listed twice counts twice).  Returns out [sequences, q_heads,
    head_dim] of q's dtype, with return_lse also the float32 [sequences,
    q_heads] natural logarithm of the sum of exponentials of the logits.  A
    sequence without tokens gives zeros and -inf, a query that is not finite
    NaN in its row.  No gradient is defined.
    workspace: optional device uint8 scratch of at least
    attend_cache_paged_workspace_bytes (C) bytes.
    """
    what = "attend_cache_paged"
    fmt = _format(format, block_size, what)
    kc, ks, (P, H, S, D) = _cache(k_cache, format, block_size, "k_cache")
    D = D if fmt == 0 else 2 * D
    vc, vs = _second(v_cache, format, block_size, "v_cache", kc)
    dev = kc.device
    q, q_stride, host = _queries(q, dev, H, D, what)
    n, Hq, _ = q.shape
    M = _table(page_table, what)[1]
    page_table = _ints(page_table, (n, M), dev, "page_table")
    lengths = _ints(lengths, (n,), dev, "lengths")
    top, listed = 0, None
    if pages is not None:
        if pages.dim() != 3:
            raise ValueError("%s: pages must be [sequences, kv_heads, n]" % what)
        top = pages.shape[2]
        if top == 0:
            raise ValueError("%s: pages must list at least one page" % what)
        pages = _ints(pages, (n, H, top), dev, "pages")
        listed = pages.data_ptr()
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("%s: window must be at least 1" % what)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dt = q.dtype
    out, target = _out(out, (n, Hq, D), dt, dev, "out")
    lse = torch.empty((n, Hq), dtype=torch.float32, device=dev) if return_lse else None
    key = (Hq, H, D, dev.index)
    need = _attend_need.get(key)
    if need is None:
        with torch.cuda.device(dev):
            need = _attend_need[key] = lib().attend_cache_paged_workspace_bytes(Hq, H, D)
    ws = _scratch(workspace, need, dev)
    _run(dev, what, lib().attend_cache_paged, q.data_ptr(), _DTYPES[dt], n, Hq, H, D, q_stride,
         kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), fmt, block_size, P, S,
         page_table.data_ptr(), lengths.data_ptr(), M, listed, top, int(window), scale,
         out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(),
         _word(status, dev))
    out = _result(out, target, host)
    return (out, _result(lse, None, host)) if return_lse else out
