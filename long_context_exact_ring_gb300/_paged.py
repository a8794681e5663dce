"""Binding of the paged key/value cache calls: argument marshalling only, as
in _binding.py, for tensors of any device (the call runs on the device of its
tensors, on that device's current stream unless ``stream``, a torch stream or a
handle, names one: the caller orders it behind what writes the inputs, and what
reads the results behind it)."""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import _check, _new, load_library

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_LL2, _LL3 = ctypes.c_longlong * 2, ctypes.c_longlong * 3
_I32 = torch.int32
# A stream's handle without a Stream object; absent from a torch without CUDA.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(t, name, dtype, shape, device, rows):
    """Says what is wrong with an argument that failed its check."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must have contiguous {'d-element rows' if rows else 'rows'}"
                     if t.dim() > 1 else f"{name} must be contiguous")


def _whole(t, name, dtype, shape, device):
    """A contiguous tensor; its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape
            and t.is_contiguous()):
        _refuse(t, name, dtype, shape, device, False)
    return t.data_ptr()


def _elems(t, name, dtype, shape, device):
    """A tensor of d-element rows placed by any strides: its address and the C
    array of the other dimensions' strides, None where it is contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape):
        _refuse(t, name, dtype, shape, device, True)
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[-1] != 1:
        _refuse(t, name, dtype, shape, device, True)
    return t.data_ptr(), (_LL2(st[0], st[1]) if len(st) == 3 else _LL3(st[0], st[1], st[2]))


def _first(t, name, dim):
    """Type and rank of the tensor that the other arguments are checked against;
    its device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, has {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _table(t, device):
    """[n, max_pages] with contiguous rows: address, n, max_pages, row stride."""
    _first(t, "block_table", 2)
    n, max_pages = t.shape
    if t.dtype is not _I32 or t.get_device() != device or (max_pages > 1 and t.stride(1) != 1):
        _refuse(t, "block_table", _I32, t.shape, device, False)
    return t.data_ptr(), n, max_pages, t.stride(0) if n > 1 else max_pages


def _typed(t, name):
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return t.dtype


def _pool_shape(k_cache):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, H_kv, d]")
    return tuple(k_cache.shape)


def _call(device, stream, what, fn, *args):
    """fn(*args, stream) with `device` current."""
    if stream is None:
        handle = _current_stream(device)
    else:
        handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if _current_device() == device:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc:
        _check(rc, what)


def paged_kv_plan(seq_lens, new_lens, block_table, free_list, counts, page_size: int, tokens: int, *,
                  seq_lens_out=None, cu_q=None, slots=None, counts_out=None, stream=None):
    """The bookkeeping of one step of a paged key/value cache, on the GPU.

    seq_lens, new_lens [n]; block_table [n, max_pages]; free_list
    [num_pages], a stack whose first counts[0] entries are free; all int32.
    new_lens[i] tokens are added to request i (a negative value ends it);
    pages go from the stack into block_table, and back, in place.  Returns
    (seq_lens_out [n], cu_q [n + 1], slots [tokens], counts_out [2]):
    the lengths after the step, where each request's new tokens start, the
    slot of every new token (-1: none) and {free pages, requests not
    granted}.  seq_lens_out may be seq_lens and counts_out may be counts."""
    dev = _first(block_table, "block_table", 2)
    table, n, max_pages, stride = _table(block_table, dev)
    _first(free_list, "free_list", 1)
    pages = free_list.shape[0]
    tokens, page_size = int(tokens), int(page_size)
    if not 0 <= tokens < 2 ** 31 or abs(page_size) >= 2 ** 31:
        raise ValueError("tokens and page_size must be 32-bit integers, tokens not negative")
    shapes = ((n,), (n + 1,), (tokens,), (2,))
    out = tuple(_new(stream, block_table, shape, _I32) if t is None else t
                for t, shape in zip((seq_lens_out, cu_q, slots, counts_out), shapes))
    seq_lens_out, cu_q, slots, counts_out = out
    _call(dev, stream, "paged_kv_plan", load_library().paged_kv_plan,
          _whole(seq_lens, "seq_lens", _I32, (n,), dev), _whole(new_lens, "new_lens", _I32, (n,), dev), n, table,
          stride, max_pages, _whole(free_list, "free_list", _I32, (pages,), dev), pages,
          _whole(counts, "counts", _I32, (2,), dev), page_size, tokens,
          _whole(seq_lens_out, "seq_lens_out", _I32, (n,), dev), _whole(cu_q, "cu_q", _I32, (n + 1,), dev),
          _whole(slots, "slots", _I32, (tokens,), dev), _whole(counts_out, "counts_out", _I32, (2,), dev))
    return out


def paged_kv_append(k, v, k_cache, v_cache, slots, *, stream=None):
    """The new tokens' K and V rows, [tokens, H_kv, d] bf16 or fp16, into the
    pools [num_pages, page_size, H_kv, d], at slots [tokens] int32 (-1: the
    row is skipped).  All may be strided views whose d-element rows are
    contiguous; [num_pages, H_kv, page_size, d] storage is
    ``pool.transpose(1, 2)``.  Returns (k_cache, v_cache)."""
    dev = _first(k, "k", 3)
    dtype = _typed(k, "k")
    shape = k.shape
    T, H_kv, d = shape
    num_pages, page_size = _pool_shape(k_cache)[:2]
    pool = (num_pages, page_size, H_kv, d)
    _call(dev, stream, "paged_kv_append", load_library().paged_kv_append,
          *_elems(k, "k", dtype, shape, dev), *_elems(v, "v", dtype, shape, dev),
          *_elems(k_cache, "k_cache", dtype, pool, dev), *_elems(v_cache, "v_cache", dtype, pool, dev),
          _whole(slots, "slots", _I32, (T,), dev), T, H_kv, d, num_pages, page_size)
    return k_cache, v_cache


@functools.lru_cache(maxsize=256)
def paged_attn_workspace_size(n: int, tokens: int, H: int, H_kv: int, d: int) -> int:
    return int(load_library().paged_attn_workspace_size(n, tokens, H, H_kv, d))


def paged_attn_fwd(q, k_cache, v_cache, block_table, seq_lens, cu_q, causal: bool, scale: float | None = None, *,
                   max_q: int | None = None, o=None, lse=None, workspace=None, stream=None):
    """O, LSE of new tokens over their requests' paged contexts.

    q [tokens, H, d] bf16 or fp16 holds the new tokens of n requests one
    after the other, request i's in rows cu_q[i] .. cu_q[i + 1]; its context
    is the first seq_lens[i] keys of the pages block_table[i], the new ones
    last.  Pools as in paged_kv_append, H_kv of their heads for H query heads
    (query head h reads key/value head h // (H / H_kv)); causal lets a token
    see the keys up to its own.  O [tokens, H, d] has q's layout by default,
    LSE is [H, tokens] fp32 (natural log).  max_q, an upper bound of the new
    tokens of one request, only guides the choice of kernels: pass it where
    it is known, 1 for a decode step."""
    dev = _first(q, "q", 3)
    dtype = _typed(q, "q")
    shape = q.shape
    T, H, d = shape
    num_pages, page_size, H_kv, _ = _pool_shape(k_cache)
    if H_kv < 1 or H % H_kv:
        raise ValueError(f"query heads ({H}) must be a multiple of key/value heads ({H_kv})")
    pool = (num_pages, page_size, H_kv, d)
    table, n, max_pages, stride = _table(block_table, dev)
    lib = load_library()
    # what is made here needs no check
    q_at = _elems(q, "q", dtype, shape, dev)
    if o is None:
        o = _new(stream, q)
        o_at = (o.data_ptr(), q_at[1] and _LL2(o.stride(0), o.stride(1)))
    else:
        o_at = _elems(o, "o", dtype, shape, dev)
    if lse is None:
        lse = _new(stream, q, (H, T), torch.float32)
        lse_at = lse.data_ptr()
    else:
        lse_at = _whole(lse, "lse", torch.float32, (H, T), dev)
    if workspace is None:
        ws_bytes = paged_attn_workspace_size(n, T, H, H_kv, d)
        workspace = _new(stream, q, (max(ws_bytes, 1),), torch.uint8)
        ws_at = workspace.data_ptr()
    else:
        ws_at = _whole(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev)
        ws_bytes = workspace.numel()
    _call(dev, stream, "paged_attn_fwd", lib.paged_attn_fwd, *q_at,
          *_elems(k_cache, "k_cache", dtype, pool, dev), *_elems(v_cache, "v_cache", dtype, pool, dev), table, stride,
          _whole(seq_lens, "seq_lens", _I32, (n,), dev), _whole(cu_q, "cu_q", _I32, (n + 1,), dev), *o_at, lse_at,
          _DTYPES[dtype], n, T, H, H_kv, d, num_pages, page_size, max_pages, T if max_q is None else min(T, int(max_q)),
          int(bool(causal)), 1.0 / math.sqrt(d) if scale is None else float(scale), ws_at, ws_bytes)
    return o, lse
