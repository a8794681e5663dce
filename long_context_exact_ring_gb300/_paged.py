"""Binding of the paged key/value cache calls: argument marshalling only, as
in _binding.py, for tensors of any device (the call runs on the device of its
tensors, on that device's current stream unless ``stream`` names one)."""
from __future__ import annotations

import ctypes
import math

import torch

from ._binding import _check, load_library

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_LL2, _LL3 = ctypes.c_longlong * 2, ctypes.c_longlong * 3


def _ints(t, name, shape, device):
    """An int32 CUDA tensor of the given shape, its last dimension contiguous
    (a 1-D one wholly)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    _where(t, name, device)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


def _where(t, name, device):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _elems(t, name, dtype, shape, device):
    """A tensor of d-element rows placed by any strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _where(t, name, device)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.stride(-1) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must have contiguous d-element rows")
    return t


def _first(t, name, dim):
    """Type and rank of the tensor that the other arguments are checked against."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, has {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _pool(k_cache, v_cache, dtype, H_kv, d, device):
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, H_kv, d]")
    shape = (k_cache.shape[0], k_cache.shape[1], H_kv, d)
    _elems(k_cache, "k_cache", dtype, shape, device)
    _elems(v_cache, "v_cache", dtype, shape, device)
    return shape[0], shape[1]


def _call(device, stream, own, what, fn, *args):
    """fn(*args, stream) with `device` current.  `own` are tensors made for
    this call: on a stream that is not the one they were allocated on, their
    memory must outlive the call there."""
    if stream is None:
        handle = torch.cuda.current_stream(device).cuda_stream
    else:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        handle = stream.cuda_stream
        for t in own:
            t.record_stream(stream)
    if torch.cuda.current_device() == device.index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
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
    n, max_pages = block_table.shape
    _ints(block_table, "block_table", (n, max_pages), dev)
    _ints(seq_lens, "seq_lens", (n,), dev)
    _ints(new_lens, "new_lens", (n,), dev)
    _first(free_list, "free_list", 1)
    _ints(free_list, "free_list", (free_list.shape[0],), dev)
    _ints(counts, "counts", (2,), dev)
    tokens = int(tokens)

    def out(t, name, shape):
        if t is None:
            return torch.empty(shape, dtype=torch.int32, device=dev)
        return _ints(t, name, shape, dev)

    if tokens < 0:
        raise ValueError("tokens must not be negative")
    own = [x for x in (seq_lens_out, cu_q, slots, counts_out)]
    seq_lens_out = out(seq_lens_out, "seq_lens_out", (n,))
    cu_q = out(cu_q, "cu_q", (n + 1,))
    slots = out(slots, "slots", (tokens,))
    counts_out = out(counts_out, "counts_out", (2,))
    results = (seq_lens_out, cu_q, slots, counts_out)
    own = [r for r, given in zip(results, own) if given is None]
    stride = block_table.stride(0) if n > 1 else max_pages
    _call(dev, stream, own, "paged_kv_plan", load_library().paged_kv_plan, seq_lens.data_ptr(), new_lens.data_ptr(),
          n, block_table.data_ptr(), stride, max_pages, free_list.data_ptr(), free_list.shape[0], counts.data_ptr(),
          int(page_size), tokens, seq_lens_out.data_ptr(), cu_q.data_ptr(), slots.data_ptr(), counts_out.data_ptr())
    return results


def paged_kv_append(k, v, k_cache, v_cache, slots, *, stream=None):
    """The new tokens' K and V rows, [tokens, H_kv, d] bf16 or fp16, into the
    pools [num_pages, page_size, H_kv, d], at slots [tokens] int32 (-1: the
    row is skipped).  All may be strided views whose d-element rows are
    contiguous; [num_pages, H_kv, page_size, d] storage is
    ``pool.transpose(1, 2)``.  Returns (k_cache, v_cache)."""
    dev = _first(k, "k", 3)
    dtype = k.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"k must be torch.bfloat16 or torch.float16, got {dtype}")
    T, H_kv, d = k.shape
    _elems(k, "k", dtype, (T, H_kv, d), dev)
    _elems(v, "v", dtype, (T, H_kv, d), dev)
    num_pages, page_size = _pool(k_cache, v_cache, dtype, H_kv, d, dev)
    _ints(slots, "slots", (T,), dev)
    _call(dev, stream, (), "paged_kv_append", load_library().paged_kv_append, k.data_ptr(), _LL2(*k.stride()[:2]),
          v.data_ptr(), _LL2(*v.stride()[:2]), k_cache.data_ptr(), _LL3(*k_cache.stride()[:3]), v_cache.data_ptr(),
          _LL3(*v_cache.stride()[:3]), slots.data_ptr(), T, H_kv, d, num_pages, page_size)
    return k_cache, v_cache


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
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"q must be torch.bfloat16 or torch.float16, got {dtype}")
    T, H, d = q.shape
    _elems(q, "q", dtype, (T, H, d), dev)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, H_kv, d]")
    H_kv = k_cache.shape[2]
    if H_kv < 1 or H % H_kv:
        raise ValueError(f"query heads ({H}) must be a multiple of key/value heads ({H_kv})")
    num_pages, page_size = _pool(k_cache, v_cache, dtype, H_kv, d, dev)
    _first(block_table, "block_table", 2)
    n, max_pages = block_table.shape
    _ints(block_table, "block_table", (n, max_pages), dev)
    _ints(seq_lens, "seq_lens", (n,), dev)
    _ints(cu_q, "cu_q", (n + 1,), dev)
    own = []
    if o is None:
        o = torch.empty_like(q)
        own.append(o)
    else:
        _elems(o, "o", dtype, (T, H, d), dev)
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=dev)
        own.append(lse)
    elif not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32:
        raise TypeError("lse must be a torch.float32 tensor")
    else:
        _where(lse, "lse", dev)
        if tuple(lse.shape) != (H, T) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous {(H, T)}, has shape {tuple(lse.shape)}")
    lib = load_library()
    if workspace is None:
        need = lib.paged_attn_workspace_size(n, T, H, H_kv, d)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        own.append(workspace)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a torch.uint8 tensor")
    else:
        _where(workspace, "workspace", dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    stride = block_table.stride(0) if n > 1 else max_pages
    _call(dev, stream, own, "paged_attn_fwd", lib.paged_attn_fwd, q.data_ptr(), _LL2(*q.stride()[:2]),
          k_cache.data_ptr(), _LL3(*k_cache.stride()[:3]), v_cache.data_ptr(), _LL3(*v_cache.stride()[:3]),
          block_table.data_ptr(), stride, seq_lens.data_ptr(), cu_q.data_ptr(), o.data_ptr(), _LL2(*o.stride()[:2]),
          lse.data_ptr(), _DTYPES[dtype], n, T, H, H_kv, d, num_pages, page_size, max_pages,
          T if max_q is None else int(max_q), int(bool(causal)), 1.0 / math.sqrt(d) if scale is None else float(scale),
          workspace.data_ptr(), workspace.numel())
    return o, lse
