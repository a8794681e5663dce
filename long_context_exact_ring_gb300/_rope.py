"""Binding of the norm and rotation of queries and keys: argument marshalling
only, as in _paged.py, and the frequencies, which are made once on the host."""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import _new, load_library
from ._paged import _DTYPES, _I32, _call, _elems, _first, _pool_shape, _refuse, _typed, _whole

_LL3 = ctypes.c_longlong * 3
_F32 = torch.float32


def rope_inv_freq(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                  original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                  device="cuda"):
    """The frequencies base^(-2i / rot_dim) of a rotation of rot_dim elements,
    scaled for contexts `factor` times as long as those of training.  Returns
    (inv_freq [rot_dim / 2] fp32, amplitude).

    scaling  None      as they are
             "linear"  divided by factor
             "base"    the base raised by factor^(rot_dim / (rot_dim - 2)), so
                       that the slowest is divided by factor and the fastest stays
             "parts"   (YaRN, arXiv 2309.00071) those with fewer than
                       beta_slow turns over original_length are divided by
                       factor, those with more than beta_fast stay, between
                       them a mixture, linear in the turns as the paper has
                       it; the amplitude is 0.1 ln(factor) + 1.  Many models
                       of that name are trained with a mixture linear in the
                       pair's index instead, whose frequencies differ by up
                       to a factor of several: for those pass their own
                       inv_freq, which may be any tensor"""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be a positive even number, got {rot_dim}")
    if not (base > 1.0 and math.isfinite(base) and factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1, both finite")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs a rot_dim of at least 4")
        base *= factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    amplitude = 1.0
    if scaling == "linear":
        freq = [x / factor for x in freq]
    elif scaling == "parts":
        if original_length is None or original_length < 1 or not beta_fast > beta_slow:
            raise ValueError("scaling 'parts' needs original_length, and beta_fast above beta_slow")

        def kept(x):
            return min(1.0, max(0.0, (original_length * x / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)))
        freq = [x / factor * (1.0 - kept(x)) + x * kept(x) for x in freq]
        amplitude = 0.1 * math.log(factor) + 1.0
    return torch.tensor(freq, dtype=torch.float64).to(_F32).to(device), amplitude


def _rows(t, name, dtype, shape, device):
    """As _elems, for [B, heads, S, d]: (batch, head, position) strides."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape):
        _refuse(t, name, dtype, shape, device, True)
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[3] != 1:
        _refuse(t, name, dtype, shape, device, True)
    return t.data_ptr(), _LL3(st[0], st[1], st[2])


def _output(t, like, at, stream, name, dtype, device):
    """An output of the layout of `like`, which was checked: the tensor, its
    address and strides.  What is made here needs no check."""
    if t is not None:
        return (t, *_rows(t, name, dtype, like.shape, device))
    t = _new(stream, like)
    if at[1] is None:
        return t, t.data_ptr(), None
    st = t.stride()
    return t, t.data_ptr(), _LL3(st[0], st[1], st[2])


def _optional(t, name, shape, device):
    return None if t is None else _whole(t, name, _F32, shape, device)


def _freq(t, device):
    _first(t, "inv_freq", 1)
    return _whole(t, "inv_freq", _F32, t.shape, device), 2 * t.shape[0]


def _places(positions, B, S, device):
    """Address of positions [S] or [B, S], and which of the two."""
    per_batch = isinstance(positions, torch.Tensor) and positions.dim() == 2
    return _whole(positions, "positions", _I32, (B, S) if per_batch else (S,), device), int(per_batch)


def _key_shape(q, k):
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [B, H_kv, S, d]")
    B, _, S, d = q.shape
    return (B, k.shape[1], S, d)


def qk_norm_rope_fwd(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False, amplitude: float = 1.0, q_out=None, k_out=None, stream=None):
    """q [B, H, S, d] and k [B, H_kv, S, d], bf16 or fp16, normed and rotated:
    (q_out, k_out), ready for ring_attn_fwd.

    A weight [d] fp32 norms that tensor's rows: x * weight / sqrt(mean(x^2) +
    eps).  The first 2 * len(inv_freq) elements (a multiple of 16) turn by
    positions * inv_freq, positions int32 [S] or [B, S]; pair i is (i, i +
    len(inv_freq)), or (2i, 2i + 1) if interleaved; amplitude multiplies what
    is turned (rope_inv_freq gives both).  All may be strided views whose
    d-element rows are contiguous; outputs default to the inputs' layouts.
    q_out may be q, k_out may be k."""
    dev = _first(q, "q", 4)
    dtype = _typed(q, "q")
    B, H, S, d = q.shape
    ks = _key_shape(q, k)
    q_at, k_at = _rows(q, "q", dtype, q.shape, dev), _rows(k, "k", dtype, ks, dev)
    freq, rot = _freq(inv_freq, dev)
    q_out, *q_out_at = _output(q_out, q, q_at, stream, "q_out", dtype, dev)
    k_out, *k_out_at = _output(k_out, k, k_at, stream, "k_out", dtype, dev)
    _call(dev, stream, "qk_norm_rope_fwd", load_library().qk_norm_rope_fwd, *q_at, *k_at,
          _optional(q_weight, "q_weight", (d,), dev), _optional(k_weight, "k_weight", (d,), dev), float(eps),
          *_places(positions, B, S, dev), freq, rot, int(bool(interleaved)), float(amplitude),
          *q_out_at, *k_out_at, _DTYPES[dtype], B, H, ks[1], S, d)
    return q_out, k_out


@functools.lru_cache(maxsize=16)
def qk_norm_rope_bwd_workspace_size(d: int) -> int:
    return int(load_library().qk_norm_rope_bwd_workspace_size(d))


def qk_norm_rope_bwd(dq, dk, q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False, amplitude: float = 1.0, dq_in=None, dk_in=None, dq_weight=None,
                     dk_weight=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd's q, k and weights from those of its
    outputs: (dq_in, dk_in, dq_weight, dk_weight), the last two [d] fp32, or
    None where there is no weight.  dq_in and dk_in default to the layouts of q
    and k, and may be dq and dk.  q (k) gives the shapes; without its weight its
    values are not read, so that any tensor of its shape, dq (dk) itself too,
    will do.  The same call gives the same bits."""
    dev = _first(q, "q", 4)
    dtype = _typed(q, "q")
    B, H, S, d = q.shape
    ks = _key_shape(q, k)
    q_at, k_at = _rows(q, "q", dtype, q.shape, dev), _rows(k, "k", dtype, ks, dev)
    freq, rot = _freq(inv_freq, dev)
    dq_in, *dq_in_at = _output(dq_in, q, q_at, stream, "dq_in", dtype, dev)
    dk_in, *dk_in_at = _output(dk_in, k, k_at, stream, "dk_in", dtype, dev)
    for w, g, name in ((q_weight, dq_weight, "q_weight"), (k_weight, dk_weight, "k_weight")):
        if w is None and g is not None:
            raise ValueError(f"d{name} needs {name}")
    if q_weight is not None and dq_weight is None:
        dq_weight = _new(stream, q, (d,), _F32)
    if k_weight is not None and dk_weight is None:
        dk_weight = _new(stream, q, (d,), _F32)
    ws_at, ws_bytes = None, 0
    if q_weight is not None or k_weight is not None:
        if workspace is None:
            ws_bytes = qk_norm_rope_bwd_workspace_size(d)
            workspace = _new(stream, q, (max(ws_bytes, 1),), torch.uint8)
            ws_at = workspace.data_ptr()
        else:
            ws_at = _whole(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev)
            ws_bytes = workspace.numel()
    _call(dev, stream, "qk_norm_rope_bwd", load_library().qk_norm_rope_bwd, *_rows(dq, "dq", dtype, q.shape, dev),
          *_rows(dk, "dk", dtype, ks, dev), *q_at, *k_at, _optional(q_weight, "q_weight", (d,), dev),
          _optional(k_weight, "k_weight", (d,), dev), float(eps), *_places(positions, B, S, dev), freq, rot,
          int(bool(interleaved)), float(amplitude), *dq_in_at, *dk_in_at,
          _optional(dq_weight, "dq_weight", (d,), dev), _optional(dk_weight, "dk_weight", (d,), dev), _DTYPES[dtype],
          B, H, ks[1], S, d, ws_at, ws_bytes)
    return dq_in, dk_in, dq_weight, dk_weight


def paged_kv_append_rope(q, k, v, k_cache, v_cache, slots, seq_lens, cu_q, inv_freq, *, q_weight=None, k_weight=None,
                         eps: float = 1e-6, interleaved: bool = False, amplitude: float = 1.0, q_out=None,
                         stream=None):
    """A step's new tokens, normed and rotated as by qk_norm_rope_fwd, in one
    launch: q [tokens, H, d] to q_out, k [tokens, H_kv, d] to its slots of the
    pool k_cache, v as it is to v_cache (as paged_kv_append).

    slots [tokens], seq_lens [n] and cu_q [n + 1] are what paged_kv_plan
    returns: token t of request i stands at position seq_lens[i] - cu_q[i + 1]
    + t.  Tokens of no request are left out, q_out's rows too.  q_out has q's
    layout by default and may be q.  Returns (q_out, k_cache, v_cache)."""
    dev = _first(q, "q", 3)
    dtype = _typed(q, "q")
    T, H, d = q.shape
    num_pages, page_size, H_kv = _pool_shape(k_cache)[:3]
    pool, rows = (num_pages, page_size, H_kv, d), (T, H_kv, d)
    _first(seq_lens, "seq_lens", 1)
    n = seq_lens.shape[0]
    q_at = _elems(q, "q", dtype, q.shape, dev)
    q_out = _new(stream, q) if q_out is None else q_out
    freq, rot = _freq(inv_freq, dev)
    _call(dev, stream, "paged_kv_append_rope", load_library().paged_kv_append_rope, *q_at,
          *_elems(k, "k", dtype, rows, dev), *_elems(v, "v", dtype, rows, dev),
          _optional(q_weight, "q_weight", (d,), dev), _optional(k_weight, "k_weight", (d,), dev), float(eps), freq,
          rot, int(bool(interleaved)), float(amplitude), *_elems(q_out, "q_out", dtype, q.shape, dev),
          *_elems(k_cache, "k_cache", dtype, pool, dev), *_elems(v_cache, "v_cache", dtype, pool, dev),
          _whole(slots, "slots", _I32, (T,), dev), _whole(seq_lens, "seq_lens", _I32, (n,), dev),
          _whole(cu_q, "cu_q", _I32, (n + 1,), dev), _DTYPES[dtype], n, T, H, H_kv, d, num_pages, page_size)
    return q_out, k_cache, v_cache
