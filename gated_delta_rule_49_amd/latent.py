"""The layer of full attention that a hybrid model runs beside its recurrent
ones: latent attention, its positions and its paged cache (C ABI in
``include/kda.h``).  Like the rest of the binding these functions only check
and marshal torch tensors, allocate outputs and workspaces with torch, and
launch on torch's current stream of the tensors' device.

``rotary_frequencies``  the frequencies of rotary positions, scaled for long contexts
``rotary`` / ``rotary_backward``  rotary positions on part of each head
``latent_append``   new tokens' rows into the paged cache (norm, rotation, write)
``latent_prefill`` / ``latent_backward``  the expanded form and its gradients
``latent_decode``   the absorbed form over the cache, for a few tokens
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (KDAError, LatentAppendArgs, LatentBackwardArgs, LatentDecodeArgs, LatentPrefillArgs, RotaryArgs, _check_buffer, _dt, lib)
from .sublayer import _p, _run, _workspace

_F32 = (torch.float32,)
_F64 = (torch.float64,)
_I32 = (torch.int32,)
_FLOATS = (torch.float32, torch.bfloat16)


def _device(*ts):
    """The GPU that all tensors given are on."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if dev is None:
            dev = t.device
            if dev.type != "cuda":
                raise ValueError("all tensors must be on the GPU (no CPU path exists)")
        elif t.device != dev:
            raise ValueError("tensors are on different devices" if t.is_cuda else "all tensors must be on the GPU (no CPU path exists)")
    return dev


def _dense(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _lead_strides(t, name):
    """Strides of all axes but the last, which must be contiguous; 0 for an axis of one."""
    n, s = t.shape, t.stride()
    if 0 in n:
        return (0,) * (len(n) - 1)
    if s[-1] != 1 and n[-1] > 1:
        raise ValueError(f"{name}: channels must be contiguous")
    return tuple(a if b > 1 else 0 for a, b in zip(s[:-1], n)) if 1 in n else s[:-1]


# -------------------------------------------------------------------- rotary
def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=4096, fast_turns=32.0, slow_turns=1.0, device=None):
    """(frequencies float64 [rotary_dim/2] in radians per position, magnitude)
    for ``rotary`` and ``latent_append``: f_i = base^(-2i / rotary_dim), for
    contexts ``factor`` times the ``original_length`` scaled by

    None       not at all
    "linear"   f_i / factor: positions squeezed into the original range
    "base"     a base of base * factor^(d / (d - 2)): the slowest pair turns
               ``factor`` times slower, the fastest as before
    "turns"    pair by pair, by the turns it makes over the original length:
               those of ``fast_turns`` or more stay, those of ``slow_turns`` or
               fewer are divided by factor, between them linearly in the turns;
               the magnitude is then 1 + 0.1 ln(factor)"""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not factor >= 1:
        raise ValueError("factor must be at least 1")
    at = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    magnitude = 1.0
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError('scaling "base" needs a rotary_dim of 4 or more')
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** -at
    if scaling == "linear":
        f = f / factor
    elif scaling == "turns":
        if not fast_turns > slow_turns:
            raise ValueError("fast_turns must be above slow_turns")
        keep = ((original_length * f / (2 * math.pi) - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        magnitude = 1.0 + 0.1 * math.log(factor)
    elif scaling not in (None, "base"):
        raise ValueError(f'scaling must be None, "linear", "base" or "turns", got {scaling!r}')
    return f.to(device), magnitude


def _rotary(fn, what, x, freqs, positions, offset, interleaved, magnitude, out):
    dev = _device(x, freqs, positions, out)
    _dense(freqs)
    if x.dim() != 4:
        raise ValueError("x must be [B,T,H,D]")
    B, T, H, D = x.shape
    if freqs.dim() != 1:
        raise ValueError("freqs must be float64 [rotary_dim/2]")
    _check_buffer(freqs, "freqs", freqs.shape, _F64)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check_buffer(out, "out", x.shape, (x.dtype,))
    a = RotaryArgs(B=B, T=T, H=H, D=D, rotary_dim=2 * freqs.numel(), offset=offset, interleaved=1 if interleaved else 0, dtype=_dt(x.dtype),
                   magnitude=magnitude, x=_p(x), positions=_p(positions), freqs=_p(freqs), out=_p(out))
    a.x_stride_b, a.x_stride_t, a.x_stride_h = _lead_strides(x, "x")
    a.out_stride_b, a.out_stride_t, a.out_stride_h = _lead_strides(out, "out")
    if positions is not None:
        if positions.dtype != torch.int32 or tuple(positions.shape) not in ((T,), (B, T)):
            raise ValueError(f"positions must be int32 [{T}] or [{B},{T}]")
        a.pos_stride_t = positions.stride(-1) if T > 1 else 0
        a.pos_stride_b = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    _run(fn, a, dev, what)
    return out


def rotary(x, freqs, positions=None, offset=0, interleaved=False, magnitude=1.0, out=None):
    """Rotary positions on the channels [offset, offset + 2 len(freqs)) of each
    head of x [B,T,H,D] (float32 or bfloat16, channels contiguous, any other
    strides); the other channels are copied.  Pairs are neighbours
    (``interleaved``) or half the rotated part apart; each is turned by
    position * frequency and multiplied by ``magnitude``.  ``freqs`` float64 as
    from ``rotary_frequencies``; ``positions`` int32 [T] or [B,T] (None: 0 ..
    T-1 in every row).  ``out`` may be x itself (then only the rotated part is
    touched); another overlap is refused.  Returns out."""
    return _rotary(lib().kda_rotary, "kda_rotary", x, freqs, positions, offset, interleaved, magnitude, out)


def rotary_backward(d_out, freqs, positions=None, offset=0, interleaved=False, magnitude=1.0, out=None):
    """The gradient of ``rotary`` with the same arguments with respect to x,
    from d_out [B,T,H,D]: every pair turned back, with the same magnitude."""
    return _rotary(lib().kda_rotary_backward, "kda_rotary_backward", d_out, freqs, positions, offset, interleaved, magnitude, out)


# --------------------------------------------------------------------- cache
def _pages(a, cache, page_table, num_seqs, d, dtype):
    """The cache's and the table's fields, checked."""
    if cache.dim() != 3 or cache.shape[2] != d:
        raise ValueError(f"cache must be [pages,page_size,{d}]")
    if cache.dtype != dtype:
        raise TypeError(f"cache must be {dtype}, got {cache.dtype}")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != num_seqs:
        raise ValueError(f"page_table must be int32 [{num_seqs},max_pages]")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table: a sequence's entries must be contiguous")
    a.num_pages, a.page_size, a.max_pages = cache.shape[0], cache.shape[1], page_table.shape[1]
    a.page_stride, a.row_stride = _lead_strides(cache, "cache")
    a.table_stride = page_table.stride(0) if num_seqs > 1 else 0
    a.cache, a.page_table = _p(cache), _p(page_table)


def latent_append(kv, cache, page_table, lengths, d_latent, norm_weight=None, eps=1e-6, freqs=None, magnitude=1.0, interleaved=False, cu_seqlens=None,
                  output_rows=False, rows=None, device_status=None):
    """Writes new tokens into a paged latent cache.  kv [B,T,d_latent+d_rope]
    (float32 or bfloat16; tokens may be slices of wider ones) holds a latent
    vector and a position key each; token t of sequence n stands at position
    lengths[n] + t, and its row goes to page page_table[n, position //
    page_size] of ``cache`` [pages,page_size,d_latent+d_rope] (kv's dtype):
    the latent normed with ``norm_weight`` (float32 [d_latent]; None: as it
    is), the key turned with ``freqs`` (float64 [d_rope/2]; None: as it is).

    ``lengths`` int32 [N] (tokens in the cache already; not changed),
    ``page_table`` int32 [N,max_pages]; ``cu_seqlens`` (int32 [N+1], batch 1)
    packs N sequences along T; tokens before the first offset or behind the last
    are padding, for which nothing is written.  With ``output_rows``, or a buffer
    ``rows``, the rows are returned too, [B,T,d_latent+d_rope] (a prompt expands
    them; padding's are left as they were), else None.  A token without a page of its own (a position outside the table, an
    entry outside the cache) is left out; ``device_status`` (int32 [1] on the
    device) tells so.  Nothing synchronises."""
    dev = _device(kv, cache, page_table, lengths, norm_weight, freqs, cu_seqlens, rows, device_status)
    _dense(norm_weight, freqs, lengths, cu_seqlens, rows, device_status)
    if kv.dim() != 3:
        raise ValueError("kv must be [B,T,d_latent+d_rope]")
    B, T, d = kv.shape
    if not 0 < d_latent <= d:
        raise ValueError(f"d_latent must be in [1,{d}]")
    if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2):
        raise TypeError("cu_seqlens must be int32 [N+1]")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _check_buffer(lengths, "lengths", (N,), _I32)
    _check_buffer(norm_weight, "norm_weight", (d_latent,), _F32)
    _check_buffer(freqs, "freqs", ((d - d_latent) // 2,), _F64)
    _check_buffer(device_status, "device_status", (1,), _I32)
    _check_buffer(rows, "rows", (B, T, d), (kv.dtype,))
    if rows is None and output_rows:
        rows = torch.empty((B, T, d), dtype=kv.dtype, device=dev)
    a = LatentAppendArgs(B=B, T=T, num_seqs=N, d_latent=d_latent, d_rope=d - d_latent, interleaved=1 if interleaved else 0, dtype=_dt(kv.dtype), eps=eps,
                         magnitude=magnitude, kv=_p(kv), norm_weight=_p(norm_weight), freqs=_p(freqs), cu_seqlens=_p(cu_seqlens), lengths=_p(lengths),
                         rows=_p(rows), device_status=_p(device_status))
    a.kv_stride_b, a.kv_stride_t = _lead_strides(kv, "kv")
    _pages(a, cache, page_table, N, d, kv.dtype)
    _run(lib().kda_latent_append, a, dev, "kda_latent_append")
    return rows


# ------------------------------------------------------------------ expanded
def _latent_args(q, k_nope, k_rope, v, scale, causal, cu_q, cu_k, precise, *more):
    dev = _device(q, k_nope, k_rope, v, cu_q, cu_k, *more)
    _dense(cu_q, cu_k)
    if q.dim() != 4 or k_nope.dim() != 4 or v.dim() != 4 or (k_rope is not None and k_rope.dim() != 3):
        raise ValueError("q must be [B,T,H,d_nope+d_rope], k_nope [B,S,H,d_nope], k_rope [B,S,d_rope], v [B,S,H,d_v]")
    B, T, H, d = q.shape
    S, dn, dv = k_nope.shape[1], k_nope.shape[3], v.shape[3]
    dr = k_rope.shape[2] if k_rope is not None else 0
    if d != dn + dr or tuple(k_nope.shape) != (B, S, H, dn) or tuple(v.shape) != (B, S, H, dv) or (k_rope is not None and tuple(k_rope.shape) != (B, S, dr)):
        raise ValueError("q must be [B,T,H,d_nope+d_rope], k_nope [B,S,H,d_nope], k_rope [B,S,d_rope], v [B,S,H,d_v]")
    if any(t is not None and t.dtype != q.dtype for t in (k_nope, k_rope, v)):
        raise TypeError("q, k_nope, k_rope, v must share one dtype")
    if cu_k is not None and cu_q is None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    N = B
    if cu_q is not None:
        if cu_k is None:
            cu_k = cu_q
        for c in (cu_q, cu_k):
            if c.dtype != torch.int32 or c.dim() != 1 or c.numel() < 2:
                raise TypeError("cu_seqlens must be int32 [N+1]")
        if cu_k.shape != cu_q.shape:
            raise ValueError("cu_seqlens and cu_seqlens_k must have one length")
        N = cu_q.numel() - 1
    a = LatentPrefillArgs(B=B, T=T, S=S, H=H, d_nope=dn, d_rope=dr, d_v=dv, num_seqs=N, in_dtype=_dt(q.dtype), out_dtype=_dt(q.dtype),
                          causal=1 if causal else 0, precise=1 if precise else 0, scale=1 / math.sqrt(d) if scale is None else scale, q=_p(q), k_nope=_p(k_nope), k_rope=_p(k_rope), v=_p(v),
                          cu_seqlens_q=_p(cu_q), cu_seqlens_k=_p(cu_k))
    a.q_stride_b, a.q_stride_t, a.q_stride_h = _lead_strides(q, "q")
    a.k_stride_b, a.k_stride_t, a.k_stride_h = _lead_strides(k_nope, "k_nope")
    a.v_stride_b, a.v_stride_t, a.v_stride_h = _lead_strides(v, "v")
    if k_rope is not None:
        a.r_stride_b, a.r_stride_t = _lead_strides(k_rope, "k_rope")
    return a, dev, (B, T, S, H, dn, dr, dv)


def latent_prefill(q, k_nope, k_rope, v, scale=None, causal=True, cu_seqlens=None, cu_seqlens_k=None, out_dtype=None, o=None, lse=None, check_seqlens=True,
                   device_status=None, precise=False):
    """Latent attention in its expanded form over whole sequences.

    q [B,T,H,d_nope+d_rope], k_nope [B,S,H,d_nope], v [B,S,H,d_v], all float32
    or all bfloat16 (channels contiguous, other axes strided as they come: k_nope
    and v may be slices of one projection), and k_rope [B,S,d_rope], shared by
    the heads (None without one).  The queries stand at the end of the keys: with
    ``causal`` query i sees keys up to i + S - T.  ``scale`` multiplies the
    scores (None: 1 / sqrt(d_nope + d_rope)).  ``cu_seqlens`` (int32 [N+1], batch
    1) packs N sequences' queries along T, ``cu_seqlens_k`` their keys along S
    (None: the same offsets).

    Returns (o [B,T,H,d_v] of out_dtype, default q's; lse float32 [B,T,H], the
    log of the sum of exponentials).  A query without a key has o = 0 and lse =
    -inf.  ``o`` and ``lse`` are optional preallocated buffers;
    ``check_seqlens`` and ``device_status`` as for ``prefill``.

    With bfloat16 inputs the probabilities are rounded to bfloat16 for their
    product with v (a float32 o is the bfloat16 one before its own rounding);
    with ``precise`` they enter it in two parts, exact to 2^-16, which takes about
    a third longer.  float32 inputs are computed in float32 throughout."""
    a, dev, (B, T, S, H, dn, dr, dv) = _latent_args(q, k_nope, k_rope, v, scale, causal, cu_seqlens, cu_seqlens_k, precise, o, lse, device_status)
    _dense(o, lse, device_status)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype or q.dtype, device=dev)
    else:
        _check_buffer(o, "o", (B, T, H, dv), _FLOATS)
        if out_dtype is not None and out_dtype != o.dtype:
            raise TypeError(f"out_dtype {out_dtype} disagrees with o.dtype {o.dtype}")
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    else:
        _check_buffer(lse, "lse", (B, T, H), _F32)
    _check_buffer(device_status, "device_status", (1,), _I32)
    check = check_seqlens and cu_seqlens is not None and device_status is None
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else device_status
    a.out_dtype, a.o, a.lse, a.device_status = _dt(o.dtype), _p(o), _p(lse), _p(status)
    L = lib()
    need = int(L.kda_latent_prefill_workspace_bytes(ctypes.byref(a)))
    if need == 0:
        raise KDAError(L.kda_latent_prefill(ctypes.byref(a), None), "kda_latent_prefill")  # reports why
    ws = _workspace(need, dev)
    a.workspace, a.workspace_bytes = _p(ws), need
    _run(L.kda_latent_prefill, a, dev, "kda_latent_prefill")
    if check and int(status.item()) != 0:
        raise KDAError(int(status.item()), "kda_latent_prefill (device check)")
    return o, lse


def latent_backward(q, k_nope, k_rope, v, o, lse, d_o, scale=None, causal=True, cu_seqlens=None, cu_seqlens_k=None, device_status=None, precise=False):
    """Gradients of ``latent_prefill`` with the same arguments, from d_o (like
    o, q's dtype) and the forward's o and lse (all three strided as they come,
    channels contiguous): (dq, dk_nope, dk_rope, dv),
    contiguous, q's dtype, dk_rope summed over the heads that share it (None
    without one).  o may be float32 with bfloat16 inputs (the forward's
    ``out_dtype``): the gradients of scores are differences with rowsum(d_o o),
    into which a rounded o brings its rounding.  The probabilities and the scores'
    gradients are rounded to bfloat16 for their products, or with ``precise`` enter
    them in two parts, as in the forward.  Nothing synchronises; ``device_status`` (int32 [1] on the
    device) receives the call's device-side status: with malformed offsets the
    gradients are not written."""
    a, dev, (B, T, S, H, dn, dr, dv) = _latent_args(q, k_nope, k_rope, v, scale, causal, cu_seqlens, cu_seqlens_k, precise, o, lse, d_o, device_status)
    _dense(device_status)
    _check_buffer(o, "o", (B, T, H, dv), _FLOATS)
    _check_buffer(d_o, "d_o", (B, T, H, dv), (q.dtype,))
    _check_buffer(lse, "lse", (B, T, H), _F32)
    _check_buffer(device_status, "device_status", (1,), _I32)
    a.out_dtype, a.o, a.lse, a.device_status = _dt(o.dtype), _p(o), _p(lse), _p(device_status)
    like = dict(dtype=q.dtype, device=dev)
    dq, dk_nope, d_v = torch.empty((B, T, H, dn + dr), **like), torch.empty((B, S, H, dn), **like), torch.empty((B, S, H, dv), **like)
    dk_rope = torch.empty((B, S, dr), **like) if k_rope is not None else None
    g = LatentBackwardArgs(f=a, d_o=_p(d_o), dq=_p(dq), dk_nope=_p(dk_nope), dk_rope=_p(dk_rope), dv=_p(d_v))
    g.o_stride_b, g.o_stride_t, g.o_stride_h = _lead_strides(o, "o")
    g.d_o_stride_b, g.d_o_stride_t, g.d_o_stride_h = _lead_strides(d_o, "d_o")
    g.lse_stride_b, g.lse_stride_t, g.lse_stride_h = _lead_strides(lse[..., None], "lse")
    L = lib()
    need = int(L.kda_latent_backward_workspace_bytes(ctypes.byref(g)))
    if need == 0:
        raise KDAError(L.kda_latent_backward(ctypes.byref(g), None), "kda_latent_backward")
    ws = _workspace(need, dev)
    g.workspace, g.workspace_bytes = _p(ws), need
    _run(L.kda_latent_backward, g, dev, "kda_latent_backward")
    return dq, dk_nope, dk_rope, d_v


# ------------------------------------------------------------------ absorbed
def latent_decode(q, cache, page_table, lengths, d_latent, scale, out_dtype=None, o=None, lse=None, device_status=None):
    """Latent attention in its absorbed form over a paged cache, for a few
    tokens of each of B sequences.

    q [B,m,H,d_latent+d_rope] (float32 or bfloat16) lives in the latent space
    (the keys' up-projection absorbed); a row of ``cache``
    [pages,page_size,d_latent+d_rope] (q's dtype, as ``latent_append`` writes
    it) is the key of every head, its first d_latent channels the value.
    ``lengths`` int32 [B] counts each sequence's rows, its m tokens among them:
    token j sees the rows before lengths - m + 1 + j.  ``page_table`` int32
    [B,max_pages].  ``scale`` is that of the expanded form.

    Returns (o [B,m,H,d_latent] of out_dtype, default q's, still latent; lse
    float32 [B,m,H]).  With bfloat16 inputs the probabilities enter their product
    with the values in two parts, exact to 2^-16.  An empty slot (length 0) has o = 0 and lse = -inf.
    Nothing synchronises; ``device_status`` (int32 [1] on the device) tells of
    pages or lengths outside the cache, whose sequences' results are undefined."""
    dev = _device(q, cache, page_table, lengths, o, lse, device_status)
    _dense(lengths, o, lse, device_status)
    if q.dim() != 4:
        raise ValueError("q must be [B,m,H,d_latent+d_rope]")
    B, m, H, d = q.shape
    if not 0 < d_latent <= d:
        raise ValueError(f"d_latent must be in [1,{d}]")
    _check_buffer(lengths, "lengths", (B,), _I32)
    if o is None:
        o = torch.empty((B, m, H, d_latent), dtype=out_dtype or q.dtype, device=dev)
    else:
        _check_buffer(o, "o", (B, m, H, d_latent), _FLOATS)
        if out_dtype is not None and out_dtype != o.dtype:
            raise TypeError(f"out_dtype {out_dtype} disagrees with o.dtype {o.dtype}")
    if lse is None:
        lse = torch.empty((B, m, H), dtype=torch.float32, device=dev)
    else:
        _check_buffer(lse, "lse", (B, m, H), _F32)
    _check_buffer(device_status, "device_status", (1,), _I32)
    a = LatentDecodeArgs(B=B, H=H, n_tokens=m, d_latent=d_latent, d_rope=d - d_latent, in_dtype=_dt(q.dtype), out_dtype=_dt(o.dtype), scale=scale, q=_p(q),
                         lengths=_p(lengths), o=_p(o), lse=_p(lse), device_status=_p(device_status))
    a.q_stride_b, a.q_stride_t, a.q_stride_h = _lead_strides(q, "q")
    _pages(a, cache, page_table, B, d, q.dtype)
    L = lib()
    need = int(L.kda_latent_decode_workspace_bytes(ctypes.byref(a)))
    if need == 0:
        raise KDAError(L.kda_latent_decode(ctypes.byref(a), None), "kda_latent_decode")
    ws = _workspace(need, dev)
    a.workspace, a.workspace_bytes = _p(ws), need
    _run(L.kda_latent_decode, a, dev, "kda_latent_decode")
    return o, lse
