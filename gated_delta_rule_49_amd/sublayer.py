"""The stages around the recurrence and the state space scan (C ABI in
``include/kda.h``): like the rest of the binding these functions only check
and marshal torch tensors, allocate outputs and workspaces with torch, and
launch on torch's current stream of the tensors' device.

``short_conv_backward``  gradients of the short causal convolution
``ssm_prefill`` / ``ssm_decode`` / ``ssm_backward``  the selective state space
    scan for prompts, for a few tokens, and its gradients
``block_norm`` / ``block_norm_backward``  the norm after a block with its
    gate, the scaled residual and the norm before the next block
"""
from __future__ import annotations

import ctypes

import torch

from . import (GATE_SIGMOID, GATE_SILU, SSM_CHUNK, BlockNormArgs, BlockNormBackwardArgs, ConvBackwardArgs, KDAError,
               SsmArgs, SsmBackwardArgs, SsmDecodeArgs, _check_buffer, _check_dev, _dt, _host_chunk_count, lib)

_F32 = (torch.float32,)


def _p(t):
    return None if t is None else t.data_ptr()


def _run(fn, a, dev, what):
    """Launches on torch's current stream of ``dev``, with ``dev`` current."""
    stream = torch.cuda.current_stream(dev).cuda_stream
    if dev.index is None or dev.index == torch.cuda.current_device():
        st = fn(ctypes.byref(a), stream)
    else:
        with torch.cuda.device(dev):
            st = fn(ctypes.byref(a), stream)
    if st != 0:
        raise KDAError(st, what)


def _need_device(dev, *ts):
    """Tensors that may have strides: on the GPU the others are on."""
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be on the GPU (no CPU path exists)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors are on different devices")
    return dev


def _dense(dev, *ts):
    """Contiguous tensors, on ``dev``."""
    _check_dev(*ts)
    _need_device(dev, *ts)


def _workspace(need, dev):
    return torch.empty(need, dtype=torch.uint8, device=dev)


# ------------------------------------------------------ convolution gradients
def short_conv_backward(x, weight, d_y, initial_state=None, bias=None, cu_seqlens=None, silu=False, d_final_state=None):
    """Gradients of ``short_conv`` with the same x, weight, initial_state,
    bias, cu_seqlens and silu: (dx like x, dweight fp32 [C,W], dbias fp32 [C],
    d_initial_state fp32 [N,C,W-1]) from d_y [B,T,C] (float32 or bfloat16) and
    d_final_state fp32 [N,C,W-1] (None = zeros).  dbias is the bias's gradient
    also where none was added; d_initial_state also where it was zeros."""
    dev = _check_dev(x, weight, d_y, initial_state, bias, cu_seqlens, d_final_state)
    if x.dim() != 3:
        raise ValueError("x must be [B,T,C]")
    B, T, C = x.shape
    if weight.dtype != torch.float32 or weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight must be float32 [{C},W]")
    W = weight.shape[1]
    if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1):
        raise TypeError("cu_seqlens must be int32 [N+1]")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _check_buffer(d_y, "d_y", (B, T, C), (torch.float32, torch.bfloat16))
    _check_buffer(bias, "bias", (C,), _F32)
    _check_buffer(initial_state, "initial_state", (N, C, W - 1), _F32)
    _check_buffer(d_final_state, "d_final_state", (N, C, W - 1), _F32)
    dx = torch.empty_like(x)
    dweight = torch.empty_like(weight)
    dbias = torch.empty(C, dtype=torch.float32, device=dev)
    d_initial = torch.empty((N, C, W - 1), dtype=torch.float32, device=dev)
    a = ConvBackwardArgs(B=B, T=T, C=C, W=W, num_seqs=N, in_dtype=_dt(x.dtype), grad_dtype=_dt(d_y.dtype),
                         activation=1 if silu else 0, x=_p(x), weight=_p(weight), bias=_p(bias), cu_seqlens=_p(cu_seqlens),
                         initial_state=_p(initial_state), d_y=_p(d_y), d_final_state=_p(d_final_state), dx=_p(dx),
                         dweight=_p(dweight), dbias=_p(dbias), d_initial_state=_p(d_initial))
    L = lib()
    ws = _workspace(int(L.kda_short_conv_backward_workspace_bytes(ctypes.byref(a))), dev)
    a.workspace, a.workspace_bytes = _p(ws), ws.numel()
    _run(L.kda_short_conv_backward, a, dev, "kda_short_conv_backward")
    return dx, dweight, dbias, d_initial


# ------------------------------------------------------------ state space scan
def _strides(t, name):
    """(batch, token) strides of [B, T, heads, channels], whose last two axes
    must be dense (a slice of a wider token is fine)."""
    if t.shape[3] > 1 and t.stride(3) != 1 or t.shape[2] > 1 and t.stride(2) != t.shape[3]:
        raise ValueError(f"{name}: the last two axes must be contiguous")
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def _scan_args(cls, x, dt, A, B, C, D, dt_bias, dt_softplus):
    dev = _need_device(_check_dev(dt, A, D, dt_bias), x, B, C)
    if x.dim() != 4 or B.dim() != 4 or C.shape != B.shape or B.shape[:2] != x.shape[:2]:
        raise ValueError("x must be [B,T,H,d_head], B and C [B,T,G,d_state]")
    nb, t, h, p = x.shape
    g, n = B.shape[2:]
    if not (x.dtype == dt.dtype == B.dtype == C.dtype):
        raise TypeError("x, dt, B, C must share one dtype")
    _check_buffer(dt, "dt", (nb, t, h), (x.dtype,))
    for name, v in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        _check_buffer(v, name, (h,), _F32)
    a = cls(B=nb, H=h, G=g, d_head=p, d_state=n, in_dtype=_dt(x.dtype), dt_softplus=1 if dt_softplus else 0,
            x=_p(x), dt=_p(dt), Bm=_p(B), Cm=_p(C), A=_p(A), D=_p(D), dt_bias=_p(dt_bias))
    a.x_stride_b, a.x_stride_t = _strides(x, "x")
    a.b_stride_b, a.b_stride_t = _strides(B, "B")
    a.c_stride_b, a.c_stride_t = _strides(C, "C")
    return a, dev, (nb, t, h, p, g, n)


def _packed(cu_seqlens, nb, dev):
    if cu_seqlens is None:
        return nb
    _need_device(dev, cu_seqlens)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise TypeError("cu_seqlens must be contiguous int32 [N+1]")
    return cu_seqlens.numel() - 1


def ssm_prefill(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, initial_state=None, output_final_state=True,
                cu_seqlens=None, out_dtype=None, chunk_states=False, final_state=None, y=None, check_seqlens=True,
                device_status=None):
    """Selective state space scan over whole sequences.

    x [B,T,H,d_head], B and C [B,T,G,d_state] (head h reads group h // (H/G);
    slices of a wider token are taken as they are), dt [B,T,H], all float32 or
    all bfloat16; A, D, dt_bias float32 [H].  Per token and head
    dt = softplus(dt + dt_bias) (with ``dt_softplus``, else dt + dt_bias),
    S = exp(A dt) S + dt B x^T, y = S^T C + D x.  A step of 0 leaves the state
    as it is; under the softplus the dtype's lowest value or -inf is one.  ``cu_seqlens`` (int32 [N+1],
    batch 1) packs N documents along T; ``initial_state`` fp32
    [N,H,d_state,d_head] or None (zeros).  Returns (y, final_state or None) or,
    with ``chunk_states``, (y, final_state, states entering every SSM_CHUNK
    tokens, documents in order).

    ``y`` ([B,T,H,d_head] float32 or bfloat16, default x's dtype) and
    ``final_state`` are optional preallocated buffers; final_state may be
    initial_state.  ``check_seqlens`` and ``device_status`` as for
    ``prefill``."""
    a, dev, (nb, t, h, p, g, n) = _scan_args(SsmArgs, x, dt, A, B, C, D, dt_bias, dt_softplus)
    N = _packed(cu_seqlens, nb, dev)
    _dense(dev, initial_state, final_state, y, device_status)
    for name, v in (("initial_state", initial_state), ("final_state", final_state)):
        _check_buffer(v, name, (N, h, n, p), _F32)
    if y is not None:
        _check_buffer(y, "y", (nb, t, h, p), (torch.float32, torch.bfloat16))
        if out_dtype is not None and out_dtype != y.dtype:
            raise TypeError(f"out_dtype {out_dtype} disagrees with y.dtype {y.dtype}")
    else:
        y = torch.empty((nb, t, h, p), dtype=out_dtype or x.dtype, device=dev)
    status = device_status
    if device_status is not None:
        _check_buffer(device_status, "device_status", (1,), (torch.int32,))
    elif check_seqlens and cu_seqlens is not None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, h, n, p), dtype=torch.float32, device=dev)
    a.T, a.num_seqs, a.out_dtype = t, N, _dt(y.dtype)
    a.cu_seqlens, a.initial_state, a.final_state = _p(cu_seqlens), _p(initial_state), _p(final_state)
    a.y, a.device_status = _p(y), _p(status)
    L = lib()
    need = int(L.kda_ssm_workspace_bytes(ctypes.byref(a)))
    if need == 0:
        raise KDAError(L.kda_ssm_prefill(ctypes.byref(a), None), "kda_ssm_prefill")  # reports why
    cs = None
    if chunk_states:
        cs = torch.empty((int(L.kda_ssm_max_chunks(ctypes.byref(a))), h, n, p), dtype=torch.float32, device=dev)
        a.chunk_states = _p(cs)
    ws = _workspace(need, dev)
    a.workspace, a.workspace_bytes = _p(ws), need
    _run(L.kda_ssm_prefill, a, dev, "kda_ssm_prefill")
    if check_seqlens and cu_seqlens is not None and int(status.item()) != 0:
        raise KDAError(int(status.item()), "kda_ssm_prefill (device check)")
    if chunk_states:
        return y, final_state, cs[:_host_chunk_count(nb, t, cu_seqlens, SSM_CHUNK)]
    return y, final_state


def ssm_decode(x, dt, A, B, C, state, D=None, dt_bias=None, dt_softplus=False, out_dtype=None, update_state=True,
               token_states=False, y=None, final_state=None):
    """m consecutive tokens of the scan for each of B sequences in one launch.

    Arguments as for ``ssm_prefill`` with T = m tokens; ``state`` fp32
    [B,H,d_state,d_head] is the state before the first token.  With
    ``update_state`` the state after the last token is written back into it
    (else into ``final_state`` if given, else nowhere).  ``token_states``
    also returns the state after every token, [B,m,H,d_state,d_head].
    Returns (y [B,m,H,d_head], final state or None, token states or None)."""
    a, dev, (nb, m, h, p, g, n) = _scan_args(SsmDecodeArgs, x, dt, A, B, C, D, dt_bias, dt_softplus)
    _dense(dev, state, final_state, y)
    for name, v in (("state", state), ("final_state", final_state)):
        _check_buffer(v, name, (nb, h, n, p), _F32)
    if update_state and final_state is not None and final_state.data_ptr() != state.data_ptr():
        raise ValueError("update_state writes the final state into `state`; do not pass final_state too")
    if y is None:
        y = torch.empty((nb, m, h, p), dtype=out_dtype or x.dtype, device=dev)
    else:
        _check_buffer(y, "y", (nb, m, h, p), (torch.float32, torch.bfloat16))
        if out_dtype is not None and out_dtype != y.dtype:
            raise TypeError(f"out_dtype {out_dtype} disagrees with y.dtype {y.dtype}")
    if update_state:
        final_state = state
    ts = torch.empty((nb, m, h, n, p), dtype=torch.float32, device=dev) if token_states else None
    a.n_tokens, a.out_dtype = m, _dt(y.dtype)
    a.initial_state, a.final_state, a.token_states, a.y = _p(state), _p(final_state), _p(ts), _p(y)
    _run(lib().kda_ssm_decode, a, dev, "kda_ssm_decode")
    return y, final_state, ts


def ssm_backward(x, dt, A, B, C, d_y, D=None, dt_bias=None, dt_softplus=False, initial_state=None, d_final_state=None,
                 cu_seqlens=None, device_status=None):
    """Gradients of the scan from d_y [B,T,H,d_head] (x's dtype) and
    d_final_state fp32 [N,H,d_state,d_head] (None = zeros): (dx, ddt, dA, dB,
    dC, dD, ddt_bias, d_initial_state).  dx, ddt, dB and dC have x's dtype
    (dt's through its softplus and bias; those of B and C summed over a
    group's heads), the others are float32; dD is None without D, ddt_bias
    without dt_bias.  The states entering the chunks are recomputed from
    ``initial_state``.  Nothing synchronises; ``device_status`` (int32 [1] on
    the device) receives the call's device-side status: with malformed
    cu_seqlens the gradients are not written."""
    a, dev, (nb, t, h, p, g, n) = _scan_args(SsmBackwardArgs, x, dt, A, B, C, D, dt_bias, dt_softplus)
    N = _packed(cu_seqlens, nb, dev)
    _dense(dev, d_y, initial_state, d_final_state, device_status)
    _check_buffer(d_y, "d_y", (nb, t, h, p), (x.dtype,))
    for name, v in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        _check_buffer(v, name, (N, h, n, p), _F32)
    _check_buffer(device_status, "device_status", (1,), (torch.int32,))
    like = dict(dtype=x.dtype, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    dx, ddt = torch.empty((nb, t, h, p), **like), torch.empty((nb, t, h), **like)
    dB, dC = torch.empty((nb, t, g, n), **like), torch.empty((nb, t, g, n), **like)
    dA, d_initial = torch.empty(h, **f32), torch.empty((N, h, n, p), **f32)
    dD = torch.empty(h, **f32) if D is not None else None
    dbias = torch.empty(h, **f32) if dt_bias is not None else None
    a.T, a.num_seqs = t, N
    a.cu_seqlens, a.initial_state = _p(cu_seqlens), _p(initial_state)
    a.d_y, a.d_final_state = _p(d_y), _p(d_final_state)
    a.dx, a.ddt, a.dB, a.dC, a.dA, a.dD, a.ddt_bias = _p(dx), _p(ddt), _p(dB), _p(dC), _p(dA), _p(dD), _p(dbias)
    a.d_initial_state = _p(d_initial)
    L = lib()
    need = int(L.kda_ssm_backward_workspace_bytes(ctypes.byref(a)))
    if need == 0:
        raise KDAError(L.kda_ssm_backward(ctypes.byref(a), None), "kda_ssm_backward")
    ws = _workspace(need, dev)
    a.workspace, a.workspace_bytes = _p(ws), need
    _run(L.kda_ssm_backward, a, dev, "kda_ssm_backward")
    if device_status is not None:  # the workspace's first word is the call's status
        device_status.copy_(ws[:4].view(torch.int32))
    return dx, ddt, dA, dB, dC, dD, dbias, d_initial


# ----------------------------------------------------------------- block norm
_GATES = {"sigmoid": GATE_SIGMOID, "silu": GATE_SILU}


def _row_stride(t, name, shape, dtype):
    """Elements between rows of [..., dim] (channels contiguous, the leading
    axes one evenly spaced row axis)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return shape[-1]
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    axes = [(s, n) for s, n in zip(t.stride()[:-1], shape[:-1]) if n != 1]
    for (outer, _), (inner, n) in zip(axes, axes[1:]):
        if outer != inner * n:
            raise ValueError(f"{name}: rows must be evenly spaced")
    return axes[-1][0] if axes else shape[-1]


def _norm_args(x, residual, post_weight, gate, scale, pre_weight, gate_activation, gate_first, eps):
    dev = _need_device(_check_dev(post_weight, scale, pre_weight), x, residual, gate)
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    dim = x.shape[-1]
    if gate_activation not in _GATES:
        raise ValueError(f"gate_activation must be one of {sorted(_GATES)}, got {gate_activation!r}")
    a = BlockNormArgs(rows=x.numel() // dim if dim else 0, dim=dim, group=dim, dtype=_dt(x.dtype),
                      gate_activation=_GATES[gate_activation], gate_first=1 if gate_first else 0, eps=eps,
                      x_stride=_row_stride(x, "x", x.shape, x.dtype), x=_p(x), post_weight=_p(post_weight),
                      scale=_p(scale), pre_weight=_p(pre_weight))
    if gate is not None:
        a.gate, a.gate_stride = _p(gate), _row_stride(gate, "gate", x.shape, x.dtype)
    if residual is not None:
        a.residual, a.residual_stride = _p(residual), _row_stride(residual, "residual", x.shape, x.dtype)
    _check_buffer(scale, "scale", (dim,), _F32)
    _check_buffer(pre_weight, "pre_weight", (dim,), _F32)
    return a, dev, dim


def _post_group(a, post_weight, group_size, dim):
    """The groups of the norm after the block: ``group_size`` channels, or as
    many as post_weight has."""
    if post_weight is None:
        if group_size is not None:
            raise ValueError("group_size needs a post_weight")
        return
    if post_weight.dtype != torch.float32 or post_weight.dim() != 1:
        raise TypeError("post_weight must be a float32 vector")
    group = post_weight.numel() if group_size is None else int(group_size)
    if group < 1 or dim % group or post_weight.numel() not in (group, dim):
        raise ValueError(f"post_weight must be float32 [group] or [{dim}], with groups that divide {dim}")
    a.group = group
    a.post_per_channel = 1 if post_weight.numel() == dim else 0


def block_norm(x, residual=None, post_weight=None, gate=None, scale=None, pre_weight=None, group_size=None,
               gate_activation="sigmoid", gate_first=False, eps=1e-6, out=None, normed=None):
    """The stages between a block and the next one, in one pass over the rows
    of x [..., dim] (float32 or bfloat16): rms(v) = v / sqrt(mean(v^2) + eps),

        p = rms(x) * post_weight, over groups of ``group_size`` channels
        p = p * act(gate)          (``gate_first``: x * act(gate) before the norm)
        out = residual + scale * p
        normed = rms(out) * pre_weight     (of out before it is rounded)

    Every stage whose argument is None is left out.  ``post_weight`` float32
    [dim], or [group_size] shared by the groups (the group is post_weight's
    size when group_size is None); ``scale`` and ``pre_weight`` float32 [dim];
    ``gate`` and ``residual`` like x (all three may be slices of wider rows);
    ``gate_activation`` "sigmoid" or "silu".  Returns (out, normed or None),
    contiguous, x's dtype; ``out`` and ``normed`` may each be x's, the
    residual's or the gate's own memory (any other overlap is refused)."""
    a, dev, dim = _norm_args(x, residual, post_weight, gate, scale, pre_weight, gate_activation, gate_first, eps)
    _post_group(a, post_weight, group_size, dim)
    _dense(dev, out, normed)
    _check_buffer(out, "out", x.shape, (x.dtype,))
    _check_buffer(normed, "normed", x.shape, (x.dtype,))
    if normed is not None and pre_weight is None:
        raise ValueError("normed needs a pre_weight")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if normed is None and pre_weight is not None:
        normed = torch.empty(x.shape, dtype=x.dtype, device=dev)
    a.out, a.normed = _p(out), _p(normed)
    _run(lib().kda_block_norm, a, dev, "kda_block_norm")
    return out, normed


def block_norm_backward(x, d_out, d_normed=None, residual=None, post_weight=None, gate=None, scale=None, pre_weight=None,
                        group_size=None, gate_activation="sigmoid", gate_first=False, eps=1e-6):
    """Gradients of ``block_norm`` with the same arguments, from d_out and
    d_normed (contiguous, like x; either may be None = zeros): (dx, dresidual,
    dpost_weight, dgate, dscale, dpre_weight), None for what was not given.
    Those of the weights are float32 sums over all rows (over the groups too
    where post_weight is shared)."""
    a, dev, dim = _norm_args(x, residual, post_weight, gate, scale, pre_weight, gate_activation, gate_first, eps)
    _post_group(a, post_weight, group_size, dim)
    _dense(dev, d_out, d_normed)
    _check_buffer(d_out, "d_out", x.shape, (x.dtype,))
    _check_buffer(d_normed, "d_normed", x.shape, (x.dtype,))
    if d_normed is not None and pre_weight is None:
        raise ValueError("d_normed needs a pre_weight")

    def like(t):
        return None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev)

    dx, dresidual, dpost, dgate, dscale, dpre = (like(t) for t in (x, residual, post_weight, gate, scale, pre_weight))
    g = BlockNormBackwardArgs(f=a, d_out=_p(d_out), d_normed=_p(d_normed), dx=_p(dx), dgate=_p(dgate),
                              dresidual=_p(dresidual), dpost_weight=_p(dpost), dscale=_p(dscale), dpre_weight=_p(dpre))
    L = lib()
    need = int(L.kda_block_norm_backward_workspace_bytes(ctypes.byref(g)))
    if need == 0:
        raise KDAError(L.kda_block_norm_backward(ctypes.byref(g), None), "kda_block_norm_backward")
    ws = _workspace(need, dev)
    g.workspace, g.workspace_bytes = _p(ws), need
    _run(L.kda_block_norm_backward, g, dev, "kda_block_norm_backward")
    return dx, dresidual, dpost, dgate, dscale, dpre
