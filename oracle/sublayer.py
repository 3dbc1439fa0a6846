"""Plain fp64 forms of the stages around the recurrence and of the selective
state space scan (tests only).  Token by token and row by row, straight from
the formulas in include/kda.h.

    ssm_scan / ssm_scan_backward    S_t = a_t S_{t-1} + dt_t B_t x_t^T, y_t = S_t^T C_t + D x_t
    short_conv_backward             gradients of reference.short_conv
    block_norm / block_norm_backward
"""
from __future__ import annotations

import numpy as np


def _sig(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def _f8(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def _bounds(shape, cu_seqlens):
    """(batch row, first token, end) of every sequence."""
    if cu_seqlens is None:
        return [(b, 0, shape[1]) for b in range(shape[0])]
    return [(0, int(a), int(e)) for a, e in zip(cu_seqlens[:-1], cu_seqlens[1:])]


def step_sizes(dt, dt_bias, softplus):
    z = dt if dt_bias is None else dt + dt_bias
    return np.logaddexp(z, 0.0) if softplus else z


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=False, initial_state=None, cu_seqlens=None, chunk=64):
    """(y, final states, states entering every `chunk` tokens, state after
    every token of the flattened token axis)."""
    x, dt, A, B, C, D, dt_bias, initial_state = _f8(x, dt, A, B, C, D, dt_bias, initial_state)
    h, p = x.shape[2:]
    g, n = B.shape[2:]
    B, C = np.repeat(B, h // g, 2), np.repeat(C, h // g, 2)
    dt = step_sizes(dt, dt_bias, softplus)
    y = np.zeros_like(x)
    final, entering, after = [], [], []
    for k, (b, t0, t1) in enumerate(_bounds(x.shape, cu_seqlens)):
        S = np.zeros((h, n, p)) if initial_state is None else initial_state[k].copy()
        for t in range(t0, t1):
            if (t - t0) % chunk == 0:
                entering.append(S)
            a = np.exp(A * dt[b, t])
            S = a[:, None, None] * S + B[b, t][:, :, None] * (dt[b, t][:, None] * x[b, t])[:, None, :]
            y[b, t] = np.einsum("hnp,hn->hp", S, C[b, t]) + (0 if D is None else D[:, None] * x[b, t])
            after.append(S)
        final.append(S)
    none = np.zeros((0, h, n, p))
    return y, np.array(final), np.array(entering) if entering else none, np.array(after) if after else none


def ssm_scan_backward(x, dt, A, B, C, dy, D=None, dt_bias=None, softplus=False, initial_state=None, d_final=None,
                      cu_seqlens=None):
    """(dx, ddt, dA, dB, dC, dD, ddt_bias, d_initial)."""
    x, dt, A, B, C, dy, D, dt_bias, initial_state, d_final = _f8(x, dt, A, B, C, dy, D, dt_bias, initial_state, d_final)
    h, p = x.shape[2:]
    g, n = B.shape[2:]
    Bh, Ch = np.repeat(B, h // g, 2), np.repeat(C, h // g, 2)
    step = step_sizes(dt, dt_bias, softplus)
    slope = _sig(dt if dt_bias is None else dt + dt_bias) if softplus else np.ones_like(dt)
    dx, ddt, dBh, dCh = np.zeros_like(x), np.zeros_like(dt), np.zeros_like(Bh), np.zeros_like(Ch)
    dA = np.zeros(h)
    d_initial = []
    for k, (b, t0, t1) in enumerate(_bounds(x.shape, cu_seqlens)):
        S = np.zeros((h, n, p)) if initial_state is None else initial_state[k]
        states = [S]
        for t in range(t0, t1):
            S = np.exp(A * step[b, t])[:, None, None] * S + Bh[b, t][:, :, None] * (step[b, t][:, None] * x[b, t])[:, None, :]
            states.append(S)
        G = np.zeros((h, n, p)) if d_final is None else d_final[k].copy()
        for t in range(t1 - 1, t0 - 1, -1):
            before, S, a = states[t - t0], states[t - t0 + 1], np.exp(A * step[b, t])
            dCh[b, t] = np.einsum("hnp,hp->hn", S, dy[b, t])
            G = G + Ch[b, t][:, :, None] * dy[b, t][:, None, :]
            u = step[b, t][:, None] * x[b, t]
            dBh[b, t] = np.einsum("hnp,hp->hn", G, u)
            du = np.einsum("hnp,hn->hp", G, Bh[b, t])
            dx[b, t] = step[b, t][:, None] * du + (0 if D is None else D[:, None] * dy[b, t])
            dlog = np.einsum("hnp,hnp->h", G, before) * a
            dA += dlog * step[b, t]
            ddt[b, t] = ((du * x[b, t]).sum(-1) + dlog * A) * slope[b, t]
            G = a[:, None, None] * G
        d_initial.append(G)
    fold = lambda v: v.reshape(*v.shape[:2], g, h // g, n).sum(3)  # noqa: E731
    return (dx, ddt, dA, fold(dBh), fold(dCh), None if D is None else (dy * x).sum((0, 1, 3)), ddt.sum((0, 1)), np.array(d_initial))


def short_conv_backward(x, w, dy, initial_state=None, bias=None, cu_seqlens=None, silu=False, d_final=None):
    """(dx, dw, dbias, d_initial)."""
    x, w, dy, initial_state, bias, d_final = _f8(x, w, dy, initial_state, bias, d_final)
    c, width = w.shape
    dx, dw, db, d_initial = np.zeros_like(x), np.zeros_like(w), np.zeros(c), []
    for k, (b, t0, t1) in enumerate(_bounds(x.shape, cu_seqlens)):
        before = np.zeros((width - 1, c)) if initial_state is None else initial_state[k].T
        xs = np.concatenate([before, x[b, t0:t1]])
        d = np.zeros_like(xs)
        for t in range(t1 - t0):
            pre = (w.T * xs[t:t + width]).sum(0) + (0 if bias is None else bias)
            s = _sig(pre)
            g = dy[b, t0 + t] * (s + pre * s * (1 - s) if silu else 1.0)
            d[t:t + width] += w.T * g
            dw += (g * xs[t:t + width]).T
            db += g
        if d_final is not None and width > 1:
            d[t1 - t0:] += d_final[k].T
        dx[b, t0:t1] = d[width - 1:]
        d_initial.append(d[:width - 1].T)
    return dx, dw, db, np.array(d_initial).reshape(len(d_initial), c, width - 1)


def _gate(z, kind):
    s = _sig(z)
    return (z * s, s + z * s * (1 - s)) if kind == "silu" else (s, s * (1 - s))


def block_norm(x, residual=None, post=None, gate=None, scale=None, pre=None, group=None, activation="sigmoid", gate_first=False,
               eps=1e-6):
    """(out, normed or None); every intermediate value as attributes of the
    returned dict is not needed: block_norm_backward recomputes them."""
    x, residual, post, gate, scale, pre = _f8(x, residual, post, gate, scale, pre)
    v = x
    act = None if gate is None else _gate(gate, activation)[0]
    if gate is not None and gate_first:
        v = v * act
    if post is not None:
        k = group or post.size
        vg = v.reshape(*v.shape[:-1], -1, k)
        v = (vg / np.sqrt((vg ** 2).mean(-1, keepdims=True) + eps)).reshape(v.shape) * np.resize(post, v.shape[-1])
    if gate is not None and not gate_first:
        v = v * act
    if scale is not None:
        v = v * scale
    if residual is not None:
        v = v + residual
    return v, None if pre is None else v / np.sqrt((v ** 2).mean(-1, keepdims=True) + eps) * pre


def block_norm_backward(x, d_out, d_normed=None, residual=None, post=None, gate=None, scale=None, pre=None, group=None,
                        activation="sigmoid", gate_first=False, eps=1e-6):
    """(dx, dresidual, dpost, dgate, dscale, dpre), None for what is not there."""
    x, d_out, d_normed, residual, post, gate, scale, pre = _f8(x, d_out, d_normed, residual, post, gate, scale, pre)
    rows = tuple(range(x.ndim - 1))
    dim = x.shape[-1]
    act, slope = (1.0, 0.0) if gate is None else _gate(gate, activation)
    a = x * act if gate_first else x
    w = None if post is None else np.resize(post, dim)
    if post is not None:
        k = group or post.size
        ag = a.reshape(*a.shape[:-1], -1, k)
        q = np.repeat(1 / np.sqrt((ag ** 2).mean(-1) + eps), k, -1)
        n1 = a * q * w
    else:
        n1 = a
    v = n1 if gate_first else n1 * act
    out = (v if scale is None else v * scale) + (0 if residual is None else residual)
    d = np.zeros_like(x) if d_out is None else d_out.copy()
    dpre = None
    if pre is not None:
        q2 = 1 / np.sqrt((out ** 2).mean(-1, keepdims=True) + eps)
        dn = np.zeros_like(x) if d_normed is None else d_normed
        dpre = (dn * out * q2).sum(rows)
        e = dn * pre
        d = d + q2 * e - out * q2 ** 3 * (e * out).mean(-1, keepdims=True)
    dres = None if residual is None else d
    dscale = None if scale is None else (d * v).sum(rows)
    d = d if scale is None else d * scale
    dgate = None
    if gate is not None and not gate_first:
        dgate, d = d * n1 * slope, d * act
    dpost = None
    if post is not None:
        full = (d * a * q).sum(rows)
        dpost = full if post.size == dim else full.reshape(-1, post.size).sum(0)
        e = d * w
        s = (e * a).reshape(*a.shape[:-1], -1, k).mean(-1)
        d = q * e - a * q ** 3 * np.repeat(s, k, -1)
    if gate is not None and gate_first:
        dgate, d = d * x * slope, d * act
    return d, dres, dpost, dgate, dscale, dpre
