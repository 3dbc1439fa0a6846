"""Plain fp64 forms of latent attention, its positions and its cache (numpy),
one sequence and one head at a time.  They share no code with the HIP path."""
import numpy as np


def rotary(x, positions, freqs, offset=0, interleaved=False, magnitude=1.0, back=False):
    """x [T, H, D], positions [T]."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    for i in range(n):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + n + i)
        angle = np.asarray(positions, dtype=np.float64)[:, None] * float(freqs[i]) * (-1 if back else 1)
        u, w = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
        y[..., a] = magnitude * (u * np.cos(angle) - w * np.sin(angle))
        y[..., b] = magnitude * (u * np.sin(angle) + w * np.cos(angle))
    return y


def append_row(row, position, d_latent, weight=None, eps=1e-6, freqs=None, interleaved=False, magnitude=1.0):
    """One token's cache row from its latent and its position key."""
    out = np.array(row, dtype=np.float64)
    c = out[:d_latent]
    if weight is not None:
        out[:d_latent] = c / np.sqrt(np.mean(c * c) + eps) * weight
    if freqs is not None and len(freqs):
        out[d_latent:] = rotary(out[None, None, d_latent:], [position], freqs, 0, interleaved, magnitude)[0, 0]
    return out


def attention(q, k, v, scale, causal):
    """One head of one sequence: q [tq, d], k [tk, d], v [tk, dv] -> (o, lse, p).
    The queries stand at the end of the keys; a query without a key has 0 and -inf."""
    tq, tk = q.shape[0], k.shape[0]
    s = scale * (q @ k.T)
    sees = np.arange(tk)[None, :] <= np.arange(tq)[:, None] + tk - tq if causal else np.ones((tq, tk), dtype=bool)
    p, lse = np.zeros((tq, tk)), np.full(tq, -np.inf)
    for i in range(tq):
        if not sees[i].any():
            continue
        x = s[i, sees[i]]
        lse[i] = x.max() + np.log(np.exp(x - x.max()).sum())
        p[i, sees[i]] = np.exp(x - lse[i])
    return p @ v, lse, p


def attention_backward(q, k, v, d_o, scale, causal, o=None):
    """(dq, dk, dv) of one head of one sequence; with the rowsum of d_o o for a given (rounded) o."""
    own, _, p = attention(q, k, v, scale, causal)
    dp = d_o @ v.T
    ds = scale * p * (dp - (d_o * (own if o is None else o)).sum(-1, keepdims=True))
    return ds @ k, ds.T @ q, p.T @ d_o


def backward_terms(q, k, v, d_o, scale, causal):
    """The sizes of the terms that cancel inside dq and dk: every score's gradient is a difference of
    d_o . v and rowsum(d_o o), here the sum of their products' magnitudes."""
    o, _, p = attention(q, k, v, scale, causal)
    size = abs(scale) * p * (np.abs(d_o) @ np.abs(v).T + (np.abs(d_o) * np.abs(o)).sum(-1, keepdims=True))
    return size @ np.abs(k), size.T @ np.abs(q)


def _heads(q, k_nope, k_rope, v, h):
    k = k_nope[:, h] if k_rope is None else np.concatenate([k_nope[:, h], k_rope], -1)
    return q[:, h], k, v[:, h]


def prefill(q, k_nope, k_rope, v, scale, causal=True):
    """One sequence, all heads: q [tq, H, d] .. -> (o [tq, H, dv], lse [tq, H])."""
    o, lse = np.zeros((*q.shape[:2], v.shape[-1])), np.zeros(q.shape[:2])
    for h in range(q.shape[1]):
        o[:, h], lse[:, h], _ = attention(*_heads(q, k_nope, k_rope, v, h), scale, causal)
    return o, lse


def prefill_backward(q, k_nope, k_rope, v, d_o, scale, causal=True, o=None):
    """(dq, dk_nope, dk_rope or None, dv) of one sequence."""
    n = k_nope.shape[-1]
    dq, dkn, dv = np.zeros_like(q), np.zeros_like(k_nope), np.zeros_like(v)
    dkr = None if k_rope is None else np.zeros_like(k_rope)
    for h in range(q.shape[1]):
        a, b, c = attention_backward(*_heads(q, k_nope, k_rope, v, h), d_o[:, h], scale, causal, None if o is None else o[:, h])
        dq[:, h], dkn[:, h], dv[:, h] = a, b[:, :n], c
        if dkr is not None:
            dkr += b[:, n:]
    return dq, dkn, dkr, dv


def prefill_backward_terms(q, k_nope, k_rope, v, d_o, scale, causal=True):
    """``backward_terms`` as (dq, dk_nope, dk_rope or None, zeros for dv)."""
    n = k_nope.shape[-1]
    dq, dkn = np.zeros_like(q), np.zeros_like(k_nope)
    dkr = None if k_rope is None else np.zeros_like(k_rope)
    for h in range(q.shape[1]):
        a, b = backward_terms(*_heads(q, k_nope, k_rope, v, h), d_o[:, h], scale, causal)
        dq[:, h], dkn[:, h] = a, b[:, :n]
        if dkr is not None:
            dkr += b[:, n:]
    return dq, dkn, dkr, np.zeros_like(v)


def decode(q, rows, d_latent, scale):
    """One sequence: q [m, H, d], its cache rows [n, d] -> (o [m, H, d_latent], lse [m, H])."""
    m, heads, _ = q.shape
    o, lse = np.zeros((m, heads, d_latent)), np.full((m, heads), -np.inf)
    for j in range(m):
        sees = rows[:max(0, len(rows) - m + 1 + j)]
        if len(sees):
            o[j], lse[j], _ = attention(q[j], sees, sees[:, :d_latent], scale, False)
    return o, lse
