"""Shared by the tests of latent attention: seeded inputs, the paged cache, and
tolerances counted in roundings.

Errors are 2-norms over the 2-norm of the fp64 value, per tensor.  bf16: a value
rounded once is off by at most 2^-8 of itself.  The forward rounds twice (the
probabilities as operands, the result), so do the gradients (the probabilities
or the scores' gradients as operands, the result); the fp32 parts inside add
less than a third rounding.  A gradient's o is an input: where it is rounded the
fp64 form takes the rounded one.  fp32: an exponent of magnitude up to 64 carries 2^-24 of itself, 2^-18
absolute, into a probability; the sums' own roundings stay below that; the
gradients take the product of two such values."""
import numpy as np
import torch

from oracle import latent as R
from sublayer_testutil import check, rounded

BF16, FP32 = torch.bfloat16, torch.float32
FORWARD = {BF16: 2 * 2.0 ** -8, FP32: 2.0 ** -18}
BACKWARD = {BF16: 3 * 2.0 ** -8, FP32: 2.0 ** -17}
LSE = 2.0 ** -18  # statistics are fp32 whatever the type


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


def make(seed, lead_q, lead_k, H, dn, dr, dv, dtype, wide=1.5):
    """Device tensors as a layer has them (k_nope and v slices of one
    up-projection, k_rope a slice of the down-projection) and fp64 values."""
    rng = np.random.default_rng(seed)
    q, q64 = rounded(wide * rng.standard_normal((*lead_q, H, dn + dr)), dtype)
    up, up64 = rounded(rng.standard_normal((*lead_k, H, dn + dv)), dtype)
    down, down64 = rounded(rng.standard_normal((*lead_k, 24 + dr)), dtype)
    d_o, d64 = rounded(rng.standard_normal((*lead_q, H, dv)), dtype)
    up, down = up.cuda(), down.cuda()
    t = dict(q=q.cuda(), k_nope=up[..., :dn], k_rope=down[..., 24:] if dr else None, v=up[..., dn:])
    w = dict(q=q64, k_nope=up64[..., :dn], k_rope=down64[..., 24:] if dr else None, v=up64[..., dn:])
    return t, w, d_o.cuda(), d64


def cut(w, b, q_from, q_to, k_from, k_to):
    """One sequence's arrays."""
    return dict(q=w["q"][b, q_from:q_to], k_nope=w["k_nope"][b, k_from:k_to], v=w["v"][b, k_from:k_to],
                k_rope=None if w["k_rope"] is None else w["k_rope"][b, k_from:k_to])


def check_gradient(name, got, want, tol, terms):
    """A score's gradient is a difference of two sums of up to 128 products, which may
    cancel (with one key they are equal).  Either sum is off by some roundings, 2^-24 each,
    of its terms: 16 of them are allowed for, 2^-20 of ``terms``, the terms' own sizes
    carried into the gradient."""
    g, w = got.double().cpu().numpy(), np.asarray(want)
    assert g.shape == w.shape and np.isfinite(g).all()
    e, most = np.linalg.norm(g - w), tol * np.linalg.norm(w) + 2.0 ** -20 * np.linalg.norm(terms)
    print(f"[parity] {name}: {e:.3e} (<= {most:.3e})", flush=True)
    assert e <= most, f"{name}: {e:.3e} > {most:.3e}"


def check_lse(name, got, want):
    g, w = got.double().cpu().numpy(), np.asarray(want)
    none = np.isneginf(w)
    assert np.array_equal(np.isneginf(g), none), f"{name}: rows without a key"
    check(name, torch.from_numpy(np.where(none, 0, g)), np.where(none, 0, w), LSE)


class Cache:
    """Pages in no order over a pool that holds NaN wherever no row is."""

    def __init__(self, seed, lengths, room, d, page, dtype, fill=True, spare=2):
        rng = np.random.default_rng(seed)
        self.page, self.d, self.dtype = page, d, dtype
        need = [-(-max(n, r) // page) for n, r in zip(lengths, room)]
        pool = sum(need) + spare
        order = rng.permutation(pool)
        width = max(max(need), 1)
        # entries behind a sequence's pages point nowhere
        table = np.full((len(lengths), width), 2 ** 30, dtype=np.int32)
        at = 0
        for n, c in enumerate(need):
            table[n, :c] = order[at:at + c]
            at += c
        cache = np.full((pool, page, d), np.nan)
        self.rows = []
        for n, length in enumerate(lengths):
            t, r64 = rounded(rng.standard_normal((length, d)), dtype)
            self.rows.append(r64)
            for i in range(length if fill else 0):
                cache[table[n, i // page], i % page] = r64[i]
        self.cache = torch.from_numpy(cache).to(dtype).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.lengths = torch.tensor(lengths, dtype=torch.int32).cuda()
        self.np_table = table


def decode_reference(q64, cache, d_latent, scale, lengths):
    o, lse = zip(*(R.decode(q64[b], cache.rows[b][:max(0, n)], d_latent, scale) for b, n in enumerate(lengths)))
    return np.stack(o), np.stack(lse)
