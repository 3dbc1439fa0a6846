"""Single elements of the absorbed form's results, and of the expanded form's where
the caller asks for precise products, against the fp64 form: every element within half a step of its type, and a share of the magnitudes that were
added up for it, so that a sum whose terms cancel shows how its terms were
rounded."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from latent_testutil import BF16, FP32, Cache, cut, make, offsets, same
from oracle import latent as R
from sublayer_testutil import rounded

pytestmark = pytest.mark.gpu


def check_elements(name, got, want, bound):
    worst = float((np.abs(got.double().cpu().numpy() - want) / bound).max())
    print(f"[parity] {name}: worst element at {worst:.3f} of its bound", flush=True)
    assert worst <= 1, f"{name}: an element is off by {worst:.3f} of its bound"


@pytest.mark.parametrize("out_dtype,half", [(BF16, 2.0 ** -8), (FP32, 2.0 ** -24)])
@pytest.mark.parametrize("dc,dr,H,m", [(512, 64, 8, 1), (256, 32, 20, 2), (128, 64, 33, 3), (8, 8, 1, 1)])
def test_absorbed_elements_of_bf16_inputs(out_dtype, half, dc, dr, H, m):
    # Roundings relative to a term p |v|: two bf16 parts of p 2^-16; the exponent,
    # whose score is a sum of at most 32 products' sums in fp32, none larger than
    # the sum of magnitudes; the same again in the sum that divides; the sums over
    # the keys, the exponential and the division, below 100 roundings, 2^-17.
    scale, lengths = 0.07, [70, 5, 300, 129]
    c = Cache(dc + H, lengths, lengths, dc + dr, 16, BF16)
    q, q64 = rounded(1.5 * np.random.default_rng(H).standard_normal((len(lengths), m, H, dc + dr)), BF16)
    o, _ = kda.latent_decode(q.cuda(), c.cache, c.table, c.lengths, dc, scale, out_dtype=out_dtype)
    for b, n in enumerate(lengths):
        rows = c.rows[b][:n]
        want, _ = R.decode(q64[b], rows, dc, scale)
        sums = scale * np.einsum("mhd,nd->mhn", np.abs(q64[b]), np.abs(rows)).max(-1)[..., None]
        magnitudes = np.zeros_like(want)
        for j in range(m):
            sees = rows[:n - m + 1 + j]
            for h in range(H):
                s = scale * (q64[b, j, h] @ sees.T)
                p = np.exp(s - s.max())
                magnitudes[j, h] = (p / p.sum()) @ np.abs(sees[:, :dc])
        bound = half * np.abs(want) + (2.0 ** -16 + 2.0 ** -17 + 2 * 32 * 2.0 ** -24 * sums) * magnitudes
        check_elements(f"{dc} {dr} {H} {m} {out_dtype} sequence {b}", o[b], want, bound)


def expanded(seed, H, dims, lens, lens_k, causal, out_dtype, precise):
    """The expanded form and its gradients of packed bf16 sequences, and for every result its value and the magnitudes
    added up for it, in 64 bits (the gradients with the forward's o as it is).  The last: the largest score's sum of magnitudes."""
    dn, dr, dv = dims
    t, w, d_o, d64 = make(seed, (1, sum(lens)), (1, sum(lens_k)), H, dn, dr, dv, BF16)
    kw = dict(cu_seqlens=offsets(lens), cu_seqlens_k=offsets(lens_k), causal=causal, precise=precise)
    o, lse = kda.latent_prefill(**t, out_dtype=out_dtype, **kw)
    got = [o, *kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, **kw)]
    want, size = [[] for _ in got], [[] for _ in got]
    scale, at, at_k, sums = (dn + dr) ** -0.5, 0, 0, 0.0
    for n, m in zip(lens, lens_k):
        s = cut(w, 0, at, at + n, at_k, at_k + m)
        g, given = d64[0, at:at + n], o[0, at:at + n].double().cpu().numpy()
        at, at_k = at + n, at_k + m
        a = {k: None if v is None else np.abs(v) for k, v in s.items()}
        value = [R.prefill(**s, scale=scale, causal=causal)[0], *R.prefill_backward(**s, d_o=g, scale=scale, causal=causal, o=given)]
        terms = [R.prefill(**dict(s, v=a["v"]), scale=scale, causal=causal)[0], *R.prefill_backward_terms(**s, d_o=g, scale=scale, causal=causal)[:3],
                 R.prefill_backward(**s, d_o=np.abs(g), scale=scale, causal=causal)[3]]
        for k, (x, y) in enumerate(zip(value, terms)):
            want[k].append(x)
            size[k].append(y)
        if n and m:
            k = np.concatenate([a["k_nope"]] + ([] if dr == 0 else [np.repeat(a["k_rope"][:, None], H, 1)]), -1)
            sums = max(sums, scale * np.einsum("thd,shd->hts", a["q"], k).max())
    join = lambda parts, like: np.concatenate(parts).reshape(like.shape) if like is not None else None  # noqa: E731
    return got, [join(p, g) for p, g in zip(want, got)], [join(p, g) for p, g in zip(size, got)], sums


@pytest.mark.parametrize("out_dtype,half", [(BF16, 2.0 ** -8), (FP32, 2.0 ** -24)])
@pytest.mark.parametrize("dims", [(128, 64, 128), (128, 0, 128), (64, 32, 80), (32, 16, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_precise_expanded_elements_of_bf16_inputs(out_dtype, half, dims, causal):
    # Roundings relative to a term: two bf16 parts of p, or of a score's gradient,
    # 2^-16; the exponent as above, in the probabilities and in lse; the difference
    # of two sums of up to 128 products in a score's gradient, the sums over tokens
    # and (of dk_rope) heads, the exponential, below 200 roundings, 2^-16.
    got, want, size, sums = expanded(dims[0] + dims[1], 3, dims, [70, 1, 0, 130], [70, 40, 5, 161], causal, out_dtype, True)
    for name, g, w, s in zip(("o", "dq", "dk_nope", "dk_rope", "dv"), got, want, size):
        if g is not None:
            own = half if name == "o" else 2.0 ** -8
            check_elements(f"{dims} {causal} {name}", g, w, own * np.abs(w) + (2 * 2.0 ** -16 + 2 * 32 * 2.0 ** -24 * sums) * s + 1e-30)


def test_precise_is_the_callers_choice():
    """Without it the bits are those of one part; float32 inputs have all of theirs either way."""
    t, _, d_o, _ = make(5, (1, 90), (1, 90), 2, 64, 32, 64, BF16)
    o, lse = kda.latent_prefill(**t)
    p, lse_p = kda.latent_prefill(**t, precise=True)
    assert same(lse, lse_p) and not same(o, p)
    assert not same(kda.latent_backward(**t, o=o, lse=lse, d_o=d_o)[0], kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, precise=True)[0])
    wide = kda.latent_prefill(**t, precise=True, out_dtype=FP32)[0]
    assert same(wide.to(BF16), p)
    u = {k: v.float() for k, v in t.items()}
    a, b = kda.latent_prefill(**u), kda.latent_prefill(**u, precise=True)
    assert all(same(x, y) for x, y in zip(a, b))
    grads = [kda.latent_backward(**u, o=a[0], lse=a[1], d_o=d_o.float(), precise=x) for x in (False, True)]
    assert all(same(x, y) for x, y in zip(*grads))
