"""Single elements of the absorbed form's result against the fp64 form: every
element within half a step of its type, and a share of the magnitudes that were
added up for it, so that a sum whose terms cancel shows how its terms were
rounded."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from latent_testutil import BF16, FP32, Cache
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
