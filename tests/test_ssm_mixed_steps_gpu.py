"""Heads whose steps are large and small side by side: within one chunk the
sums of logs run to hundreds and more, while neighbouring tokens differ by one
small log.  Every element of y is held to a share of the magnitudes that were
added up for it (the scan of the absolute values)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import sublayer as R
from sublayer_testutil import rounded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
H, G, P, N = 4, 2, 32, 64


def inputs(seed, B, T, dtype, small, large, share=0.25, clear=False):
    """Steps of `small`, a random share of them `large`; clear: x = 0 there."""
    rng = np.random.default_rng(seed)
    big = rng.uniform(size=(B, T, H)) < share
    z = {k: rng.standard_normal(s) for k, s in (("x", (B, T, H, P)), ("B", (B, T, G, N)), ("C", (B, T, G, N)))}
    if clear:
        z["x"][big] = 0
    z["dt"] = np.where(big, large, small) * rng.uniform(0.9, 1.1, (B, T, H))
    t, r = {}, {}
    for k, v in z.items():
        t[k], r[k] = rounded(v, dtype)
    t["A"], r["A"] = rounded(np.linspace(-16, -1, H), F32)
    t["state"], r["state"] = rounded(rng.standard_normal((B, H, N, P)), F32)
    return {k: v.cuda() for k, v in t.items()}, r, big


def magnitudes(r):
    return R.ssm_scan(np.abs(r["x"]), r["dt"], r["A"], np.abs(r["B"]), np.abs(r["C"]), initial_state=np.abs(r["state"]))


def check_elements(name, got, want, bound):
    e = np.abs(got.double().cpu().numpy() - want)
    assert np.isfinite(e).all(), f"{name}: non-finite values"
    worst = float((e / np.maximum(bound, 1e-30)).max())
    print(f"[parity] {name}: worst element at {worst:.3f} of its bound", flush=True)
    assert worst <= 1, f"{name}: an element is off by {worst:.3f} of its bound"


# Relative to a term.  fp32 inputs, three parts each: products left out 2^-20,
# logs (three roundings of 2^-24, of logs that still matter: e 2^-e < 1) and
# their exponentials 2^-22, below 200 fp32 additions into an accumulator
# 2^-16.4: 2^-16 together.  bf16 inputs: two parts of the scores, of w x in y
# and of the state, 2^-12 with the rest, and y's own half step.
def bound_of(dtype, out, want, mag):
    return (2.0 ** -16 if dtype == F32 else 2.0 ** -12) * mag + (2.0 ** -8 * np.abs(want) if out == BF else 0)


STEPS = [(0.02, 8.0), (0.02, 20.0), (0.01, 50.0), (0.02, 2000.0)]


@pytest.mark.parametrize("small,large", STEPS)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32)])
def test_mixed_steps(dtype, out, small, large):
    t, r, _ = inputs(1, 2, 200, dtype, small, large)
    y, S = kda.ssm_prefill(*(t[k] for k in ("x", "dt", "A", "B", "C")), initial_state=t["state"], out_dtype=out)
    want, S_r, _, _ = R.ssm_scan(*(r[k] for k in ("x", "dt", "A", "B", "C")), initial_state=r["state"])
    mag, S_mag, _, _ = magnitudes(r)
    check_elements(f"{small} {large} y", y, want, bound_of(dtype, out, want, mag))
    check_elements(f"{small} {large} S", S, S_r, 2.0 ** -16 * S_mag)


@pytest.mark.parametrize("large", [1e4, 1e10, 1e30])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32)])
def test_tokens_that_forget_the_state(dtype, out, large):
    """A huge step with x = 0 ends what came before it; the tokens on either
    side of it in the same chunk keep their own small logs."""
    t, r, _ = inputs(2, 2, 200, dtype, 0.02, large, share=0.05, clear=True)
    y, S = kda.ssm_prefill(*(t[k] for k in ("x", "dt", "A", "B", "C")), initial_state=t["state"], out_dtype=out)
    want, S_r, _, _ = R.ssm_scan(*(r[k] for k in ("x", "dt", "A", "B", "C")), initial_state=r["state"])
    mag, S_mag, _, _ = magnitudes(r)
    check_elements(f"{large} y", y, want, bound_of(dtype, out, want, mag))
    check_elements(f"{large} S", S, S_r, 2.0 ** -16 * S_mag)
