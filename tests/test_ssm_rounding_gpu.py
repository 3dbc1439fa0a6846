"""Single elements of the scan's y against the fp64 form: every element within
half a step of its type, and a share of the magnitudes that were added up for
it (the scan of the absolute values), so that a sum whose terms cancel shows
how its terms were rounded."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import sublayer as R
from sublayer_testutil import rounded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, B, T, H, G, P, N, dtype, step):
    """Centred values, so that the sums cancel; dt in [0, step]."""
    rng = np.random.default_rng(seed)
    names = dict(x=(B, T, H, P), dt=(B, T, H), B=(B, T, G, N), C=(B, T, G, N))
    t, r = {}, {}
    for name, shape in names.items():
        v = step * rng.uniform(size=shape) if name == "dt" else rng.standard_normal(shape)
        t[name], r[name] = rounded(v, dtype)
        t[name] = t[name].cuda()
    for name, v in (("A", -rng.uniform(1, 16, H)), ("state", rng.standard_normal((B, H, N, P)))):
        t[name], r[name] = rounded(v, F32)
        t[name] = t[name].cuda()
    return t, r


def check_elements(name, got, want, bound):
    worst = float((np.abs(got.double().cpu().numpy() - want) / bound).max())
    print(f"[parity] {name}: worst element at {worst:.3f} of its bound", flush=True)
    assert worst <= 1, f"{name}: an element is off by {worst:.3f} of its bound"


@pytest.mark.parametrize("N,P", [(16, 16), (32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 70])
def test_the_state_behind_a_bf16_y(N, P, T):
    # Steps of 0 leave y_t = C_t^T S_0.  Roundings: y's own, 2^-8 of itself;
    # two bf16 parts of S_0, the first cut off and the second rounded, 2^-15 of
    # each term; fp32 accumulators, at most 4 products' sums of 2 parts, 2^-21.
    B, H, G = 2, 4, 2
    t, r = inputs(1, B, T, H, G, P, N, BF, 0.0)
    y, S = kda.ssm_prefill(t["x"], t["dt"], t["A"], t["B"], t["C"], initial_state=t["state"])
    C = np.repeat(r["C"], H // G, 2)
    want = np.einsum("bhnp,bthn->bthp", r["state"], C)
    mag = np.einsum("bhnp,bthn->bthp", np.abs(r["state"]), np.abs(C))
    assert torch.equal(S, t["state"])
    check_elements(f"{N}x{P} T={T}", y, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * mag)


@pytest.mark.parametrize("step", [0.01, 0.3])
@pytest.mark.parametrize("H,G,P,N", [(4, 2, 64, 128), (3, 1, 32, 64), (2, 1, 16, 32)])
def test_a_bf16_y(H, G, P, N, step):
    # Roundings relative to a term: w x cut to two parts in y 2^-14, scores in
    # two parts 2^-16, the product of both second parts left out 2^-15, the
    # state in two parts 2^-15, logs and their exponentials below 2^-16, fp32
    # accumulators (below 100 additions) 2^-17: 2^-12.8 together.
    t, r = inputs(2, 2, 200, H, G, P, N, BF, step)
    y, _ = kda.ssm_prefill(t["x"], t["dt"], t["A"], t["B"], t["C"], initial_state=t["state"])
    want = R.ssm_scan(*(r[k] for k in ("x", "dt", "A", "B", "C")), initial_state=r["state"])[0]
    mag = R.ssm_scan(np.abs(r["x"]), r["dt"], r["A"], np.abs(r["B"]), np.abs(r["C"]), initial_state=np.abs(r["state"]))[0]
    check_elements(f"H={H} {P}x{N} step {step}", y, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag)


@pytest.mark.parametrize("N,P", [(16, 16), (32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_an_fp32_y_of_one_state_row(dtype, N, P):
    # Steps of 0 and a C that picks one row: y is that row of the state, all 24
    # bits of it (three bf16 parts hold them, and their sums are exact).
    B, T, H, G = 2, 70, 4, 2
    t, _ = inputs(3, B, T, H, G, P, N, dtype, 0.0)
    row = torch.from_numpy(np.random.default_rng(4).integers(0, N, (B, T, G))).cuda()
    C = torch.nn.functional.one_hot(row, N).to(dtype)
    y, _ = kda.ssm_prefill(t["x"], t["dt"], t["A"], t["B"], C, initial_state=t["state"], out_dtype=F32)
    rows = row.repeat_interleave(H // G, 2).permute(0, 2, 1)[..., None].expand(B, H, T, P)
    assert torch.equal(y.transpose(1, 2), t["state"].gather(2, rows))


@pytest.mark.parametrize("step", [0.01, 0.3])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_an_fp32_y(dtype, step):
    # One chunk.  Relative to a term: products of parts left out 2^-20 + 2^-21,
    # accumulators (6 products' sums for each 32 of d_state and of the tokens)
    # 36 x 2^-24, logs and exponentials 2^-21: below 2^-18.
    B, H, G, P, N = 2, 4, 2, 64, 128
    T = 64 if dtype == BF else 32
    t, r = inputs(5, B, T, H, G, P, N, dtype, step)
    y, _ = kda.ssm_prefill(t["x"], t["dt"], t["A"], t["B"], t["C"], initial_state=t["state"], out_dtype=F32)
    want = R.ssm_scan(*(r[k] for k in ("x", "dt", "A", "B", "C")), initial_state=r["state"])[0]
    mag = R.ssm_scan(np.abs(r["x"]), r["dt"], r["A"], np.abs(r["B"]), np.abs(r["C"]), initial_state=np.abs(r["state"]))[0]
    check_elements(f"{dtype} step {step}", y, want, 2.0 ** -18 * mag)
