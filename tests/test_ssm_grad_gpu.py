"""Gradients of the selective state space scan against the fp64 token-by-token
form and against differences."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import sublayer as R
from sublayer_testutil import TOL, TOL_SPLIT, check, rounded, scan_inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "d_initial")


def run(seed, B, T, H, G, P, N, dtype, lens=None, carry=True, steps=(0.001, 0.1), D=True, bias=True, softplus=True, name=""):
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = T if lens is None else int(cu[-1])
    ns = B if lens is None else len(lens)
    t, r = scan_inputs(seed, (B, T), H, G, P, N, dtype, steps=steps)
    rng = np.random.default_rng(seed + 1)
    dy, dy64 = rounded(rng.standard_normal((B, T, H, P)), dtype)
    s64, d64 = (rng.standard_normal((ns, H, N, P)).astype(np.float32) for _ in range(2)) if carry else (None, None)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    got = kda.ssm_backward(t["x"], t["dt"], t["A"], t["B"], t["C"], dy.cuda(), D=t["D"] if D else None,
                           dt_bias=t["dt_bias"] if bias else None, dt_softplus=softplus, initial_state=dev(s64), d_final_state=dev(d64),
                           cu_seqlens=dev(cu))
    want = R.ssm_scan_backward(r["x"], r["dt"], r["A"], r["B"], r["C"], dy64, r["D"] if D else None, r["dt_bias"] if bias else None, softplus,
                               s64, d64, cu)
    # sums over the tokens of bf16 inputs' gradients inherit the two-part operands' bound
    fp = TOL_SPLIT if dtype == BF else TOL[F32]
    for n, a, b in zip(NAMES, got, want):
        if n == "ddt_bias" and not bias or n == "dD" and not D:
            assert a is None
            continue
        check(f"{name} {n}", a, b, TOL[BF] if a.dtype == BF else fp)
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_state_sizes(dtype, N, P):
    run(N * P, 2, 150, 2, 1, P, N, dtype, name=f"{N}x{P}")


@pytest.mark.parametrize("T", [0, 1, 2, 31, 32, 33, 63, 64, 65, 97, 128, 257])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_lengths(T, dtype):
    run(10 + T, 2, T, 2, 2, 32, 32, dtype, name=f"T={T}")


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (8, 8), (10, 2), (20, 1), (6, 3)])
def test_head_layouts(H, G):
    run(30 + H, 1, 200, H, G, 64, 64, BF, name=f"H={H} G={G}")
    run(31 + H, 1, 70, H, G, 16, 16, F32, name=f"H={H} G={G}")


@pytest.mark.parametrize("lens", [[5, 0, 1, 64, 200, 65, 0], [700, 1, 333], [0], [1, 1, 1, 1], [0, 0, 1500]])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_packed(lens, dtype):
    run(40, 1, 0, 4, 2, 32, 64, dtype, lens=lens, name=f"{lens}")
    run(41, 1, 0, 4, 2, 32, 64, dtype, lens=lens, carry=False, name=f"{lens} no state")


@pytest.mark.parametrize("steps", [(1e-5, 1e-4), (0.5, 2.0), (5.0, 50.0)], ids=["slow", "fast", "extreme"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_decays(steps, dtype):
    run(50, 1, 300, 4, 1, 64, 64, dtype, steps=steps, name=f"steps {steps}")


def test_without_the_optional_arguments():
    run(60, 2, 100, 4, 2, 32, 32, F32, carry=False, D=False, bias=False, name="plain")
    run(61, 2, 100, 4, 2, 32, 32, BF, carry=False, D=False, bias=False, name="plain bf16")


def test_long_sequences():
    """Few heads: the state passes run in segments; many chunks' shares of the sums."""
    run(70, 1, 3000, 2, 1, 64, 128, BF, name="3000 tokens")
    run(71, 1, 2000, 1, 1, 16, 32, F32, name="2000 tokens")


def test_against_differences():
    t, r = scan_inputs(80, (1, 70), 2, 1, 16, 16, F32)
    rng = np.random.default_rng(81)
    dy = rng.standard_normal((1, 70, 2, 16))
    got = kda.ssm_backward(t["x"], t["dt"], t["A"], t["B"], t["C"], torch.from_numpy(dy).float().cuda(), D=t["D"], dt_bias=t["dt_bias"],
                           dt_softplus=True)
    grads = dict(zip(("x", "dt", "A", "B", "C", "D", "dt_bias"), got))

    def loss(**over):
        v = dict(r, **over)
        return (R.ssm_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["dt_bias"], True)[0] * dy).sum()

    for name, at in [("x", (0, 3, 1, 5)), ("x", (0, 69, 0, 0)), ("dt", (0, 10, 0)), ("dt", (0, 64, 1)), ("A", (1,)), ("B", (0, 20, 0, 7)),
                     ("C", (0, 65, 0, 2)), ("D", (0,)), ("dt_bias", (1,))]:
        e = np.zeros_like(r[name])
        e[at] = 1e-5
        d = (loss(**{name: r[name] + e}) - loss(**{name: r[name] - e})) / 2e-5
        g = float(grads[name][at])
        assert abs(d - g) <= 2e-5 * max(1.0, abs(d)), (name, at, d, g)


def test_malformed_offsets_write_no_gradient():
    t, _ = scan_inputs(82, (1, 100), 2, 1, 32, 32, BF)
    cu = torch.tensor([0, 60, 50, 100], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.ssm_backward(t["x"], t["dt"], t["A"], t["B"], t["C"], t["x"].contiguous(), cu_seqlens=cu, device_status=status)
    assert int(status) == 6


def test_same_results_from_run_to_run():
    a = run(90, 1, 1000, 6, 2, 64, 64, BF, name="once")
    b = run(90, 1, 1000, 6, 2, 64, 64, BF, name="twice")
    assert all(torch.equal(u, v) for u, v in zip(a, b))
