"""Gradients of the short causal convolution against the fp64 form: widths,
types, packed documents shorter than the window, carried windows."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import sublayer as R
from sublayer_testutil import TOL, check, rounded

pytestmark = pytest.mark.gpu


def run(seed, B, T, C, W, dtype, silu, lens=None, carry=True, gdtype=None, bias=True, name=""):
    rng = np.random.default_rng(seed)
    N = B if lens is None else len(lens)
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = T if lens is None else int(cu[-1])
    x, x64 = rounded(rng.standard_normal((B, T, C)), dtype)
    dy, dy64 = rounded(rng.standard_normal((B, T, C)), gdtype or dtype)
    w, w64 = rounded(rng.standard_normal((C, W)) / np.sqrt(W), torch.float32)
    b, b64 = rounded(0.1 * rng.standard_normal(C), torch.float32) if bias else (None, None)
    s0, s64 = rounded(rng.standard_normal((N, C, W - 1)), torch.float32) if carry else (None, None)
    df, df64 = rounded(rng.standard_normal((N, C, W - 1)), torch.float32) if carry else (None, None)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = kda.short_conv_backward(dev(x), dev(w), dev(dy), initial_state=dev(s0), bias=dev(b),
                                  cu_seqlens=None if cu is None else torch.from_numpy(cu).cuda(), silu=silu, d_final_state=dev(df))
    want = R.short_conv_backward(x64, w64, dy64, s64, b64, cu, silu, df64)
    for n, a, r in zip(("dx", "dweight", "dbias", "d_initial"), got, want):
        check(f"{name} {n}", a, r, TOL[a.dtype])


@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("dtype,gdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                          (torch.float32, torch.bfloat16)])
def test_widths_and_types(W, dtype, gdtype):
    run(W, 2, 75, 64, W, dtype, True, gdtype=gdtype, name=f"W={W}")


@pytest.mark.parametrize("T", [0, 1, 2, 3, 7, 8, 9, 33, 257])
@pytest.mark.parametrize("carry", [False, True])
def test_lengths(T, carry):
    run(20 + T, 3, T, 24, 4, torch.float32, True, carry=carry, name=f"T={T}")


@pytest.mark.parametrize("C", [8, 16, 40, 72, 520, 1032])
def test_channel_counts(C):
    run(40, 1, 300, C, 4, torch.bfloat16, True, name=f"C={C}")


@pytest.mark.parametrize("lens", [[5, 0, 1, 2, 40, 16, 3], [100, 0, 3, 64, 1, 200, 2], [0, 0, 1]])
@pytest.mark.parametrize("W,silu", [(4, True), (8, False), (2, True)])
def test_packed(lens, W, silu):
    run(50, 1, 0, 48, W, torch.float32, silu, lens=lens, name=f"{lens} W={W}")
    run(51, 1, 0, 48, W, torch.bfloat16, silu, lens=lens, carry=False, bias=False, name=f"{lens} W={W} bf16")


def test_forward_backward_agree_with_differences():
    rng = np.random.default_rng(60)
    x, w, dy = rng.standard_normal((1, 9, 8)), rng.standard_normal((8, 4)), rng.standard_normal((1, 9, 8))
    from oracle import reference
    f = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    dx, dw, _, _ = kda.short_conv_backward(f(x), f(w), f(dy), silu=True)

    def loss(x, w):
        return (reference.short_conv(x, w, silu=True)[0] * dy).sum()

    for t, c in [(0, 0), (5, 3), (8, 7)]:
        e = np.zeros_like(x)
        e[0, t, c] = 1e-5
        d = (loss(x + e, w) - loss(x - e, w)) / 2e-5
        assert abs(d - float(dx[0, t, c])) <= 2e-5 * max(1, abs(d))
    e = np.zeros_like(w)
    e[2, 1] = 1e-5
    d = (loss(x, w + e) - loss(x, w - e)) / 2e-5
    assert abs(d - float(dw[2, 1])) <= 2e-5 * max(1, abs(d))


def test_far_gradients_do_not_cross_documents():
    """Non-finite values of one document stay out of its neighbours."""
    C, cu = 16, torch.tensor([0, 5, 10, 15], dtype=torch.int32, device="cuda")
    x = torch.randn((1, 15, C), device="cuda")
    dy = torch.randn((1, 15, C), device="cuda")
    w = torch.randn((C, 4), device="cuda")
    want = kda.short_conv_backward(x, w, dy, cu_seqlens=cu, silu=True)[0]
    x2, dy2 = x.clone(), dy.clone()
    x2[:, 5:10], dy2[:, 5:10] = float("nan"), float("inf")
    got = kda.short_conv_backward(x2, w, dy2, cu_seqlens=cu, silu=True)[0]
    assert torch.equal(got[:, :5], want[:, :5]) and torch.equal(got[:, 10:], want[:, 10:])


def test_same_results_from_run_to_run():
    x = torch.randn((2, 1000, 520), device="cuda").bfloat16()
    w = torch.randn((520, 4), device="cuda")
    a = kda.short_conv_backward(x, w, x, silu=True)
    b = kda.short_conv_backward(x, w, x, silu=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
