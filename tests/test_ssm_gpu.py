"""The selective state space scan for prompts and for a few tokens, against
the fp64 token-by-token form."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import sublayer as R
from sublayer_testutil import TOL, TOL_SPLIT, check, scan_inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def call(fn, t, **kw):
    return fn(t["x"], t["dt"], t["A"], t["B"], t["C"], **kw)


def prefill(seed, B, T, H, G, P, N, dtype, lens=None, carry=True, out_dtype=None, steps=(0.001, 0.1), D=True, bias=True, softplus=True,
            name=""):
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = T if lens is None else int(cu[-1])
    ns = B if lens is None else len(lens)
    t, r = scan_inputs(seed, (B, T), H, G, P, N, dtype, steps=steps)
    rng = np.random.default_rng(seed + 1)
    s64 = rng.standard_normal((ns, H, N, P)).astype(np.float32) if carry else None
    s0 = None if s64 is None else torch.from_numpy(s64).cuda()
    kw = dict(D=t["D"] if D else None, dt_bias=t["dt_bias"] if bias else None, dt_softplus=softplus, initial_state=s0,
              cu_seqlens=None if cu is None else torch.from_numpy(cu).cuda(), out_dtype=out_dtype)
    y, S, cs = call(kda.ssm_prefill, t, chunk_states=True, **kw)
    y_r, S_r, cs_r, _ = R.ssm_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"] if D else None, r["dt_bias"] if bias else None,
                                   softplus, s64, cu)
    split = TOL_SPLIT if dtype == BF else TOL[F32]
    check(f"{name} y", y, y_r, TOL[BF] if y.dtype == BF else split)
    check(f"{name} S", S, S_r, split)
    check(f"{name} chunk states", cs, cs_r, split)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_state_sizes(dtype, N, P):
    prefill(N * P, 2, 150, 2, 1, P, N, dtype, name=f"{N}x{P}")


@pytest.mark.parametrize("dtype,out", [(BF, F32), (F32, BF)])
def test_output_types(dtype, out):
    prefill(3, 1, 130, 3, 3, 64, 128, dtype, out_dtype=out, name=f"{dtype}->{out}")


@pytest.mark.parametrize("T", [0, 1, 2, 31, 32, 33, 63, 64, 65, 128, 257])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_lengths(T, dtype):
    prefill(10 + T, 2, T, 2, 2, 32, 32, dtype, name=f"T={T}")


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (8, 8), (10, 2), (20, 1), (6, 3)])
def test_head_layouts(H, G):
    prefill(30 + H, 1, 200, H, G, 64, 64, BF, name=f"H={H} G={G}")
    prefill(31 + H, 1, 70, H, G, 16, 16, F32, name=f"H={H} G={G}")


@pytest.mark.parametrize("lens", [[5, 0, 1, 64, 200, 65, 0], [700, 1, 333], [0], [1, 1, 1, 1], [0, 0, 1500]])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_packed(lens, dtype):
    prefill(40, 1, 0, 4, 2, 32, 64, dtype, lens=lens, name=f"{lens}")
    prefill(41, 1, 0, 4, 2, 32, 64, dtype, lens=lens, carry=False, name=f"{lens} no state")


@pytest.mark.parametrize("steps", [(1e-5, 1e-4), (0.5, 2.0), (5.0, 50.0)], ids=["slow", "fast", "extreme"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_decays(steps, dtype):
    """Slow decays (a long memory), and ones past the border of the factored
    form (a chunk decays by far more than 2^-56)."""
    prefill(50, 1, 300, 4, 1, 64, 64, dtype, steps=steps, name=f"steps {steps}")


def test_without_the_optional_arguments():
    t, r = scan_inputs(60, (2, 100), 4, 2, 32, 32, F32)
    dt = t["dt"].abs() * 0.1
    y, S = kda.ssm_prefill(t["x"], dt, t["A"], t["B"], t["C"])
    y_r, S_r, _, _ = R.ssm_scan(r["x"], dt.double().cpu().numpy(), r["A"], r["B"], r["C"])
    check("plain y", y, y_r, TOL[F32])
    check("plain S", S, S_r, TOL[F32])


def test_long_sequence_is_cut_and_agrees():
    """Few heads and many tokens: the segments' path."""
    prefill(70, 1, 3000, 2, 1, 64, 128, BF, name="3000 tokens")
    prefill(71, 1, 2000, 1, 1, 16, 32, F32, name="2000 tokens")


def test_state_in_place_and_continuation():
    """Two calls, the second continuing the first's state in place, equal the
    fp64 scan over both."""
    t, r = scan_inputs(80, (2, 192), 4, 2, 64, 64, BF)
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], dt_softplus=True)
    S = torch.zeros((2, 4, 64, 64), device="cuda")
    ys = []
    for a, b in ((0, 100), (100, 192)):
        y, S2 = kda.ssm_prefill(t["x"][:, a:b], t["dt"][:, a:b].contiguous(), t["A"], t["B"][:, a:b], t["C"][:, a:b], initial_state=S,
                                final_state=S, **kw)
        assert S2.data_ptr() == S.data_ptr()
        ys.append(y)
    y_r, S_r, _, _ = R.ssm_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"], r["dt_bias"], True)
    check("continued y", torch.cat(ys, 1), y_r, TOL[BF])
    check("continued S", S, S_r, TOL_SPLIT)


def test_malformed_offsets_write_nothing():
    t, _ = scan_inputs(81, (1, 100), 2, 1, 32, 32, BF)
    for bad in ([0, 60, 50, 100], [1, 100], [0, 90], [0, 200]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = torch.full((1, 100, 2, 32), 7.0, device="cuda", dtype=BF)
        S = torch.full((len(bad) - 1, 2, 32, 32), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(kda.ssm_prefill, t, cu_seqlens=cu, y=y, final_state=S, check_seqlens=False, device_status=status)
        assert int(status) == 6 and (y == 7).all() and (S == 7).all()
        with pytest.raises(kda.KDAError):
            call(kda.ssm_prefill, t, cu_seqlens=cu)


def test_same_results_from_run_to_run():
    t, _ = scan_inputs(82, (1, 3000), 4, 2, 64, 128, BF)
    a = call(kda.ssm_prefill, t, D=t["D"], dt_bias=t["dt_bias"], dt_softplus=True)
    b = call(kda.ssm_prefill, t, D=t["D"], dt_bias=t["dt_bias"], dt_softplus=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


# ------------------------------------------------------------------- tokens ----
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,P", [(16, 16), (16, 128), (32, 64), (64, 32), (128, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("m", [1, 3])
def test_decode(dtype, N, P, m):
    B, H, G = 3, 4, 2
    t, r = scan_inputs(N + P + m, (B, m), H, G, P, N, dtype)
    s64 = np.random.default_rng(1).standard_normal((B, H, N, P)).astype(np.float32)
    S = torch.from_numpy(s64).cuda()
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], dt_softplus=True)
    y_r, S_r, _, after = R.ssm_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"], r["dt_bias"], True, s64)
    keep = S.clone()
    y, none, ts = call(kda.ssm_decode, t, state=S, update_state=False, token_states=True, **kw)
    assert none is None and torch.equal(S, keep)
    check("token states", ts, after.reshape(B, m, H, N, P), TOL[F32])
    y2, S2, _ = call(kda.ssm_decode, t, state=S, **kw)
    assert S2.data_ptr() == S.data_ptr() and torch.equal(y, y2)
    check("y", y, y_r, TOL[dtype])
    check("S", S, S_r, TOL[F32])


@pytest.mark.parametrize("B", [1, 70])
def test_decode_steps_follow_a_prompt(B):
    t, r = scan_inputs(90, (B, 70), 4, 1, 64, 64, BF)
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], dt_softplus=True)
    cut = lambda a, b: (t["x"][:, a:b], t["dt"][:, a:b].contiguous(), t["A"], t["B"][:, a:b], t["C"][:, a:b])  # noqa: E731
    y0, S = kda.ssm_prefill(*cut(0, 66), **kw)
    ys = [y0] + [kda.ssm_decode(*cut(k, k + 1), S, **kw)[0] for k in range(66, 70)]
    y_r, S_r, _, _ = R.ssm_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"], r["dt_bias"], True)
    check("prompt and steps y", torch.cat(ys, 1), y_r, TOL[BF])
    check("prompt and steps S", S, S_r, TOL_SPLIT)


@pytest.mark.parametrize("dtype,steps", [(BF, (0.1, 0.2)), (F32, (0.2, 0.4))])
def test_chunks_of_wide_decays(dtype, steps):
    """Heads whose logs add up to -10 .. -230 (base 2) over a chunk: around the
    limits at which the state's scale is centred and the second form taken."""
    prefill(95, 2, 300, 24, 2, 32, 64, dtype, steps=steps, name=f"{dtype}")
    prefill(96, 1, 0, 24, 2, 64, 128, dtype, lens=[65, 130, 1, 200], steps=steps, out_dtype=F32, name=f"{dtype} packed")
