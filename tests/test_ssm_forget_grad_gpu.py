"""Gradients where a token of a huge step and x = 0 ends what came before it."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import sublayer as R
from sublayer_testutil import TOL, TOL_SPLIT, check, rounded
from test_ssm_mixed_steps_gpu import BF, F32, H, N, P, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("large", [1e4, 1e10, 1e20])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradients_around_tokens_that_forget_the_state(dtype, large):
    t, r, big = inputs(3, 2, 200, dtype, 0.02, large, share=0.05, clear=True)
    rng = np.random.default_rng(4)
    dy, dy64 = rounded(rng.standard_normal((2, 200, H, P)), dtype)
    d64 = rng.standard_normal((2, H, N, P)).astype(np.float32)
    got = kda.ssm_backward(*(t[k] for k in ("x", "dt", "A", "B", "C")), dy.cuda(), initial_state=t["state"],
                           d_final_state=torch.from_numpy(d64).cuda())
    want = R.ssm_scan_backward(*(r[k] for k in ("x", "dt", "A", "B", "C")), dy64, initial_state=r["state"], d_final=d64)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "d_initial")
    fp = TOL_SPLIT if dtype == BF else TOL[F32]
    for name, a, b in zip(names, got, want):
        if a is None:
            continue
        tol = TOL[BF] if a.dtype == BF else fp
        if name == "dx":  # dx of such a token is its huge step times what another's is: each kind by itself
            at = torch.from_numpy(big).cuda()
            check("dx of the huge steps", a[at], b[big], tol)
            check("dx", a[~at], b[~big], tol)
        else:
            check(name, a, b, tol)
