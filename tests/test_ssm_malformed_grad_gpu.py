"""With malformed offsets none of the gradients' kernels writes an output:
buffers of a known value stay as they were, with few heads (so that the group's
heads and the sequences are split) and with many."""
import ctypes

import pytest
import torch

import gated_delta_rule_49_amd as kda
from sublayer_testutil import scan_inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, P, N = 1000, 32, 32


@pytest.mark.parametrize("offsets", [[0, 600, 500, T], [1, T], [0, T - 10], [0, T + 100], [0, 10, -5, T], [0, 2 ** 31 - 1, T]])
@pytest.mark.parametrize("H,G", [(4, 1), (24, 12)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_malformed_offsets_leave_every_gradient(dtype, H, G, offsets):
    t, _ = scan_inputs(1, (1, T), H, G, P, N, dtype)
    x, B, C = (t[k].contiguous() for k in ("x", "B", "C"))
    seqs = len(offsets) - 1
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    state = torch.zeros(seqs, H, N, P, device="cuda")
    full = lambda shape, kind: torch.full(shape, 7.0, dtype=kind, device="cuda")  # noqa: E731
    out = dict(dx=full(x.shape, dtype), ddt=full((1, T, H), dtype), dB=full(B.shape, dtype), dC=full(C.shape, dtype), dA=full((H,), F32),
               dD=full((H,), F32), ddt_bias=full((H,), F32), d_initial_state=full(state.shape, F32))
    a = kda.SsmBackwardArgs(B=1, T=T, H=H, G=G, d_head=P, d_state=N, num_seqs=seqs, in_dtype=int(dtype == BF), dt_softplus=1,
                            x_stride_t=H * P, b_stride_t=G * N, c_stride_t=G * N, cu_seqlens=cu.data_ptr())
    inputs = dict(x=x, dt=t["dt"], Bm=B, Cm=C, A=t["A"], D=t["D"], dt_bias=t["dt_bias"], initial_state=state, d_y=x, d_final_state=state)
    for name, v in {**inputs, **out}.items():
        setattr(a, name, v.data_ptr())
    L = kda.lib()
    ws = torch.empty(int(L.kda_ssm_backward_workspace_bytes(ctypes.byref(a))), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    assert L.kda_ssm_backward(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert int(ws[:4].view(torch.int32)) == 6
    for name, v in out.items():
        assert (v == 7).all(), name
