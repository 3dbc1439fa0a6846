"""block_norm refuses outputs that share memory with each other, or with a part
of an input whose rows other workgroups still read (no GPU here, and the
pointers are never dereferenced)."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_49_amd as kda

OUT, BAD_SHAPE = 0x100000, 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_49_amd import build
        build.build()
    return kda.lib()


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2)])
@pytest.mark.parametrize("rows", [1, 10])
def test_out_and_normed_apart(L, rows, dtype, size):
    plane = rows * 256 * size
    for shift in (0, 16, plane - 16, 16 - plane, -16):
        a = kda.BlockNormArgs(rows=rows, dim=256, group=256, dtype=dtype, eps=1e-6, x_stride=256, x=0x1000, pre_weight=0x2000, out=OUT,
                              normed=OUT + shift)
        assert L.kda_block_norm(ctypes.byref(a), None) == BAD_SHAPE, shift


@pytest.mark.parametrize("name", ["x", "gate", "residual"])
@pytest.mark.parametrize("to", ["out", "normed"])
def test_outputs_apart_from_parts_of_inputs(L, name, to):
    # 10 rows of 256 fp32: one row before and behind, half a row, the same rows
    # with a wider stride, one row for all
    for shift, stride in ((1024, 256), (-1024, 256), (512, 256), (0, 512), (0, 0), (9 * 1024, 256)):
        a = kda.BlockNormArgs(rows=10, dim=256, group=256, dtype=0, eps=1e-6, x_stride=256, gate_stride=256, residual_stride=256, x=0x1000000,
                              gate=0x2000000, residual=0x3000000, pre_weight=0x2000, out=0x4000000, normed=0x5000000)
        setattr(a, name + "_stride", stride)
        setattr(a, to, getattr(a, name) + shift)
        assert L.kda_block_norm(ctypes.byref(a), None) == BAD_SHAPE, (shift, stride)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_on_an_input_s_rows(dtype):
    """Allowed, and the same results as with buffers of their own; neighbouring
    memory is not an overlap."""
    buf = torch.randn(30, 256, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    w = torch.rand(256, device="cuda") + 0.5
    for o, m in ((0, 1), (1, 0), (1, 2)):
        x, r, free = (b.clone() for b in buf.chunk(3))
        want = kda.block_norm(x, residual=r, post_weight=w, pre_weight=w)
        got = kda.block_norm(x, residual=r, post_weight=w, pre_weight=w, out=(x, r, free)[o], normed=(x, r, free)[m])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = buf[:10].clone()
    want = kda.block_norm(x, residual=buf[:10], post_weight=w)[0]
    got = kda.block_norm(x, residual=buf[:10], post_weight=w, out=buf[10:20])[0]
    assert torch.equal(got, want)
