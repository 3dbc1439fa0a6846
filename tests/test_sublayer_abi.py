"""Refusals of the sublayer's entry points: every call below must be turned
down on the host, before a device is touched (no GPU here, and the pointers
are never dereferenced)."""
import ctypes
import os
import subprocess

import pytest
import torch

import gated_delta_rule_49_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000
OK, NULL_ARG, BAD_SHAPE, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_49_amd import build
        build.build()
    return kda.lib()


def names(cls):
    return [f for f, _ in cls._fields_]


@pytest.mark.parametrize("cname,cls", [("kda_conv_backward_args", kda.ConvBackwardArgs), ("kda_ssm_args", kda.SsmArgs),
                                       ("kda_ssm_decode_args", kda.SsmDecodeArgs), ("kda_ssm_backward_args", kda.SsmBackwardArgs), ("kda_block_norm_args", kda.BlockNormArgs),
                                       ("kda_block_norm_backward_args", kda.BlockNormBackwardArgs)])
def test_struct_layout_matches_header(tmp_path, cname, cls):
    body = "".join(f'printf("%zu\\n", offsetof({cname}, {f}));' for f in names(cls))
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "kda.h"\nint main(void){{printf("%zu\\n", sizeof({cname}));{body}return 0;}}\n')
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in names(cls)]


def test_constants_match_header():
    src = open(os.path.join(ROOT, "include", "kda.h")).read()
    assert f"#define KDA_SSM_CHUNK {kda.SSM_CHUNK}\n" in src
    assert f"#define KDA_GATE_SIGMOID {kda.GATE_SIGMOID}\n" in src and f"#define KDA_GATE_SILU {kda.GATE_SILU}\n" in src


def fill(cls, base, over):
    a = cls(**base)
    for k, v in over.items():
        setattr(a, k, v)
    return a


CONV = dict(B=2, T=50, C=64, W=4, num_seqs=2, in_dtype=1, grad_dtype=1, x=FAKE, weight=FAKE, d_y=FAKE, dx=FAKE, dweight=FAKE,
            workspace=FAKE, workspace_bytes=1 << 30)


@pytest.mark.parametrize("over,status", [
    (dict(B=0), BAD_SHAPE), (dict(T=-1), BAD_SHAPE), (dict(num_seqs=3), BAD_SHAPE), (dict(W=0), BAD_SHAPE), (dict(C=0), BAD_SHAPE),
    (dict(W=9), UNSUPPORTED), (dict(C=60), UNSUPPORTED), (dict(in_dtype=2), UNSUPPORTED), (dict(grad_dtype=7), UNSUPPORTED),
    (dict(activation=2), UNSUPPORTED), (dict(cu_seqlens=FAKE), BAD_SHAPE), (dict(B=1, cu_seqlens=FAKE, num_seqs=0), BAD_SHAPE),
    (dict(T=1 << 26), UNSUPPORTED), (dict(x=None), NULL_ARG), (dict(d_y=None), NULL_ARG), (dict(dx=None), NULL_ARG),
    (dict(weight=None), NULL_ARG), (dict(dweight=None), NULL_ARG), (dict(workspace=None), NULL_ARG), (dict(x=FAKE + 8), UNSUPPORTED),
    (dict(workspace=FAKE + 16), BAD_SHAPE), (dict(workspace_bytes=0), TOO_SMALL)])
def test_conv_backward(L, over, status):
    assert L.kda_short_conv_backward(ctypes.byref(fill(kda.ConvBackwardArgs, CONV, over)), None) == status


SSM = dict(B=2, T=100, H=4, G=2, d_head=64, d_state=128, num_seqs=2, in_dtype=1, out_dtype=1, x_stride_b=51200, x_stride_t=512,
           b_stride_b=51200, b_stride_t=512, c_stride_b=51200, c_stride_t=512, x=FAKE, dt=FAKE, Bm=FAKE, Cm=FAKE, A=FAKE, y=FAKE,
           workspace=FAKE, workspace_bytes=1 << 40)
SSM_REFUSED = [
    (dict(H=0), BAD_SHAPE), (dict(G=0), BAD_SHAPE), (dict(G=3), BAD_SHAPE), (dict(d_head=0), BAD_SHAPE), (dict(d_state=-1), BAD_SHAPE),
    (dict(d_head=48), UNSUPPORTED), (dict(d_state=256), UNSUPPORTED), (dict(in_dtype=5), UNSUPPORTED), (dict(dt_softplus=2), UNSUPPORTED),
    (dict(x_stride_t=-8), BAD_SHAPE), (dict(x_stride_t=500), UNSUPPORTED), (dict(b_stride_b=4), UNSUPPORTED), (dict(c_stride_t=1), UNSUPPORTED),
    (dict(x=None), NULL_ARG), (dict(dt=None), NULL_ARG), (dict(Bm=None), NULL_ARG), (dict(Cm=None), NULL_ARG), (dict(A=None), NULL_ARG),
    (dict(x=FAKE + 2), UNSUPPORTED), (dict(Bm=FAKE + 8), UNSUPPORTED), (dict(initial_state=FAKE + 4), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", SSM_REFUSED + [
    (dict(B=0), BAD_SHAPE), (dict(T=-1), BAD_SHAPE), (dict(num_seqs=1), BAD_SHAPE), (dict(cu_seqlens=FAKE), BAD_SHAPE),
    (dict(T=1 << 29), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED), (dict(y=None), NULL_ARG), (dict(workspace=None), NULL_ARG),
    (dict(workspace=FAKE + 128), BAD_SHAPE), (dict(workspace_bytes=8), TOO_SMALL), (dict(chunk_states=FAKE + 4), UNSUPPORTED)])
def test_scan(L, over, status):
    a = fill(kda.SsmArgs, SSM, over)
    assert L.kda_ssm_prefill(ctypes.byref(a), None) == status
    if status in (BAD_SHAPE, UNSUPPORTED) and not any(k in over for k in ("x", "Bm", "initial_state", "chunk_states", "workspace")):
        assert L.kda_ssm_workspace_bytes(ctypes.byref(a)) == 0 and L.kda_ssm_max_chunks(ctypes.byref(a)) == 0


def test_scan_sizes(L):
    a = fill(kda.SsmArgs, SSM, {})
    assert L.kda_ssm_max_chunks(ctypes.byref(a)) == 4 and L.kda_ssm_workspace_bytes(ctypes.byref(a)) > 0
    a = fill(kda.SsmArgs, SSM, dict(B=1, cu_seqlens=FAKE, num_seqs=5))
    assert L.kda_ssm_max_chunks(ctypes.byref(a)) == 7


SSM_GRAD = dict({k: v for k, v in SSM.items() if k not in ("out_dtype", "y")}, d_y=FAKE, dx=FAKE, ddt=FAKE, dB=FAKE, dC=FAKE, dA=FAKE)


@pytest.mark.parametrize("over,status", SSM_REFUSED + [
    (dict(B=0), BAD_SHAPE), (dict(T=-1), BAD_SHAPE), (dict(num_seqs=1), BAD_SHAPE), (dict(cu_seqlens=FAKE), BAD_SHAPE),
    (dict(T=1 << 29), UNSUPPORTED), (dict(d_y=None), NULL_ARG), (dict(dx=None), NULL_ARG), (dict(ddt=None), NULL_ARG), (dict(dB=None), NULL_ARG),
    (dict(dC=None), NULL_ARG), (dict(dA=None), NULL_ARG), (dict(dD=FAKE), BAD_SHAPE), (dict(ddt_bias=FAKE), BAD_SHAPE),
    (dict(workspace=None), NULL_ARG), (dict(workspace=FAKE + 128), BAD_SHAPE), (dict(workspace_bytes=8), TOO_SMALL),
    (dict(d_y=FAKE + 8), UNSUPPORTED), (dict(d_initial_state=FAKE + 4), UNSUPPORTED), (dict(dB=FAKE + 2), UNSUPPORTED)])
def test_scan_backward(L, over, status):
    assert L.kda_ssm_backward(ctypes.byref(fill(kda.SsmBackwardArgs, SSM_GRAD, over)), None) == status


DECODE = dict({k: v for k, v in SSM.items() if k not in ("T", "num_seqs", "workspace", "workspace_bytes")}, n_tokens=2, initial_state=FAKE)


@pytest.mark.parametrize("over,status", SSM_REFUSED + [
    (dict(B=-1), BAD_SHAPE), (dict(n_tokens=0), BAD_SHAPE), (dict(y=None), NULL_ARG), (dict(initial_state=None), NULL_ARG),
    (dict(final_state=FAKE + 4), UNSUPPORTED), (dict(token_states=FAKE + 8), UNSUPPORTED), (dict(B=1 << 30), UNSUPPORTED)])
def test_tokens(L, over, status):
    assert L.kda_ssm_decode(ctypes.byref(fill(kda.SsmDecodeArgs, DECODE, over)), None) == status


def test_no_sequences_is_no_work(L):
    assert L.kda_ssm_decode(ctypes.byref(fill(kda.SsmDecodeArgs, DECODE, dict(B=0))), None) == OK


NORM = dict(rows=10, dim=256, group=64, dtype=1, eps=1e-6, x_stride=256, gate_stride=256, residual_stride=256, x=FAKE, out=FAKE)
NORM_REFUSED = [(dict(rows=-1), BAD_SHAPE), (dict(dim=0), BAD_SHAPE), (dict(group=0), BAD_SHAPE), (dict(group=60), BAD_SHAPE),
                (dict(dim=16448), UNSUPPORTED), (dict(rows=1 << 33), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
                (dict(gate_activation=2), UNSUPPORTED), (dict(eps=-1.0), BAD_SHAPE), (dict(eps=float("nan")), BAD_SHAPE), (dict(x=None), NULL_ARG),
                (dict(x_stride=100), BAD_SHAPE), (dict(gate=FAKE, gate_stride=-256), BAD_SHAPE), (dict(residual=FAKE, residual_stride=8), BAD_SHAPE)]


@pytest.mark.parametrize("over,status", NORM_REFUSED + [(dict(out=None), NULL_ARG), (dict(pre_weight=FAKE), NULL_ARG), (dict(normed=FAKE), BAD_SHAPE)])
def test_block_norm(L, over, status):
    assert L.kda_block_norm(ctypes.byref(fill(kda.BlockNormArgs, NORM, over)), None) == status


def test_no_rows_is_no_work(L):
    assert L.kda_block_norm(ctypes.byref(fill(kda.BlockNormArgs, NORM, dict(rows=0))), None) == OK


@pytest.mark.parametrize("inner,over,status", [(o, {}, s) for o, s in NORM_REFUSED] + [
    ({}, dict(dx=None), NULL_ARG), ({}, dict(workspace=None), NULL_ARG), ({}, dict(workspace=FAKE + 8), BAD_SHAPE),
    ({}, dict(workspace_bytes=4), TOO_SMALL), ({}, dict(d_normed=FAKE), BAD_SHAPE), ({}, dict(dgate=FAKE), BAD_SHAPE),
    ({}, dict(dresidual=FAKE), BAD_SHAPE), ({}, dict(dscale=FAKE), BAD_SHAPE), ({}, dict(dpost_weight=FAKE), BAD_SHAPE),
    ({}, dict(dpre_weight=FAKE), BAD_SHAPE)])
def test_block_norm_backward(L, inner, over, status):
    a = fill(kda.BlockNormBackwardArgs, dict(dx=FAKE, workspace=FAKE, workspace_bytes=1 << 40), over)
    a.f = fill(kda.BlockNormArgs, NORM, inner)
    assert L.kda_block_norm_backward(ctypes.byref(a), None) == status


def test_null_arguments(L):
    for fn in (L.kda_short_conv_backward, L.kda_ssm_prefill, L.kda_ssm_decode, L.kda_ssm_backward, L.kda_block_norm, L.kda_block_norm_backward):
        assert fn(None, None) == NULL_ARG
    for fn in (L.kda_short_conv_backward_workspace_bytes, L.kda_ssm_workspace_bytes, L.kda_ssm_max_chunks, L.kda_ssm_backward_workspace_bytes,
               L.kda_block_norm_backward_workspace_bytes):
        assert fn(None) == 0


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        kda.ssm_prefill(z(1, 4, 2, 16), z(1, 4, 2), z(2), z(1, 4, 1, 16), z(1, 4, 1, 16))
    with pytest.raises(ValueError, match="GPU"):
        kda.ssm_backward(z(1, 4, 2, 16), z(1, 4, 2), z(2), z(1, 4, 1, 16), z(1, 4, 1, 16), z(1, 4, 2, 16))
    with pytest.raises(ValueError, match="GPU"):
        kda.ssm_decode(z(1, 4, 2, 16), z(1, 4, 2), z(2), z(1, 4, 1, 16), z(1, 4, 1, 16), z(1, 2, 16, 16))
    with pytest.raises(ValueError, match="GPU"):
        kda.short_conv_backward(z(1, 4, 8), z(8, 4), z(1, 4, 8))
    with pytest.raises(ValueError, match="GPU"):
        kda.block_norm(z(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        kda.block_norm_backward(z(4, 8), z(4, 8))
