"""Refusals of latent attention's entry points: every call below must be turned
down on the host, before a device is touched (no GPU here, and the pointers are
never dereferenced); and the fp64 forms against closed forms and differences."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import latent as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x100000
FAR = 1 << 32  # memory of its own
OK, NULL_ARG, BAD_SHAPE, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_49_amd import build
        build.build()
    return kda.lib()


@pytest.mark.parametrize("cname,cls", [("kda_rotary_args", kda.RotaryArgs), ("kda_latent_append_args", kda.LatentAppendArgs),
                                       ("kda_latent_prefill_args", kda.LatentPrefillArgs), ("kda_latent_backward_args", kda.LatentBackwardArgs),
                                       ("kda_latent_decode_args", kda.LatentDecodeArgs)])
def test_struct_layout_matches_header(tmp_path, cname, cls):
    fields = [f for f, _ in cls._fields_]
    body = "".join(f'printf("%zu\\n", offsetof({cname}, {f}));' for f in fields)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "kda.h"\nint main(void){{printf("%zu\\n", sizeof({cname}));{body}return 0;}}\n')
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def fill(cls, base, over):
    a = cls(**base)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_new_status_has_a_text(L):
    assert b"page" in L.kda_status_string(9)


ROTARY = dict(B=2, T=5, H=4, D=64, rotary_dim=32, offset=32, interleaved=1, dtype=1, magnitude=1.0, x_stride_b=5 * 256, x_stride_t=256, x_stride_h=64,
              out_stride_b=5 * 256, out_stride_t=256, out_stride_h=64, x=FAKE, freqs=FAKE, out=FAKE << 8)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(rotary_dim=31), BAD_SHAPE), (dict(rotary_dim=-2), BAD_SHAPE), (dict(offset=33), BAD_SHAPE),
    (dict(offset=-1), BAD_SHAPE), (dict(dtype=2), UNSUPPORTED), (dict(interleaved=2), UNSUPPORTED), (dict(D=8192, offset=0), UNSUPPORTED),
    (dict(T=2 ** 30), UNSUPPORTED), (dict(x_stride_t=-256), BAD_SHAPE), (dict(x=None), NULL_ARG), (dict(out=None), NULL_ARG), (dict(freqs=None), NULL_ARG),
    (dict(x=FAKE + 1), UNSUPPORTED), (dict(out_stride_h=32), BAD_SHAPE), (dict(out_stride_b=0), BAD_SHAPE), (dict(out_stride_t=255), BAD_SHAPE),
    # the same memory with other strides, or shifted
    (dict(out=FAKE, out_stride_t=512, out_stride_b=5 * 512), BAD_SHAPE), (dict(out=FAKE + 64), BAD_SHAPE), (dict(out=FAKE + 2 * (2 * 5 * 256 - 1)), BAD_SHAPE)])
def test_rotary(L, over, status):
    for fn in (L.kda_rotary, L.kda_rotary_backward):
        assert fn(ctypes.byref(fill(kda.RotaryArgs, ROTARY, over)), None) == status


def test_no_work(L):
    assert L.kda_rotary(ctypes.byref(fill(kda.RotaryArgs, ROTARY, dict(T=0, x=None, out=None))), None) == OK
    assert L.kda_latent_append(ctypes.byref(fill(kda.LatentAppendArgs, APPEND, dict(T=0))), None) == OK
    assert L.kda_latent_prefill(ctypes.byref(fill(kda.LatentPrefillArgs, PREFILL, dict(T=0))), None) == OK
    assert L.kda_latent_decode(ctypes.byref(fill(kda.LatentDecodeArgs, DECODE, dict(B=0))), None) == OK


APPEND = dict(B=2, T=3, num_seqs=2, d_latent=64, d_rope=16, interleaved=0, dtype=1, num_pages=9, page_size=4, max_pages=3, eps=1e-6, magnitude=1.0,
              kv_stride_b=3 * 80, kv_stride_t=80, page_stride=320, row_stride=80, table_stride=3, kv=FAKE, lengths=FAKE, page_table=FAKE, cache=FAKE << 4)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), BAD_SHAPE), (dict(num_seqs=3), BAD_SHAPE), (dict(cu_seqlens=FAKE), BAD_SHAPE), (dict(d_latent=0), BAD_SHAPE), (dict(d_latent=60), UNSUPPORTED),
    (dict(d_latent=2056), UNSUPPORTED), (dict(d_rope=4), UNSUPPORTED), (dict(d_rope=264), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(interleaved=-1), UNSUPPORTED),
    (dict(eps=-1.0), BAD_SHAPE), (dict(eps=math.nan), BAD_SHAPE), (dict(num_pages=0), BAD_SHAPE), (dict(page_size=0), BAD_SHAPE), (dict(max_pages=0), BAD_SHAPE),
    (dict(max_pages=2 ** 30), UNSUPPORTED), (dict(page_stride=-8), BAD_SHAPE), (dict(row_stride=72), BAD_SHAPE), (dict(page_stride=72), BAD_SHAPE),
    (dict(row_stride=84), UNSUPPORTED), (dict(kv_stride_t=81), UNSUPPORTED), (dict(kv=None), NULL_ARG), (dict(cache=None), NULL_ARG), (dict(page_table=None), NULL_ARG),
    (dict(lengths=None), NULL_ARG), (dict(kv=FAKE + 8), UNSUPPORTED), (dict(cache=FAKE + 64), BAD_SHAPE), (dict(rows=FAKE), BAD_SHAPE), (dict(rows=FAKE << 4), BAD_SHAPE)])
def test_append(L, over, status):
    assert L.kda_latent_append(ctypes.byref(fill(kda.LatentAppendArgs, APPEND, over)), None) == status


PREFILL = dict(B=2, T=50, S=70, H=4, d_nope=128, d_rope=64, d_v=128, num_seqs=2, in_dtype=1, out_dtype=1, causal=1, scale=0.1, q_stride_b=50 * 768, q_stride_t=768,
               q_stride_h=192, k_stride_b=70 * 1024, k_stride_t=1024, k_stride_h=256, r_stride_b=70 * 64, r_stride_t=64, v_stride_b=70 * 1024, v_stride_t=1024,
               v_stride_h=256, q=FAKE, k_nope=FAKE, k_rope=FAKE, v=FAKE, o=FAR, lse=2 * FAR, workspace=FAKE, workspace_bytes=1 << 40)
PREFILL_REFUSED = [
    (dict(B=0), BAD_SHAPE), (dict(T=-1), BAD_SHAPE), (dict(S=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(num_seqs=1), BAD_SHAPE), (dict(d_nope=0), BAD_SHAPE),
    (dict(d_rope=-8), BAD_SHAPE), (dict(d_v=0), BAD_SHAPE), (dict(d_nope=100), UNSUPPORTED), (dict(d_nope=136), UNSUPPORTED), (dict(d_v=136), UNSUPPORTED),
    (dict(d_v=60), UNSUPPORTED), (dict(d_rope=12), UNSUPPORTED), (dict(in_dtype=2), UNSUPPORTED), (dict(out_dtype=-1), UNSUPPORTED), (dict(causal=2), UNSUPPORTED),
    (dict(cu_seqlens_q=FAKE), BAD_SHAPE), (dict(cu_seqlens_k=FAKE), BAD_SHAPE), (dict(cu_seqlens_q=FAKE, cu_seqlens_k=FAKE), BAD_SHAPE),
    (dict(T=2 ** 30), UNSUPPORTED), (dict(H=2 ** 22), UNSUPPORTED), (dict(q_stride_t=-8), BAD_SHAPE), (dict(k_stride_h=250), UNSUPPORTED), (dict(v_stride_t=1 << 23), UNSUPPORTED),
    (dict(q=None), NULL_ARG), (dict(k_nope=None), NULL_ARG), (dict(k_rope=None), NULL_ARG), (dict(v=None), NULL_ARG), (dict(o=None), NULL_ARG), (dict(lse=None), NULL_ARG),
    (dict(q=FAKE + 8), UNSUPPORTED), (dict(k_rope=FAKE + 4), UNSUPPORTED), (dict(o=FAKE + 2), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", PREFILL_REFUSED + [(dict(workspace=None), NULL_ARG), (dict(workspace=FAKE + 16), BAD_SHAPE), (dict(workspace_bytes=8), TOO_SMALL),
                                                          (dict(o=FAKE + 1024), BAD_SHAPE), (dict(lse=FAKE + 4), BAD_SHAPE), (dict(lse=FAR + 64), BAD_SHAPE)])
def test_prefill(L, over, status):
    a = fill(kda.LatentPrefillArgs, PREFILL, over)
    assert L.kda_latent_prefill(ctypes.byref(a), None) == status


@pytest.mark.parametrize("inner,over,status", [(o, {}, s) for o, s in PREFILL_REFUSED] + [
    ({}, dict(d_o=None), NULL_ARG), ({}, dict(dq=None), NULL_ARG), ({}, dict(dk_nope=None), NULL_ARG), ({}, dict(dk_rope=None), NULL_ARG),
    ({}, dict(dv=None), NULL_ARG), ({}, dict(dq=FAKE + 8), UNSUPPORTED), ({}, dict(d_o=FAKE + 2), UNSUPPORTED), (dict(d_rope=0, k_rope=None), {}, BAD_SHAPE),
    ({}, dict(o_stride_h=-8), BAD_SHAPE), ({}, dict(o_stride_t=4), UNSUPPORTED), ({}, dict(d_o_stride_t=1 << 23), UNSUPPORTED), ({}, dict(lse_stride_b=-1), BAD_SHAPE),
    ({}, dict(dq=FAKE), BAD_SHAPE), ({}, dict(dk_rope=FAR), BAD_SHAPE), ({}, dict(dv=4 * FAR + 16), BAD_SHAPE), ({}, dict(dk_nope=2 * FAR), BAD_SHAPE),
    ({}, dict(workspace=None), NULL_ARG), ({}, dict(workspace=FAKE + 8), BAD_SHAPE), ({}, dict(workspace_bytes=1000), TOO_SMALL)])
def test_backward(L, inner, over, status):
    a = fill(kda.LatentBackwardArgs, dict(d_o=FAKE, dq=3 * FAR, dk_nope=4 * FAR, dk_rope=5 * FAR, dv=6 * FAR, workspace=FAKE, workspace_bytes=1 << 40), over)
    a.f = fill(kda.LatentPrefillArgs, PREFILL, inner)
    assert L.kda_latent_backward(ctypes.byref(a), None) == status


DECODE = dict(B=3, H=8, n_tokens=2, d_latent=512, d_rope=64, in_dtype=1, out_dtype=1, num_pages=40, page_size=16, max_pages=9, scale=0.1, q_stride_b=2 * 8 * 576,
              q_stride_t=8 * 576, q_stride_h=576, page_stride=16 * 576, row_stride=576, table_stride=9, q=FAKE, cache=FAKE, page_table=FAKE, lengths=FAKE, o=FAR, lse=2 * FAR,
              workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(n_tokens=0), BAD_SHAPE), (dict(d_latent=0), BAD_SHAPE), (dict(d_rope=-8), BAD_SHAPE),
    (dict(d_latent=500), UNSUPPORTED), (dict(d_latent=520), UNSUPPORTED), (dict(d_rope=72), UNSUPPORTED), (dict(in_dtype=2), UNSUPPORTED), (dict(out_dtype=5), UNSUPPORTED),
    (dict(B=65537), UNSUPPORTED), (dict(H=2 ** 22, n_tokens=4), UNSUPPORTED), (dict(num_pages=0), BAD_SHAPE), (dict(page_size=0), BAD_SHAPE), (dict(max_pages=0), BAD_SHAPE),
    (dict(max_pages=2 ** 28), UNSUPPORTED), (dict(row_stride=568), BAD_SHAPE), (dict(row_stride=580), UNSUPPORTED), (dict(page_stride=0), BAD_SHAPE),
    (dict(q_stride_h=-576), BAD_SHAPE), (dict(q_stride_t=577), UNSUPPORTED), (dict(table_stride=-1), BAD_SHAPE), (dict(q=None), NULL_ARG), (dict(cache=None), NULL_ARG),
    (dict(page_table=None), NULL_ARG), (dict(lengths=None), NULL_ARG), (dict(o=None), NULL_ARG), (dict(lse=None), NULL_ARG), (dict(cache=FAKE + 8), UNSUPPORTED),
    (dict(o=FAKE), BAD_SHAPE), (dict(lse=FAKE + 512), BAD_SHAPE), (dict(lse=FAR + 32), BAD_SHAPE),
    (dict(workspace=None), NULL_ARG), (dict(workspace=FAKE + 64), BAD_SHAPE), (dict(workspace_bytes=64), TOO_SMALL)])
def test_decode(L, over, status):
    assert L.kda_latent_decode(ctypes.byref(fill(kda.LatentDecodeArgs, DECODE, over)), None) == status


def test_null_arguments(L):
    for fn in (L.kda_rotary, L.kda_rotary_backward, L.kda_latent_append, L.kda_latent_prefill, L.kda_latent_backward, L.kda_latent_decode):
        assert fn(None, None) == NULL_ARG
    for fn in (L.kda_latent_prefill_workspace_bytes, L.kda_latent_backward_workspace_bytes, L.kda_latent_decode_workspace_bytes):
        assert fn(None) == 0


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    i32, f64 = dict(dtype=torch.int32), dict(dtype=torch.float64)
    q, kn, kr, v = z(1, 4, 2, 24), z(1, 4, 2, 16), z(1, 4, 8), z(1, 4, 2, 16)
    with pytest.raises(ValueError, match="GPU"):
        kda.rotary(q, z(4, **f64))
    with pytest.raises(ValueError, match="GPU"):
        kda.rotary_backward(q, z(4, **f64))
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_prefill(q, kn, kr, v)
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_backward(q, kn, kr, v, v, z(1, 4, 2), v)
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_append(z(2, 1, 24), z(3, 4, 24), z(2, 2, **i32), z(2, **i32), 16)
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_decode(z(2, 1, 2, 24), z(3, 4, 24), z(2, 2, **i32), z(2, **i32), 16, 0.2)


# ------------------------------------------------------------- frequencies ----
def test_frequencies():
    f, m = kda.rotary_frequencies(8, base=100.0)
    assert m == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64), rtol=1e-14)
    g, _ = kda.rotary_frequencies(8, base=100.0, scaling="linear", factor=4)
    assert torch.equal(g, f / 4)
    g, _ = kda.rotary_frequencies(8, base=100.0, scaling="base", factor=4)
    assert g[0] == f[0] and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12  # the fastest stays, the slowest is 4 times slower
    f, _ = kda.rotary_frequencies(64)
    g, m = kda.rotary_frequencies(64, scaling="turns", factor=8, original_length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    assert bool((g[1:] < g[:-1]).all()) and m == 1 + 0.1 * math.log(8)
    assert kda.rotary_frequencies(64, scaling="turns", factor=1)[1] == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="cubic"), dict(rotary_dim=8, scaling="linear", factor=0.5),
                                dict(rotary_dim=2, scaling="base", factor=2.0), dict(rotary_dim=8, scaling="turns", fast_turns=1.0, slow_turns=1.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        kda.rotary_frequencies(**kw)


# ------------------------------------------------------------ the fp64 forms ----
def test_rotary_form_is_a_rotation():
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((6, 2, 12)), np.array([1.0, 0.1, 0.01])
    for inter in (False, True):
        y = R.rotary(x, np.arange(6) + 5, f, 4, inter)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1)) and np.array_equal(y[..., :4], x[..., :4]) and np.array_equal(y[..., 10:], x[..., 10:])
        assert np.allclose(R.rotary(y, np.arange(6) + 5, f, 4, inter, back=True), x)
        # scores depend on the distance alone
        a, b = R.rotary(x[:1], [3], f, 4, inter), R.rotary(x[1:2], [10], f, 4, inter)
        c, d = R.rotary(x[:1], [103], f, 4, inter), R.rotary(x[1:2], [110], f, 4, inter)
        assert np.allclose((a * b).sum(-1), (c * d).sum(-1))
    one = R.rotary(np.array([[[1.0, 0.0]]]), [1], [math.pi / 2], 0, True, 2.0)
    assert np.allclose(one, [[[0.0, 2.0]]])


def test_attention_form():
    # equal scores: the mean of what is seen
    q, k, v = np.zeros((3, 2)), np.ones((4, 2)), np.arange(4.0)[:, None]
    o, lse, _ = R.attention(q, k, v, 1.0, True)
    assert np.allclose(o[:, 0], [0.5, 1.0, 1.5]) and np.allclose(lse, np.log([2, 3, 4]))
    o, lse, _ = R.attention(np.zeros((3, 2)), k[:1], v[:1] + 7, 1.0, True)  # more queries than keys
    assert np.allclose(o[:, 0], [0, 0, 7]) and np.array_equal(lse, [-np.inf, -np.inf, 0])


def test_attention_gradients_against_differences():
    rng = np.random.default_rng(2)
    tq, tk, H, dn, dr, dv = 3, 5, 2, 4, 2, 3
    x = [rng.standard_normal(s) for s in ((tq, H, dn + dr), (tk, H, dn), (tk, dr), (tk, H, dv))]
    d_o = rng.standard_normal((tq, H, dv))
    for causal in (True, False):
        grads = R.prefill_backward(*x, d_o, 0.4, causal)
        for n, g in enumerate(grads):
            for at in np.ndindex(*g.shape):
                y = [a.copy() for a in x]
                y[n][at] += 1e-6
                up = (R.prefill(*y, 0.4, causal)[0] * d_o).sum()
                y[n][at] -= 2e-6
                assert abs((up - (R.prefill(*y, 0.4, causal)[0] * d_o).sum()) / 2e-6 - g[at]) < 1e-7


def test_absorbed_form_is_the_expanded_one():
    """Queries carried through the keys' up-projection give the expanded form's scores, their latent results its outputs."""
    rng = np.random.default_rng(3)
    n, H, dc, dn, dr, dv, m = 7, 3, 10, 4, 2, 5, 2
    rows, up_k, up_v = rng.standard_normal((n, dc + dr)), rng.standard_normal((H, dn, dc)), rng.standard_normal((H, dv, dc))
    q = rng.standard_normal((m, H, dn + dr))
    k_nope, v = np.einsum("hdc,tc->thd", up_k, rows[:, :dc]), np.einsum("hdc,tc->thd", up_v, rows[:, :dc])
    o, lse = R.prefill(q, k_nope, rows[:, dc:], v, 0.3)
    q_latent = np.concatenate([np.einsum("mhd,hdc->mhc", q[..., :dn], up_k), q[..., dn:]], -1)
    o2, lse2 = R.decode(q_latent, rows, dc, 0.3)
    assert np.allclose(np.einsum("mhc,hdc->mhd", o2, up_v), o) and np.allclose(lse2, lse)


def test_limits_of_a_launch(L):
    """What would pass 2^32 threads in a launch is refused; what comes close is sized."""
    def prefill(**over):
        return int(L.kda_latent_prefill_workspace_bytes(ctypes.byref(fill(kda.LatentPrefillArgs, PREFILL, over))))
    assert prefill(T=2 ** 24, S=2 ** 24, H=4, B=3, num_seqs=3) > 0 and prefill(T=2 ** 24, S=2 ** 24, H=4, B=4, num_seqs=4) == 0
    assert prefill(B=2 ** 19, num_seqs=2 ** 19, T=1, S=1) > 0 and prefill(B=2 ** 19 + 1, num_seqs=2 ** 19 + 1, T=1, S=1) == 0
    assert prefill(B=1, num_seqs=1, H=1, T=1, S=2 ** 27) == 0 and prefill(B=1, num_seqs=1, H=1, T=1, S=2 ** 26) > 0  # 64 channels of dk_rope each
    many = dict(B=1, num_seqs=1, T=2 ** 26, kv_stride_b=0)
    assert L.kda_latent_append(ctypes.byref(fill(kda.LatentAppendArgs, APPEND, many)), None) == UNSUPPORTED
    rows = dict(max_pages=1, page_size=2 ** 31 - 1)
    assert L.kda_latent_append(ctypes.byref(fill(kda.LatentAppendArgs, APPEND, rows)), None) == UNSUPPORTED
    assert L.kda_latent_decode(ctypes.byref(fill(kda.LatentDecodeArgs, DECODE, rows)), None) == UNSUPPORTED
