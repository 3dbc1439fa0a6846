"""Refusals of latent attention's entry points at the edges: calls that must be
turned down on the host, before a device is touched (the pointers are never
dereferenced)."""
import ctypes

import pytest

import gated_delta_rule_49_amd as kda
from test_latent_abi import APPEND, BAD_SHAPE, DECODE, FAR, NULL_ARG, PREFILL, UNSUPPORTED, L, fill  # noqa: F401


def test_precise_is_a_flag(L):  # noqa: F811
    for precise in (2, -1):
        a = fill(kda.LatentPrefillArgs, PREFILL, dict(precise=precise))
        assert L.kda_latent_prefill(ctypes.byref(a), None) == UNSUPPORTED and L.kda_latent_prefill_workspace_bytes(ctypes.byref(a)) == 0
    for precise in (0, 1):
        assert L.kda_latent_prefill_workspace_bytes(ctypes.byref(fill(kda.LatentPrefillArgs, PREFILL, dict(precise=precise)))) > 0


def test_workgroups_of_a_launch_are_whole(L):  # noqa: F811
    """A launch's threads are counted in whole workgroups: calls whose last one would make them 2^32 are refused."""
    def append(tokens):
        many = dict(B=1, num_seqs=1, T=tokens, kv_stride_b=0, kv_stride_t=0, kv=None)
        return L.kda_latent_append(ctypes.byref(fill(kda.LatentAppendArgs, APPEND, many)), None)
    assert all(append(2 ** 26 - k) == UNSUPPORTED for k in (0, 1, 2, 3))
    assert append(2 ** 26 - 4) == NULL_ARG  # past the sizes' check

    def rows(tokens):
        f = fill(kda.LatentPrefillArgs, PREFILL, dict(B=1, num_seqs=1, H=1, T=tokens, S=70, d_rope=16))
        g = kda.LatentBackwardArgs(f=f)
        return int(L.kda_latent_prefill_workspace_bytes(ctypes.byref(f))), int(L.kda_latent_backward_workspace_bytes(ctypes.byref(g)))
    for k in (1, 15):  # the gradients' statistics
        forward, backward = rows(2 ** 28 - k)
        assert forward > 0 and backward == 0
    assert min(rows(2 ** 28 - 16)) > 0


@pytest.mark.parametrize("over,status", [
    (dict(page_stride=160), BAD_SHAPE),  # page 1 begins with row 2 of page 0
    (dict(page_stride=312), BAD_SHAPE), (dict(row_stride=720, page_stride=720), BAD_SHAPE), (dict(row_stride=712, page_stride=80), BAD_SHAPE),
    # page after page with room between, all pages' first rows before their second, one page, pages of one row
    (dict(page_stride=328), NULL_ARG), (dict(row_stride=720, page_stride=80), NULL_ARG), (dict(num_pages=1, page_stride=0), NULL_ARG),
    (dict(page_size=1, row_stride=0, page_stride=80), NULL_ARG)])
def test_rows_of_the_cache_share_no_memory(L, over, status):  # noqa: F811
    assert L.kda_latent_append(ctypes.byref(fill(kda.LatentAppendArgs, APPEND, dict(over, kv=None))), None) == status


# every tensor in memory of its own, so that each case below lays one thing on another
APART = dict(PREFILL, B=1, num_seqs=2, q=1 * FAR, k_nope=2 * FAR, k_rope=3 * FAR, v=4 * FAR, o=5 * FAR, lse=6 * FAR, cu_seqlens_q=7 * FAR, cu_seqlens_k=8 * FAR,
             device_status=9 * FAR, workspace=10 * FAR)
GRADS = dict(d_o=11 * FAR, dq=12 * FAR, dk_nope=13 * FAR, dk_rope=14 * FAR, dv=15 * FAR, workspace=16 * FAR, workspace_bytes=1 << 40)


@pytest.mark.parametrize("over", [dict(o=7 * FAR), dict(lse=8 * FAR + 8), dict(o=8 * FAR - 16), dict(device_status=7 * FAR + 8), dict(device_status=1 * FAR), dict(device_status=5 * FAR + 4),
                                  dict(device_status=6 * FAR), dict(workspace=1 * FAR), dict(workspace=7 * FAR), dict(workspace=8 * FAR), dict(workspace=5 * FAR + 256),
                                  dict(workspace=6 * FAR), dict(workspace=9 * FAR), dict(workspace=4 * FAR)])
def test_prefill_memory_is_apart(L, over):  # noqa: F811
    assert L.kda_latent_prefill(ctypes.byref(fill(kda.LatentPrefillArgs, APART, over)), None) == BAD_SHAPE


@pytest.mark.parametrize("inner,over", [({}, dict(dq=7 * FAR)), ({}, dict(dv=8 * FAR)), ({}, dict(dk_rope=8 * FAR)), (dict(device_status=11 * FAR), {}), (dict(device_status=12 * FAR + 8), {}),
                                        (dict(device_status=7 * FAR), {}), (dict(device_status=6 * FAR), {})] +
                         [({}, dict(workspace=n * FAR)) for n in (1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 12, 13, 14, 15)])
def test_backward_memory_is_apart(L, inner, over):  # noqa: F811
    g = fill(kda.LatentBackwardArgs, GRADS, over)
    g.f = fill(kda.LatentPrefillArgs, APART, inner)
    assert L.kda_latent_backward(ctypes.byref(g), None) == BAD_SHAPE


@pytest.mark.parametrize("over", [dict(o=3 * FAR), dict(lse=4 * FAR + 4), dict(o=3 * FAR - 16), dict(device_status=4 * FAR), dict(device_status=3 * FAR + 4), dict(device_status=2 * FAR),
                                  dict(device_status=5 * FAR), dict(device_status=6 * FAR + 8)] + [dict(workspace=n * FAR) for n in range(1, 8)])
def test_decode_memory_is_apart(L, over):  # noqa: F811
    base = dict(DECODE, q=1 * FAR, cache=2 * FAR, page_table=3 * FAR, lengths=4 * FAR, o=5 * FAR, lse=6 * FAR, device_status=7 * FAR, workspace=8 * FAR)
    assert L.kda_latent_decode(ctypes.byref(fill(kda.LatentDecodeArgs, base, over)), None) == BAD_SHAPE
