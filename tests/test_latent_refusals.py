"""Refusals of latent attention's entry points at the edges: calls that must be
turned down on the host, before a device is touched (the pointers are never
dereferenced)."""
import ctypes

import pytest

import gated_delta_rule_49_amd as kda
from test_latent_abi import APPEND, BAD_SHAPE, DECODE, FAKE, FAR, OK, PREFILL, UNSUPPORTED, L, fill  # noqa: F401


def test_precise_is_a_flag(L):  # noqa: F811
    for precise in (2, -1):
        a = fill(kda.LatentPrefillArgs, PREFILL, dict(precise=precise))
        assert L.kda_latent_prefill(ctypes.byref(a), None) == UNSUPPORTED and L.kda_latent_prefill_workspace_bytes(ctypes.byref(a)) == 0
    for precise in (0, 1):
        assert L.kda_latent_prefill_workspace_bytes(ctypes.byref(fill(kda.LatentPrefillArgs, PREFILL, dict(precise=precise)))) > 0
