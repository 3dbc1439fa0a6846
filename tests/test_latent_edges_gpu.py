"""Calls of the latent attention layer at the edges that its operators allow:
padded batches, calls in each of the fp32 kernels, a training step's whole
gradients."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from latent_testutil import BF16, FP32, same

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [BF16, FP32])


# ------------------------------------------------------------ padded batches
@TYPES
@pytest.mark.parametrize("cu", [[0, 5, 9], [2, 5, 9], [0, 0, 9], [3, 3, 3], [0, 16, 16], [1, 2, 15]])
def test_append_leaves_padding_alone(dtype, cu):
    """Tokens that no sequence holds go nowhere: the table's entries behind a sequence's pages are pages of others."""
    T, page, d = 16, 4, 24
    g = torch.Generator().manual_seed(sum(cu))
    kv = torch.randn(1, T, d, generator=g).to(dtype).cuda()
    was = torch.randn(12, page, d, generator=g).to(dtype).cuda()
    table = torch.tensor([[0, 1, 2, 3, 4, 10, 10, 10], [5, 6, 7, 8, 9, 0, 1, 2]], dtype=torch.int32).cuda()
    before = [3, 2]
    cache, rows = was.clone(), torch.full((1, T, d), 7.0, dtype=dtype, device="cuda")
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    kda.latent_append(kv, cache, table, torch.tensor(before, dtype=torch.int32).cuda(), 16, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), rows=rows,
                      device_status=status)
    want, want_rows = was.clone(), torch.full_like(rows, 7.0)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        for t in range(a, b):
            pos = before[n] + t - a
            want[int(table[n, pos // page]), pos % page] = kv[0, t]
            want_rows[0, t] = kv[0, t]
    assert same(cache, want) and same(rows, want_rows) and int(status) == 0
