"""Calls of the latent attention layer at the edges that its operators allow:
padded batches, calls in each of the fp32 kernels, a training step's whole
gradients."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from latent_testutil import BACKWARD, BF16, FORWARD, FP32, check_gradient, check_lse, cut, make, offsets, same
from oracle import latent as R
from sublayer_testutil import check

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


# ------------------------------------------------------------- training step
@TYPES
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dn,dr,dv", [(64, 32, 64), (128, 64, 128)])
def test_training_step_whole_gradients(dtype, interleaved, dn, dr, dv):
    """Rotation, attention and their gradients in a chain: every gradient as a whole, and its rotated channels by
    themselves, against the chain in 64 bits."""
    T, H, first = 40, 3, 500
    freqs, magnitude = kda.rotary_frequencies(dr, scaling="turns", factor=4, device="cuda")
    t, w, d_o, d64 = make(23, (1, T), (1, T), H, dn, dr, dv, dtype, wide=1.0)
    at = np.arange(T) + first
    kw = dict(positions=torch.from_numpy(at).to(torch.int32).cuda(), interleaved=interleaved, magnitude=magnitude)
    q = kda.rotary(t["q"], freqs, offset=dn, **kw)
    kr = kda.rotary(t["k_rope"][:, :, None], freqs, **kw)[:, :, 0]
    o, lse = kda.latent_prefill(q, t["k_nope"], kr, t["v"], out_dtype=FP32)
    dq, dkn, dkr, dv_ = kda.latent_backward(q, t["k_nope"], kr, t["v"], o, lse, d_o)
    dq = kda.rotary_backward(dq, freqs, offset=dn, **kw)
    dkr = kda.rotary_backward(dkr[:, :, None], freqs, **kw)[:, :, 0]

    f, scale = freqs.cpu().numpy(), (dn + dr) ** -0.5

    def turn(x, offset, back=False, m=magnitude):
        return R.rotary(x, at, f, offset, interleaved, m, back)

    qt, kt = turn(w["q"][0], dn), turn(w["k_rope"][0][:, None], 0)[:, 0]
    gq, gkn, gkr, gv = R.prefill_backward(qt, w["k_nope"][0], kt, w["v"][0], d64[0], scale)
    want = [turn(gq, dn, True), gkn, turn(gkr[:, None], 0, True)[:, 0], gv]
    # beside the gradients' own roundings the chain rounds the turned query and key and, once more, their gradients: 4
    tol = BACKWARD[dtype] + 4 * (2.0 ** -8 if dtype == BF16 else 2.0 ** -20)
    for name, g, x in zip(("dq", "dk_nope", "dk_rope", "dv"), (dq, dkn, dkr, dv_), want):
        check(name, g[0], x, tol)
    check("dq, rotated channels", dq[0, ..., dn:], want[0][..., dn:], tol)
    # what the tolerance tells apart: no rotation back, one without its magnitude, one that turns on
    for wrong in (gq, turn(gq, dn, True, 1.0), turn(gq, dn)):
        part, right = wrong[..., dn:], want[0][..., dn:]
        assert np.linalg.norm(part - right) > 3 * tol * np.linalg.norm(right)


# ------------------------------------- the fp32 kernels of many tokens and heads
def many_heads(dims, H, lens, lens_k, causal, packed, scale=None, seed=0):
    """fp32 calls above 65536 tokens times heads, on either side or both: three heads against the fp64 forms, with gradients of
    theirs alone (dk_rope is then their sum), the others against calls of fewer heads."""
    dn, dr, dv = dims
    if packed:
        lead_q, lead_k = (1, sum(lens)), (1, sum(lens_k))
        kw = dict(cu_seqlens=offsets(lens), cu_seqlens_k=offsets(lens_k))
    else:
        lead_q, lead_k, kw = (len(lens), lens[0]), (len(lens), lens_k[0]), {}
    assert max(sum(lens), sum(lens_k)) * H >= 65536
    t, w, d_o, d64 = make(seed + sum(lens), lead_q, lead_k, H, dn, dr, dv, FP32)
    some = [0, H // 2 + 1, H - 1]
    rest = [h for h in range(H) if h not in some]
    d_o[:, :, rest] = 0
    kw.update(causal=causal, scale=scale)
    c = (dn + dr) ** -0.5 if scale is None else scale
    o, lse = kda.latent_prefill(**t, **kw)
    grads = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, **kw)
    w = {k: v if k == "k_rope" or v is None else v[:, :, some] for k, v in w.items()}
    keys = ("o", "lse", "dq", "dkn", "dkr", "dv")
    want, terms = {k: [] for k in keys}, {k: [] for k in keys}
    at = at_k = 0
    for b, (n, m) in enumerate(zip(lens, lens_k)):
        s = cut(w, 0, at, at + n, at_k, at_k + m) if packed else cut(w, b, 0, n, 0, m)
        g, given = ((x[0, at:at + n] if packed else x[b])[:, some] for x in (d64, o.double().cpu().numpy()))
        at, at_k = at + n, at_k + m
        for key, v in zip(keys, [*R.prefill(**s, scale=c, causal=causal), *R.prefill_backward(**s, d_o=g, scale=c, causal=causal, o=given)]):
            want[key].append(v)
        for key, v in zip(keys[2:], R.prefill_backward_terms(**s, d_o=g, scale=c, causal=causal)):
            terms[key].append(v)

    def whole(parts, like):
        return np.concatenate([v.reshape(-1, *v.shape[1:]) for v in parts]).reshape(like.shape)

    name = f"{dims} {H} {lens} {lens_k}"
    check(f"{name} o", o[:, :, some], whole(want["o"], o[:, :, some]), FORWARD[FP32])
    check_lse(f"{name} lse", lse[:, :, some], whole(want["lse"], lse[:, :, some]))
    for key, v in zip(keys[2:], grads):
        if v is None:
            assert dr == 0
            continue
        if key != "dkr":
            assert not v[:, :, rest].any()
            v = v[:, :, some]
        check_gradient(f"{name} {key}", v, whole(want[key], v), BACKWARD[FP32], whole(terms[key], v))
    for h in range(0, H, 8):  # 8 heads a call run in the kernels of few tokens
        part = {k: v if k == "k_rope" or v is None else v[:, :, h:h + 8] for k, v in t.items()}
        o8, lse8 = kda.latent_prefill(**part, **kw)
        none = torch.isinf(lse8)
        assert torch.equal(none, torch.isinf(lse[:, :, h:h + 8]))
        check("heads", o[:, :, h:h + 8], o8.double().cpu().numpy(), 2 * FORWARD[FP32])
        check("heads' lse", lse[:, :, h:h + 8].masked_fill(none, 0), lse8.masked_fill(none, 0).double().cpu().numpy(), 2.0 ** -17)


FP32_DIMS = pytest.mark.parametrize("dims", [(128, 64, 128), (128, 0, 128), (96, 32, 80), (64, 0, 64), (136, 24, 72)])


@FP32_DIMS
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_many_tokens(dims, causal):
    many_heads(dims, 96, [701], [701], causal, False)


@FP32_DIMS
def test_fp32_many_tokens_packed(dims):
    many_heads(dims, 80, [70, 0, 1, 129, 300, 0, 333], [70, 5, 40, 200, 200, 0, 333], True, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,lens_k", [([600], [777]), ([777], [600]), ([350, 350], [400, 400])])
def test_fp32_many_tokens_behind_others(lens, lens_k, causal):
    many_heads((128, 64, 128), 112, lens, lens_k, causal, False, seed=1)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,lens_k,packed", [([20], [1001], False), ([1001], [20], False), ([3, 0, 17], [600, 41, 300], True), ([600, 41, 300], [3, 0, 17], True)])
def test_fp32_many_tokens_on_one_side(lens, lens_k, packed, causal):
    """The two gradient kernels in tiles of different sizes."""
    many_heads((128, 64, 128), 96, lens, lens_k, causal, packed, seed=2)


@pytest.mark.parametrize("scale", [0.0, -0.06])
def test_fp32_many_tokens_scales(scale):
    many_heads((128, 64, 128), 96, [701], [701], True, False, scale=scale, seed=3)


# ----------------------------------------------------------- one key to be seen
@pytest.mark.parametrize("dtype,precise", [(BF16, False), (BF16, True), (FP32, False)])
@pytest.mark.parametrize("dims", [(128, 64, 128), (48, 16, 40), (96, 0, 128)])
@pytest.mark.parametrize("B,H", [(3, 5), (700, 96)])  # below and above the limit of the fp32 kernels for few tokens
def test_one_key_has_no_score_gradient(dtype, precise, dims, B, H):
    """Where a query sees one key its probability is 1 whatever the score: dq and dk are 0, dv is what comes in."""
    if B > 3 and dims[0] == 48:
        B = 701
    for T, S, causal in [(1, 1, True), (1, 1, False)] + ([(3, 1, False), (70, 1, False), (3, 1, True)] if B == 3 else []):
        t, _, d_o, _ = make(B + T, (B, T), (B, S), H, *dims, dtype)
        o, lse = kda.latent_prefill(**t, causal=causal)
        dq, dkn, dkr, dv = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, causal=causal, precise=precise)
        assert not dq.any() and not dkn.any() and (dkr is None or not dkr.any())
        seen = d_o if not causal or T == 1 else d_o[:, -1:]
        want = seen.double().sum(1, keepdim=True)
        check("dv", dv, want.cpu().numpy(), BACKWARD[dtype])


@pytest.mark.parametrize("dtype,precise", [(BF16, False), (BF16, True), (FP32, False)])
@pytest.mark.parametrize("H", [2, 512])
@pytest.mark.parametrize("tq,tk", [(2, 2), (130, 130), (200, 131), (131, 100), (5, 3)])
def test_the_first_key_alone(dtype, precise, H, tq, tk):
    """Only the query that sees the first key alone has a gradient coming in: none of the keys gets any of its score's."""
    t, w, d_o, d64 = make(tq, (1, tq), (1, tk), H, 64, 32, 64, dtype)
    one = tq - tk
    d_o[:, :one] = 0
    d_o[:, one + 1:] = 0
    o, lse = kda.latent_prefill(**t)
    dq, dkn, dkr, dv = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, precise=precise)
    assert not dq.any() and not dkn.any() and not dkr.any() and not dv[:, 1:].any()
    check("dv", dv[:, :1], d_o[:, one:one + 1].double().cpu().numpy(), BACKWARD[dtype])
