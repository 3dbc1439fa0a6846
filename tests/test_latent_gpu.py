"""Latent attention, rotary positions and the paged cache: the HIP kernels
against the fp64 forms, through the Python binding."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from latent_testutil import BACKWARD, BF16, FORWARD, FP32, Cache, check_gradient, check_lse, cut, decode_reference, make, offsets, same
from oracle import latent as R
from sublayer_testutil import check, rounded

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [BF16, FP32])
ONE = {BF16: 2.0 ** -8, FP32: 2.0 ** -21}  # one rounding of the result; fp32: a few of sums and of sine and cosine


# -------------------------------------------------------------------- rotary
@TYPES
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,offset", [(64, 64, 0), (192, 64, 128), (128, 64, 0), (96, 32, 40), (40, 24, 16), (10, 6, 3), (8, 0, 0), (7, 2, 5), (1024, 1024, 0)])
def test_rotary(dtype, interleaved, D, rot, offset):
    rng = np.random.default_rng(D + rot)
    B, T, H = 2, 5, 3
    wide, w64 = rounded(rng.standard_normal((B, T, H + 1, D + 8)), dtype)  # a slice: heads and channels cut from wider ones
    x, x64 = wide.cuda()[:, :, 1:, 8:], w64[:, :, 1:, 8:]
    freqs, mag = kda.rotary_frequencies(rot, scaling="turns", factor=4, device="cuda") if rot else (torch.zeros(0, dtype=torch.float64).cuda(), 1.0)
    pos = torch.tensor(rng.integers(0, 200000, (B, T)), dtype=torch.int32)
    kw = dict(positions=pos.cuda(), offset=offset, interleaved=interleaved, magnitude=mag)
    y, d = kda.rotary(x, freqs, **kw), kda.rotary_backward(x, freqs, **kw)
    for name, got, back in (("rotary", y, False), ("rotary gradient", d, True)):
        want = np.stack([R.rotary(x64[b], pos[b].numpy(), freqs.cpu().numpy(), offset, interleaved, mag, back) for b in range(B)])
        check(f"{name} {D} {rot} {offset}", got, want, ONE[dtype])
    rest = [c for c in range(D) if not offset <= c < offset + rot]
    assert same(y[..., rest], x[..., rest])
    z = x.clone().contiguous()  # in place, on its own memory
    assert kda.rotary(z, freqs, out=z, **kw) is z and same(z, y)


@TYPES
def test_rotary_far_positions(dtype):
    """Angles of far positions keep their accuracy: up to 2^31 - 1, and below 0."""
    freqs, _ = kda.rotary_frequencies(64, device="cuda")
    pos = torch.tensor([0, 1, 65535, 1048577, 2 ** 31 - 1, -1, -(2 ** 31)], dtype=torch.int32)
    x, x64 = rounded(np.random.default_rng(5).standard_normal((1, 7, 2, 64)), dtype)
    got = kda.rotary(x.cuda(), freqs, positions=pos.cuda())
    for t in range(7):
        want = R.rotary(x64[0, t:t + 1], [int(pos[t])], freqs.cpu().numpy())
        check(f"position {int(pos[t])}", got[0, t:t + 1], want, ONE[dtype])


def test_rotary_of_more_tokens_than_a_launch_has_workgroups():
    """2^23 workgroups of one token a launch: heads that are moved element by element."""
    T, D = 2 ** 23 + 3, 160
    x = torch.zeros((1, T, 1, D), dtype=BF16, device="cuda")
    some = [0, 1, 2 ** 23 - 1, 2 ** 23, T - 1]
    value, v64 = rounded(np.random.default_rng(3).standard_normal((1, len(some), 1, D)), BF16)
    x[:, some] = value.cuda()
    freqs, _ = kda.rotary_frequencies(2, device="cuda")
    y = kda.rotary(x, freqs)
    check("rows of both launches", y[:, some], R.rotary(v64[0], some, freqs.cpu().numpy())[None], ONE[BF16])
    y[:, some] = 0
    assert not y.any()


def test_rotary_default_positions_and_broadcast():
    x = torch.randn(3, 9, 2, 32, generator=torch.Generator().manual_seed(1)).cuda()
    freqs, _ = kda.rotary_frequencies(32, device="cuda")
    a = kda.rotary(x, freqs)
    p = torch.arange(9, dtype=torch.int32).cuda()
    assert same(a, kda.rotary(x, freqs, positions=p)) and same(a, kda.rotary(x, freqs, positions=p.expand(3, 9)))
    one = x[:1].expand(3, -1, -1, -1)  # rows that share memory are read
    assert same(kda.rotary(one, freqs)[2], a[0])
    with pytest.raises(kda.KDAError):
        kda.rotary(x, freqs, out=torch.empty(1, 9, 2, 32, device="cuda").expand(3, -1, -1, -1))  # and not written
    for n in (0, 1):
        assert kda.rotary(x[:, :n], freqs).shape == (3, n, 2, 32)


def test_rotary_gradient_against_differences():
    x, x64 = rounded(np.random.default_rng(3).standard_normal((1, 3, 1, 8)), FP32)
    g, g64 = rounded(np.random.default_rng(4).standard_normal((1, 3, 1, 8)), FP32)
    freqs, _ = kda.rotary_frequencies(4, device="cuda")
    pos = torch.tensor([4, 0, 17], dtype=torch.int32).cuda()
    d = kda.rotary_backward(g.cuda(), freqs, positions=pos, offset=2, magnitude=1.25).cpu().double().numpy()
    for at in np.ndindex(*x64.shape):
        step = np.zeros_like(x64)
        step[at] = 1.0  # linear: the difference is the derivative
        f = [R.rotary(v[0], pos.cpu().numpy(), freqs.cpu().numpy(), 2, False, 1.25) for v in (x64 + step, x64)]
        assert abs(((f[0] - f[1]) * g64[0]).sum() - d[at]) < 1e-6


# --------------------------------------------------------------------- append
@TYPES
@pytest.mark.parametrize("dc,dr,page,norm,turn,interleaved", [(512, 64, 64, True, True, True), (512, 64, 16, True, True, False), (256, 32, 1, True, True, False),
                                                               (512, 0, 7, True, False, False), (8, 8, 3, False, True, True), (384, 64, 48, True, False, False), (2048, 256, 5, True, True, False),
                                                               (136, 16, 4, False, False, False)])
@pytest.mark.parametrize("packed", [False, True])
def test_append(dtype, dc, dr, page, norm, turn, interleaved, packed):
    rng = np.random.default_rng(dc + page)
    lens = [3, 0, 70, 1, 9] if packed else [5, 5, 5]
    before = [0, 4, 61, 130, 2][:len(lens)]
    d = dc + dr
    c = Cache(dc, before, [b + n for b, n in zip(before, lens)], d, page, dtype)
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    wide, w64 = rounded(2 * rng.standard_normal((*lead, d + 16)), dtype)
    kv, kv64 = wide.cuda()[..., 16:], w64[..., 16:].reshape(-1, d)
    weight, weight64 = rounded(1 + 0.2 * rng.standard_normal(dc), FP32)
    freqs = kda.rotary_frequencies(dr)[0] if turn else None
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    was = c.cache.clone()
    rows = kda.latent_append(kv, c.cache, c.table, c.lengths, dc, norm_weight=weight.cuda() if norm else None, eps=1e-5, freqs=None if freqs is None else freqs.cuda(),
                             magnitude=1.1, interleaved=interleaved, cu_seqlens=offsets(lens) if packed else None, output_rows=True, device_status=status)
    want, at = [], 0
    untouched = torch.ones(c.cache.shape[:2], dtype=torch.bool, device="cuda")
    for n, count in enumerate(lens):
        for t in range(count):
            pos = before[n] + t
            want.append(R.append_row(kv64[at], pos, dc, weight64 if norm else None, 1e-5, None if freqs is None else freqs.numpy(), interleaved, 1.1))
            place = (int(c.np_table[n, pos // page]), pos % page)
            assert same(c.cache[place], rows.view(-1, d)[at])
            untouched[place] = False
            at += 1
    check("rows", rows, np.stack(want).reshape(*lead, d), ONE[dtype])
    assert same(c.cache[untouched], was[untouched]) and int(status) == 0
    if not norm:
        assert same(rows[..., :dc], kv[..., :dc])


def test_append_many_sequences():
    """Packed sequences are found among more than 64 and more than 4096, empty ones among them."""
    rng = np.random.default_rng(9)
    for count in (65, 4097, 5000):
        lens = rng.integers(0, 3, count)
        lens[-1] = 1
        kv = torch.randn(1, int(lens.sum()), 16, generator=torch.Generator().manual_seed(2)).cuda()
        cache = torch.zeros(count, 2, 16, device="cuda")
        kda.latent_append(kv, cache, torch.arange(count, dtype=torch.int32).cuda()[:, None], torch.zeros(count, dtype=torch.int32).cuda(), 16, cu_seqlens=offsets(lens))
        want = torch.zeros(count, 2, 16, device="cuda")
        seq = torch.from_numpy(np.repeat(np.arange(count), lens)).cuda()
        place = torch.from_numpy(np.concatenate([np.arange(n) for n in lens])).cuda()
        want[seq, place] = kv[0]
        assert torch.equal(cache, want)


def test_append_without_a_page():
    """Tokens without a page are left out and reported; the others are written."""
    kv = torch.randn(4, 2, 16, generator=torch.Generator().manual_seed(3)).cuda()
    cache = torch.zeros(5, 2, 16, device="cuda")
    table = torch.tensor([[0, 1], [2, -1], [5, 3], [4, 2 ** 30]], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = kda.latent_append(kv, cache, table, torch.tensor([3, 1, 1, -1], dtype=torch.int32).cuda(), 16, output_rows=True, device_status=status)
    want = torch.zeros_like(cache)
    want[1, 1] = kv[0, 0]  # position 4 is behind the table
    want[2, 1] = kv[1, 0]  # position 2 has entry -1
    want[3, 0] = kv[2, 1]  # position 1 has entry 5
    want[4, 0] = kv[3, 1]  # position -1
    assert torch.equal(cache, want) and torch.equal(rows, kv) and int(status) == 9


# ------------------------------------------------------------------ expanded
DIMS = [(128, 64, 128), (64, 32, 64), (128, 0, 128), (96, 32, 80), (48, 16, 40), (8, 0, 8), (64, 64, 128), (16, 16, 128), (128, 64, 16)]


def both(dtype, H, dims, lens, lens_k, causal, packed, seed=0, name="", scale=None):
    """Forward and gradients of one setting against the fp64 forms."""
    dn, dr, dv = dims
    if packed:
        lead_q, lead_k = (1, sum(lens)), (1, sum(lens_k))
        kw = dict(cu_seqlens=offsets(lens), cu_seqlens_k=offsets(lens_k))
    else:
        lead_q, lead_k, kw = (len(lens), lens[0]), (len(lens), lens_k[0]), {}
    t, w, d_o, d64 = make(seed + sum(lens), lead_q, lead_k, H, dn, dr, dv, dtype)
    kw.update(causal=causal, scale=scale)
    c = (dn + dr) ** -0.5 if scale is None else scale
    o, lse = kda.latent_prefill(**t, **kw)
    wide, lse2 = kda.latent_prefill(**t, out_dtype=FP32, **kw)
    assert same(lse, lse2) and same(wide.to(dtype), o)
    got = {kind: kda.latent_backward(**t, o=v, lse=lse, d_o=d_o, **kw) for kind, v in (("", o), ("wide ", wide))}
    o64 = o.double().cpu().numpy()
    want = {kind + m: [] for kind in ("", "wide ", "terms ") for m in ("o", "lse", "dq", "dkn", "dkr", "dv")}
    at = at_k = 0
    for b, (n, m) in enumerate(zip(lens, lens_k)):
        s = cut(w, 0, at, at + n, at_k, at_k + m) if packed else cut(w, b, 0, n, 0, m)
        g = d64[0, at:at + n] if packed else d64[b]
        at, at_k = at + n, at_k + m
        for key, v in zip(("o", "lse"), R.prefill(**s, scale=c, causal=causal)):
            want[key].append(v)
        given = o64[0, at - n:at] if packed else o64[b]
        for kind, o_in in (("", given), ("wide ", None)):
            for key, v in zip(("dq", "dkn", "dkr", "dv"), R.prefill_backward(**s, d_o=g, scale=c, causal=causal, o=o_in)):
                want[kind + key].append(v)
        for key, v in zip(("dq", "dkn", "dkr", "dv"), R.prefill_backward_terms(**s, d_o=g, scale=c, causal=causal)):
            want["terms " + key].append(v)

    def whole(key, shape):
        return np.concatenate([v.reshape(-1, *v.shape[1:]) for v in want[key]]).reshape(shape)

    check(f"{name} o", o, whole("o", o.shape), FORWARD[dtype])
    check_lse(f"{name} lse", lse, whole("lse", lse.shape))
    for kind, grads in got.items():
        for key, v in zip(("dq", "dkn", "dkr", "dv"), grads):
            if v is not None:
                check_gradient(f"{name} {kind}{key}", v, whole(kind + key, v.shape), BACKWARD[dtype], whole("terms " + key, v.shape))
        assert (grads[2] is None) == (dr == 0)


@TYPES
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_expanded_sizes(dtype, dims, causal):
    both(dtype, 2, dims, [70], [70], causal, False, name=f"{dims}")
    both(dtype, 1, dims, [33], [150], causal, False, seed=1, name=f"{dims} continued")


@TYPES
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300])
def test_expanded_lengths(dtype, n):
    both(dtype, 2, (128, 64, 128), [n], [n], True, False, name=f"{n}")
    both(dtype, 1, (128, 64, 128), [n, n], [n + 97, n + 97], True, False, seed=1, name=f"{n} behind 97")
    both(dtype, 1, (128, 64, 128), [5], [n], True, False, seed=2, name=f"5 of {n}")  # rows without a key for n < 5


@TYPES
@pytest.mark.parametrize("H", [1, 3, 8, 9])
@pytest.mark.parametrize("causal", [True, False])
def test_expanded_packed(dtype, H, causal):
    both(dtype, H, (128, 64, 128), [70, 0, 1, 129, 64, 0], [70, 5, 40, 200, 64, 0], causal, True, name="packed")
    both(dtype, H, (64, 0, 64), [3, 130, 7], [1, 64, 7], causal, True, seed=1, name="more queries than keys")


@TYPES
def test_expanded_large_scores(dtype):
    """Scores of some hundred: one key takes all; a scale of 0 and a negative one."""
    both(dtype, 2, (64, 32, 64), [90], [90], True, False, name="scale 0", scale=0.0)
    both(dtype, 2, (64, 32, 64), [90], [90], True, False, name="negative", scale=-0.1)
    t, w, d_o, d64 = make(7, (1, 80), (1, 80), 2, 64, 32, 64, dtype, wide=40.0)
    o, lse = kda.latent_prefill(**t, scale=1.0)
    want = R.prefill(**cut(w, 0, 0, 80, 0, 80), scale=1.0)
    # scores up to about 1700 in fp32 carry 1700 2^-24 into an exponent, 1e-4 of a probability
    check("o", o, want[0][None], FORWARD[dtype] + 1e-3)
    check_lse("lse", lse, want[1][None])


@TYPES
def test_expanded_empty(dtype):
    t, _, d_o, _ = make(1, (1, 6), (1, 0), 2, 64, 32, 64, dtype)
    o, lse = kda.latent_prefill(**t)
    assert not o.any() and bool((lse == -torch.inf).all())
    dq, dkn, dkr, dv = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o)
    assert not dq.any() and dkn.numel() == dkr.numel() == dv.numel() == 0
    t, _, d_o, _ = make(1, (2, 0), (2, 70), 2, 64, 32, 64, dtype)
    o, lse = kda.latent_prefill(**t)
    assert o.shape == (2, 0, 2, 64) and lse.shape == (2, 0, 2)
    dq, dkn, dkr, dv = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o)
    assert dq.numel() == 0 and not dkn.any() and not dkr.any() and not dv.any()


@TYPES
def test_expanded_strides(dtype):
    """Heads, tokens and batches in other orders, and broadcast keys: the same bits."""
    t, _, d_o, _ = make(11, (2, 75), (2, 90), 3, 128, 64, 128, dtype)
    o, lse = kda.latent_prefill(**t)
    grads = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o)

    def moved(x):  # heads outermost in memory
        return x.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) if x.dim() == 4 else x.transpose(0, 1).contiguous().transpose(0, 1)

    u = {k: moved(v) for k, v in t.items()}
    o2, lse2 = kda.latent_prefill(**u)
    assert same(o, o2) and same(lse, lse2)
    assert all(same(a, b) for a, b in zip(grads, kda.latent_backward(**u, o=o, lse=lse, d_o=d_o)))
    lse_moved = lse.permute(2, 0, 1).contiguous().permute(1, 2, 0)
    assert all(same(a, b) for a, b in zip(grads, kda.latent_backward(**u, o=moved(o), lse=lse_moved, d_o=moved(d_o))))
    ones = torch.ones((), dtype=dtype, device="cuda").expand(2, 75, 3, 128)  # d_o of a sum, as an expanded scalar
    with pytest.raises(ValueError):
        kda.latent_backward(**t, o=o, lse=lse, d_o=ones)
    rows = torch.ones(128, dtype=dtype, device="cuda").expand(2, 75, 3, 128)
    assert all(same(a, b) for a, b in zip(kda.latent_backward(**t, o=o, lse=lse, d_o=ones.contiguous()), kda.latent_backward(**t, o=o, lse=lse, d_o=rows)))
    one = {k: v[:1].expand(2, *v.shape[1:]) for k, v in t.items()}  # a batch of one row, repeated
    o3, _ = kda.latent_prefill(**one)
    assert same(o3[0], o3[1]) and same(o3[:1], o[:1])
    head = dict(t, k_nope=t["k_nope"][:, :, :1].expand(-1, -1, 3, -1), v=t["v"][:, :, :1].expand(-1, -1, 3, -1))
    o4, _ = kda.latent_prefill(**head)
    assert same(o4[:, :, :1], o[:, :, :1])
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    assert kda.latent_prefill(**t, o=out, lse=l2)[0] is out and same(out, o) and same(l2, lse)


@pytest.mark.parametrize("out_dtype", [BF16, FP32])
def test_expanded_out_dtype(out_dtype):
    """A result of another type is the same value, rounded once."""
    for dtype in (BF16, FP32):
        t, w, _, _ = make(12, (1, 100), (1, 100), 2, 128, 64, 128, dtype)
        o, _ = kda.latent_prefill(**t, out_dtype=out_dtype)
        assert o.dtype == out_dtype
        wide, _ = kda.latent_prefill(**t, out_dtype=FP32)
        assert same(o, wide.to(out_dtype))


# ------------------------------------------------------------------- decode
@TYPES
@pytest.mark.parametrize("dc,dr", [(512, 64), (512, 0), (256, 32), (384, 64), (128, 64), (8, 8), (448, 128), (64, 256)])
@pytest.mark.parametrize("H,m", [(1, 1), (8, 1), (20, 2), (32, 1), (33, 3), (128, 1)])
def test_decode_sizes(dtype, dc, dr, H, m):
    lengths = [70, 1, 0, 129]
    run_decode(dtype, dc, dr, H, m, 16, lengths, seed=dc + H)


def run_decode(dtype, dc, dr, H, m, page, lengths, seed=0, scale=0.07, out_dtype=None):
    c = Cache(seed, lengths, lengths, dc + dr, page, dtype)
    wide, w64 = rounded(1.5 * np.random.default_rng(seed + 1).standard_normal((len(lengths), m, H, dc + dr + 8)), dtype)
    status = torch.full((1,), 3, dtype=torch.int32, device="cuda")
    o, lse = kda.latent_decode(wide.cuda()[..., 8:], c.cache, c.table, c.lengths, dc, scale, out_dtype=out_dtype, device_status=status)
    want_o, want_l = decode_reference(w64[..., 8:], c, dc, scale, lengths)
    # a result in bf16 of fp32 inputs is rounded once more, 2^-8
    check(f"decode {dc} {dr} {H} {m} {page} {lengths}", o, want_o, FORWARD[dtype] + (2.0 ** -8 if dtype == FP32 and o.dtype == BF16 else 0))
    check_lse("lse", lse, want_l)
    assert int(status) == 0
    return c, o, lse


@TYPES
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 100, 256])
@pytest.mark.parametrize("m", [1, 4])
def test_decode_pages(dtype, page, m):
    run_decode(dtype, 256, 32, 4, m, page, [1, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 200, 2, 3], seed=page)


@TYPES
def test_decode_long_beside_short(dtype):
    """One sequence spread over many workgroups, its neighbours whole or empty."""
    run_decode(dtype, 128, 32, 2, 2, 64, [0, 5, 9000, 0, 1, 700, 0], seed=3)
    run_decode(dtype, 128, 32, 2, 1, 64, [12000], seed=4)
    run_decode(dtype, 16, 16, 1, 1, 16, [0, 0, 3, 0], seed=5)


@TYPES
def test_decode_many_sequences(dtype):
    rng = np.random.default_rng(8)
    run_decode(dtype, 64, 16, 2, 1, 16, [int(n) for n in rng.integers(0, 40, 700)], seed=6)


def test_decode_out_dtype():
    for dtype in (BF16, FP32):
        _, a, _ = run_decode(dtype, 256, 32, 4, 2, 16, [100, 600, 0], out_dtype=BF16)
        _, b, _ = run_decode(dtype, 256, 32, 4, 2, 16, [100, 600, 0], out_dtype=FP32)
        assert a.dtype == BF16 and b.dtype == FP32 and same(a, b.to(BF16))


@TYPES
def test_decode_strided_cache(dtype):
    """One layer of a cache of several, its rows cut from wider ones: the same bits."""
    c, o, lse = run_decode(dtype, 256, 32, 4, 1, 16, [100, 333, 0, 17], seed=13)
    pool, page, d = c.cache.shape
    layers = torch.full((pool, 3, page, d + 24), float("nan"), dtype=dtype, device="cuda")
    layers[:, 1, :, 8:8 + d] = c.cache
    q = rounded(1.5 * np.random.default_rng(14).standard_normal((4, 1, 4, d + 8)), dtype)[0].cuda()[..., 8:]
    o2, lse2 = kda.latent_decode(q, layers[:, 1, :, 8:8 + d], c.table, c.lengths, 256, 0.07)
    assert same(o, o2) and same(lse, lse2)


@TYPES
def test_decode_bad_pages(dtype):
    """Entries and lengths outside the cache are reported and touch no other sequence."""
    c, o, lse = run_decode(dtype, 128, 32, 4, 1, 16, [40, 100, 33, 64], seed=15)
    q = rounded(1.5 * np.random.default_rng(16).standard_normal((4, 1, 4, 168)), dtype)[0].cuda()[..., 8:]
    for bad in (-1, c.cache.shape[0], 2 ** 31 - 1):
        table = c.table.clone()
        table[1, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o2, lse2 = kda.latent_decode(q, c.cache, table, c.lengths, 128, 0.07, device_status=status)
        assert int(status) == 9
        for b in (0, 2, 3):
            assert same(o2[b], o[b]) and same(lse2[b], lse[b])
    lengths = c.lengths.clone()
    lengths[0], lengths[1] = -5, 16 * c.table.shape[1] + 1
    status.zero_()
    o2, lse2 = kda.latent_decode(q, c.cache, c.table.clamp(max=c.cache.shape[0] - 1), lengths, 128, 0.07, device_status=status)
    assert int(status) == 9 and not o2[0].any() and bool((lse2[0] == -torch.inf).all())
    # how the rows are dealt to the workgroups changed with the lengths, so the others agree in value, not in every bit
    for b in (2, 3):
        check("beside", o2[b], o[b].double().cpu().numpy(), FORWARD[dtype])


def test_offsets_past_32_bits():
    """Pages that lie beyond 2^32 elements of a cache (9 GB of bf16)."""
    dc, dr, page = 512, 64, 64
    pool = 2 ** 33 // (page * (dc + dr) * 2) + 4
    cache = torch.empty(pool, page, dc + dr, dtype=BF16, device="cuda")
    table = torch.tensor([[pool - 1, 0, pool - 2, pool // 2]], dtype=torch.int32).cuda()
    kv, kv64 = rounded(np.random.default_rng(17).standard_normal((1, 200, dc + dr)), BF16)
    kda.latent_append(kv.cuda(), cache, table, torch.zeros(1, dtype=torch.int32).cuda(), dc)
    assert torch.equal(cache[pool - 1], kv[0, :64].cuda()) and torch.equal(cache[pool // 2, :8], kv[0, 192:].cuda())
    q, q64 = rounded(np.random.default_rng(18).standard_normal((1, 1, 4, dc + dr)), BF16)
    o, lse = kda.latent_decode(q.cuda(), cache, table, torch.tensor([200], dtype=torch.int32).cuda(), dc, 0.07)
    want = R.decode(q64[0], kv64[0], dc, 0.07)
    check("o", o, want[0][None], FORWARD[BF16])
    check_lse("lse", lse, want[1][None])


# ------------------------------------------------------- calls at the edges ----
@TYPES
def test_expanded_many_sequences(dtype):
    """More sequences than the table keeps in LDS, most of one token, one of them long."""
    lens = [1] * 4200 + [300] + [0, 2, 3] * 3
    t, w, d_o, d64 = make(101, (1, sum(lens)), (1, sum(lens)), 1, 8, 8, 8, dtype)
    cu = offsets(lens)
    o, lse = kda.latent_prefill(**t, cu_seqlens=cu)
    grads = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, cu_seqlens=cu)
    one = {k: v[:, 4200:4500] for k, v in t.items()}
    o1, lse1 = kda.latent_prefill(**one)
    assert same(o[:, 4200:4500], o1) and same(lse[:, 4200:4500], lse1)
    for a, b in zip(grads, kda.latent_backward(**one, o=o1, lse=lse1, d_o=d_o[:, 4200:4500])):
        assert same(a[:, 4200:4500], b)
    check("single tokens", o[:, :4200], w["v"][:, :4200], FORWARD[dtype])  # one key: its value


def test_fp32_kernels_for_few_and_many_tokens_agree():
    """fp32 calls of more than 65536 tokens times heads run in other tiles: the same values."""
    t, w, d_o, d64 = make(102, (1, 1100), (1, 1100), 64, 16, 8, 16, FP32)
    o, lse = kda.latent_prefill(**t)
    grads = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o)
    part = {k: v if k == "k_rope" else v[:, :, :3] for k, v in t.items()}
    o1, lse1 = kda.latent_prefill(**part)
    check("o", o[:, :, :3], o1.double().cpu().numpy(), FORWARD[FP32])
    check("lse", lse[:, :, :3], lse1.double().cpu().numpy(), 2.0 ** -18)
    few = kda.latent_backward(**part, o=o1, lse=lse1, d_o=d_o[:, :, :3])
    for k in (0, 1, 3):
        check(f"gradient {k}", grads[k][:, :, :3], few[k].double().cpu().numpy(), BACKWARD[FP32])
    # the sum over all heads, in 64 bits
    want = np.zeros((1100, 8))
    for h in range(0, 64):
        k = np.concatenate([w["k_nope"][0, :, h], w["k_rope"][0]], -1)
        _, dk, _ = R.attention_backward(w["q"][0, :, h], k, w["v"][0, :, h], d64[0, :, h], 24 ** -0.5, True)
        want += dk[:, 16:]
    check("dk_rope", grads[2][0], want, 2 * BACKWARD[FP32])  # a sum of 64 heads: as many roundings again


@TYPES
def test_rotary_few_channels(dtype):
    """A shared key of one head: several tokens in one workgroup, the last one not full."""
    for T, D in ((1, 64), (77, 64), (513, 32), (200, 6)):
        x, x64 = rounded(np.random.default_rng(T).standard_normal((2, T, 1, D)), dtype)
        freqs, _ = kda.rotary_frequencies(D if D < 64 else 32, device="cuda")
        got = kda.rotary(x.cuda(), freqs)
        want = np.stack([R.rotary(v, np.arange(T), freqs.cpu().numpy()) for v in x64])
        check(f"{T} {D}", got, want, ONE[dtype])


def test_outputs_on_inputs_are_refused():
    t, _, d_o, _ = make(103, (1, 20), (1, 20), 2, 64, 0, 64, BF16)
    q = t["q"]
    with pytest.raises(kda.KDAError):
        kda.latent_prefill(**t, o=q)
    c = Cache(104, [20], [20], 64, 16, BF16)
    with pytest.raises(kda.KDAError):
        kda.latent_decode(c.cache[:1, :4].reshape(1, 1, 4, 64), c.cache, c.table, c.lengths, 64, 0.1, o=c.cache[1:2, :4].reshape(1, 1, 4, 64))


def test_decode_batch_of_thousands():
    """More sequences than a workgroup has threads."""
    rng = np.random.default_rng(105)
    run_decode(BF16, 16, 8, 1, 1, 16, [int(n) for n in rng.integers(0, 90, 1500)], seed=106)
    run_decode(FP32, 16, 8, 1, 1, 16, [int(n) for n in rng.integers(0, 90, 1500)], seed=107)
