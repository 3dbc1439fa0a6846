"""The operators of a latent attention layer together, as they are used: a
layer's prompt, tokens after it, its gradients; streams, captured graphs,
isolation of sequences, two calls at once."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from latent_testutil import BACKWARD, BF16, FORWARD, FP32, Cache, make, offsets, same
from oracle import latent as R
from sublayer_testutil import check, rounded

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [BF16, FP32])
H, DC, DN, DR, DV, PAGE = 4, 128, 64, 32, 64, 16


class Layer:
    """Weights of one layer and what a program does with the operators."""

    def __init__(self, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dtype = dtype

        def weight(*shape):
            return (torch.randn(shape, generator=g) / shape[-1] ** 0.5).to(dtype).cuda()

        self.up_k, self.up_v = weight(H, DN, DC), weight(H, DV, DC)
        self.norm = (1 + 0.1 * torch.randn(DC, generator=g)).cuda()
        self.freqs, self.magnitude = kda.rotary_frequencies(DR, scaling="turns", factor=4, device="cuda")
        self.scale = (DN + DR) ** -0.5

    def turn(self, q, first):
        pos = first + torch.arange(q.shape[1], dtype=torch.int32, device="cuda")
        return kda.rotary(q, self.freqs, positions=pos, offset=DN, interleaved=True, magnitude=self.magnitude)

    def append(self, kv, cache, **kw):
        return kda.latent_append(kv, cache.cache, cache.table, cache.lengths, DC, norm_weight=self.norm, freqs=self.freqs, magnitude=self.magnitude, interleaved=True, **kw)

    def expand(self, rows):
        c = rows[..., :DC].float()
        k = torch.stack([c @ self.up_k[h].float().T for h in range(H)], -2)
        v = torch.stack([c @ self.up_v[h].float().T for h in range(H)], -2)
        return k.to(self.dtype), rows[..., DC:], v.to(self.dtype)

    def absorb(self, q):
        latent = torch.stack([q[..., h, :DN].float() @ self.up_k[h].float() for h in range(H)], -2)
        return torch.cat([latent.to(self.dtype), q[..., DN:]], -1)

    def up(self, o):
        return torch.stack([o[..., h, :].float() @ self.up_v[h].float().T for h in range(H)], -2)


@TYPES
def test_prompt_then_tokens(dtype):
    """Prompts through the expanded form, then tokens through the absorbed one over the same cache,
    against one expanded pass over everything in 64 bits."""
    layer = Layer(dtype)
    lens, more = [37, 5, 100], 6
    cache = Cache(1, [0, 0, 0], [n + more for n in lens], DC + DR, PAGE, dtype)
    rng = np.random.default_rng(1)
    total = [n + more for n in lens]
    kv, kv64 = zip(*(rounded(2 * rng.standard_normal((n, DC + DR)), dtype) for n in total))
    q, q64 = zip(*(rounded(rng.standard_normal((n, H, DN + DR)), dtype) for n in total))
    got = [[] for _ in lens]
    # prompts, packed
    cu = offsets(lens)
    rows = layer.append(torch.cat([v[:n] for v, n in zip(kv, lens)])[None].cuda(), cache, cu_seqlens=cu, output_rows=True)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    qp = torch.cat([v[:n] for v, n in zip(q, lens)])[None].cuda()
    qp = kda.rotary(qp, layer.freqs, positions=pos, offset=DN, interleaved=True, magnitude=layer.magnitude)
    o, _ = kda.latent_prefill(qp, *layer.expand(rows)[:2], layer.expand(rows)[2], scale=layer.scale, cu_seqlens=cu)
    at = 0
    for n, out in zip(lens, got):
        out.append(o[0, at:at + n].double().cpu())
        at += n
    cache.lengths += torch.tensor(lens, dtype=torch.int32).cuda()
    # tokens: one, three, two
    for m in (1, 3, 2):
        done = [int(n) for n in cache.lengths]
        layer.append(torch.stack([v[d:d + m] for v, d in zip(kv, done)]).cuda(), cache)
        qt = torch.stack([v[d:d + m] for v, d in zip(q, done)]).cuda()
        pos = cache.lengths[:, None] + torch.arange(m, dtype=torch.int32).cuda()
        qt = kda.rotary(qt, layer.freqs, positions=pos, offset=DN, interleaved=True, magnitude=layer.magnitude)
        cache.lengths += m
        o, _ = kda.latent_decode(layer.absorb(qt), cache.cache, cache.table, cache.lengths, DC, layer.scale)
        for b, out in enumerate(got):
            out.append(layer.up(o)[b].double().cpu())
    for b, n in enumerate(total):
        f = layer.freqs.cpu().numpy()
        r = np.stack([R.append_row(kv64[b][i], i, DC, layer.norm.cpu().double().numpy(), 1e-6, f, True, layer.magnitude) for i in range(n)])
        k = np.einsum("tc,hdc->thd", r[:, :DC], layer.up_k.double().cpu().numpy())
        v = np.einsum("tc,hdc->thd", r[:, :DC], layer.up_v.double().cpu().numpy())
        q_turned = R.rotary(q64[b], np.arange(n), f, DN, True, layer.magnitude)
        want, _ = R.prefill(q_turned, k, r[:, DC:], v, layer.scale)
        # beside the attention's roundings: those of the row, the turned query, the keys and values (or the
        # absorbed query and the latent result), 4 at 2^-8 of scores of size 1 and of the values
        check(f"sequence {b}", torch.cat(got[b]), want, FORWARD[dtype] + 4 * (2.0 ** -8 if dtype == BF16 else 2.0 ** -20))


@TYPES
def test_training_step(dtype):
    """Rotation, attention and their gradients in a chain, against differences of the whole in 64 bits."""
    layer = Layer(dtype, 1)
    T = 9
    t, w, d_o, d64 = make(21, (1, T), (1, T), H, DN, DR, DV, dtype, wide=1.0)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    kw = dict(positions=pos, interleaved=True, magnitude=layer.magnitude)
    q = kda.rotary(t["q"], layer.freqs, offset=DN, **kw)
    kr = kda.rotary(t["k_rope"][:, :, None], layer.freqs, **kw)[:, :, 0]
    o, lse = kda.latent_prefill(q, t["k_nope"], kr, t["v"], out_dtype=FP32)
    dq, dkn, dkr, dv = kda.latent_backward(q, t["k_nope"], kr, t["v"], o, lse, d_o)
    dq = kda.rotary_backward(dq, layer.freqs, offset=DN, **kw)
    dkr = kda.rotary_backward(dkr[:, :, None], layer.freqs, **kw)[:, :, 0]
    f = layer.freqs.cpu().numpy()

    def loss(q, kn, kr, v):
        qt = R.rotary(q, np.arange(T), f, DN, True, layer.magnitude)
        kt = R.rotary(kr[:, None], np.arange(T), f, 0, True, layer.magnitude)[:, 0]
        return (R.prefill(qt, kn, kt, v, layer.scale)[0] * d64[0]).sum()

    x = [w["q"][0], w["k_nope"][0], w["k_rope"][0], w["v"][0]]
    rng = np.random.default_rng(2)
    for n, g in enumerate((dq, dkn, dkr, dv)):
        for _ in range(4):  # derivatives along directions: norms of the gradient's error bound theirs
            way = rng.standard_normal(x[n].shape)
            up, down = [a.copy() for a in x], [a.copy() for a in x]
            up[n] += 1e-5 * way
            down[n] -= 1e-5 * way
            slope = (loss(*up) - loss(*down)) / 2e-5
            g64 = g[0].double().cpu().numpy()
            # the chain rounds the turned query and key and each gradient once more
            tol = BACKWARD[dtype] + 4 * (2.0 ** -8 if dtype == BF16 else 2.0 ** -20)
            assert abs((g64 * way).sum() - slope) <= tol * np.linalg.norm(g64) * np.linalg.norm(way) + 1e-6


@TYPES
def test_sequences_are_isolated(dtype):
    """NaN and infinities of one sequence reach no other, to the bit; nor do they from behind a length."""
    lens, lens_k = [70, 33, 129, 1], [70, 90, 129, 65]
    t, _, d_o, _ = make(31, (1, sum(lens)), (1, sum(lens_k)), 2, 128, 64, 128, dtype)
    kw = dict(cu_seqlens=offsets(lens), cu_seqlens_k=offsets(lens_k))
    o, lse = kda.latent_prefill(**t, **kw)
    grads = kda.latent_backward(**t, o=o, lse=lse, d_o=d_o, **kw)
    bad = {k: v.clone() for k, v in t.items()}
    bad["q"][0, 70:103] = torch.nan
    for k in ("k_nope", "k_rope", "v"):
        bad[k][0, 70:160] = torch.inf
        bad[k][0, 80] = torch.nan
    bad_d = d_o.clone()
    bad_d[0, 70:103] = torch.nan
    o2, lse2 = kda.latent_prefill(**bad, **kw)
    g2 = kda.latent_backward(**bad, o=o2, lse=lse2, d_o=bad_d, **kw)
    for a, b, cu in [(o, o2, lens), (lse, lse2, lens)] + [(a, b, n) for a, b, n in zip(grads, g2, (lens, lens_k, lens_k, lens_k))]:
        first, second = cu[0], cu[0] + cu[1]
        assert same(a[0, :first], b[0, :first]) and same(a[0, second:], b[0, second:])
    # absorbed: one sequence's rows and queries full of NaN
    c = Cache(32, [40, 100, 65], [40, 100, 65], 160, PAGE, dtype)
    q = rounded(np.random.default_rng(33).standard_normal((3, 2, 4, 160)), dtype)[0].cuda()
    o, lse = kda.latent_decode(q, c.cache, c.table, c.lengths, 128, 0.1)
    cache = c.cache.clone()
    for page in c.np_table[1, :-(-100 // PAGE)]:
        cache[int(page)] = torch.nan
    q2 = q.clone()
    q2[1] = torch.inf
    o2, lse2 = kda.latent_decode(q2, cache, c.table, c.lengths, 128, 0.1)
    for b in (0, 2):
        assert same(o[b], o2[b]) and same(lse[b], lse2[b])


def test_malformed_offsets_write_nothing():
    t, _, d_o, _ = make(41, (1, 60), (1, 80), 2, 64, 32, 64, BF16)
    good = kda.latent_prefill(**t)
    for cu, cu_k in (([0, 70, 60], [0, 40, 80]), ([0, 20, 59], [0, 40, 80]), ([1, 20, 60], [0, 40, 80]), ([0, 20, 60], [0, 90, 80]), ([0, 20, 60], [0, -1, 80]),
                     ([0, 20, 60], [0, 40, 81]), ([0, -2 ** 31, 60], [0, 2 ** 31 - 1, 80])):
        kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), cu_seqlens_k=torch.tensor(cu_k, dtype=torch.int32).cuda())
        o, lse = torch.full((1, 60, 2, 64), 7.0, dtype=BF16, device="cuda"), torch.full((1, 60, 2), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kda.latent_prefill(**t, o=o, lse=lse, device_status=status, **kw)
        assert int(status) == 6 and bool((o == 7).all()) and bool((lse == 7).all())
        with pytest.raises(kda.KDAError):
            kda.latent_prefill(**t, **kw)
        status.zero_()
        kda.latent_backward(**t, o=good[0], lse=good[1], d_o=d_o, device_status=status, **kw)
        assert int(status) == 6


def test_malformed_gradients_write_nothing():
    """Through the C ABI, where the gradients' buffers are the caller's."""
    import ctypes
    t, _, d_o, _ = make(42, (1, 60), (1, 60), 2, 64, 32, 64, BF16)
    o, lse = kda.latent_prefill(**t)
    cu = torch.tensor([0, 61, 60], dtype=torch.int32).cuda()
    outs = [torch.full(s, 7.0, dtype=BF16, device="cuda") for s in ((1, 60, 2, 96), (1, 60, 2, 64), (1, 60, 32), (1, 60, 2, 64))]
    a = kda.LatentPrefillArgs(B=1, T=60, S=60, H=2, d_nope=64, d_rope=32, d_v=64, num_seqs=2, in_dtype=1, out_dtype=1, causal=1, scale=0.1, q_stride_t=192, q_stride_h=96,
                              k_stride_t=256, k_stride_h=128, r_stride_t=56, v_stride_t=256, v_stride_h=128, q=t["q"].data_ptr(), k_nope=t["k_nope"].data_ptr(),
                              k_rope=t["k_rope"].data_ptr(), v=t["v"].data_ptr(), cu_seqlens_q=cu.data_ptr(), cu_seqlens_k=cu.data_ptr(), o=o.data_ptr(), lse=lse.data_ptr())
    g = kda.LatentBackwardArgs(f=a, o_stride_t=128, o_stride_h=64, lse_stride_t=2, lse_stride_h=1, d_o_stride_t=128, d_o_stride_h=64, d_o=d_o.data_ptr(), dq=outs[0].data_ptr(), dk_nope=outs[1].data_ptr(), dk_rope=outs[2].data_ptr(), dv=outs[3].data_ptr())
    L = kda.lib()
    ws = torch.zeros(int(L.kda_latent_backward_workspace_bytes(ctypes.byref(g))), dtype=torch.uint8, device="cuda")
    g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel()
    assert L.kda_latent_backward(ctypes.byref(g), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert all(bool((v == 7).all()) for v in outs)


def step(layer, t, d_o, c, q, kv):
    """One of each operator, as a list of results."""
    qt = layer.turn(t["q"], 3)
    o, lse = kda.latent_prefill(qt, t["k_nope"], t["k_rope"], t["v"])
    grads = kda.latent_backward(qt, t["k_nope"], t["k_rope"], t["v"], o, lse, d_o)
    rows = layer.append(kv, c, output_rows=True)
    return [qt, o, lse, *grads, rows, *kda.latent_decode(q, c.cache, c.table, c.lengths + 1, DC, 0.1)]


def step_inputs(dtype, seed):
    layer = Layer(dtype)
    t, _, d_o, _ = make(seed, (2, 70), (2, 90), H, DN, DR, DV, dtype)
    c = Cache(seed, [40, 600, 64], [41, 601, 65], DC + DR, PAGE, dtype)
    rng = np.random.default_rng(seed)
    q = rounded(rng.standard_normal((3, 1, H, DC + DR)), dtype)[0].cuda()
    kv = rounded(rng.standard_normal((3, 1, DC + DR)), dtype)[0].cuda()
    return layer, t, d_o, c, q, kv


@TYPES
def test_same_bits_every_time_and_on_other_streams(dtype):
    args = step_inputs(dtype, 51)
    want = step(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(2):
        for s in streams:  # calls at once, each with workspaces of its own
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(*args))
    torch.cuda.synchronize()
    for run in got:
        assert all(same(a, b) for a, b in zip(want, run))


@TYPES
def test_captured_and_replayed(dtype):
    """A graph of all operators replays on new inputs, among the program's own work, and two graphs side by side."""
    def load(into, other):
        for a, b in zip([into[1]["q"], into[2], into[3].cache, into[3].lengths, into[4], into[5]], [other[1]["q"], other[2], other[3].cache, other[3].lengths, other[4], other[5]]):
            a.copy_(b)

    graphs = []
    for seed in (61, 62):
        args = step_inputs(dtype, seed)
        step(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*args)
        graphs.append((args, graph, outs))
    for k in range(4):
        for n, (args, graph, outs) in enumerate(graphs):
            new = step_inputs(dtype, 61 + n)
            new[1]["q"].mul_(1 + 0.1 * k)
            new[2].mul_(1 - 0.1 * k)
            new[3].lengths[1] -= 100 * k  # other lengths: other shares for the workgroups
            load(args, new)
            graph.replay()
            want = step(*new)  # eager work between replays
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(want, outs)), (k, n)


def test_rows_behind_are_left_alone():
    """Outputs are written where they are due and nowhere else: buffers inside larger ones."""
    t, _, _, _ = make(71, (1, 70), (1, 70), 3, 128, 64, 128, BF16)
    big = torch.full((1, 72, 3, 128), 7.0, dtype=BF16, device="cuda")
    big_l = torch.full((1, 72, 3), 7.0, device="cuda")
    kda.latent_prefill(**t, o=big[:, :70], lse=big_l[:, :70])
    assert bool((big[:, 70:] == 7).all()) and bool((big_l[:, 70:] == 7).all()) and not bool((big[:, :70] == 7).all())
    c = Cache(72, [40, 9], [40, 9], 160, PAGE, BF16)
    q = torch.randn(2, 1, 3, 160, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    o, lse = torch.full((4, 1, 3, 128), 7.0, dtype=BF16, device="cuda"), torch.full((4, 1, 3), 7.0, device="cuda")
    kda.latent_decode(q, c.cache, c.table, c.lengths, 128, 0.1, o=o[1:3], lse=lse[1:3])
    assert bool((o[::3] == 7).all()) and bool((lse[::3] == 7).all())
    was = c.cache.clone()
    kda.latent_decode(q, c.cache, c.table, c.lengths, 128, 0.1)
    assert same(was, c.cache)


def test_binding_refusals():
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    q, kn, kr, v = z(1, 4, 2, 96), z(1, 4, 2, 64), z(1, 4, 32), z(1, 4, 2, 64)
    i32 = torch.int32
    f = kda.rotary_frequencies(32, device="cuda")[0]
    for bad in (dict(q=z(1, 4, 2, 95)), dict(k_nope=z(1, 5, 2, 64)), dict(v=z(1, 4, 1, 64)), dict(k_rope=z(1, 4, 2, 32)), dict(q=z(4, 2, 96)), dict(k_rope=None),
                dict(cu_seqlens_k=z(2, dtype=i32)), dict(cu_seqlens=z(3, dtype=i32), cu_seqlens_k=z(2, dtype=i32)), dict(o=z(1, 4, 2, 32)), dict(lse=z(1, 4, 2)[..., :1]),
                dict(q=z(1, 4, 96, 2).transpose(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            kda.latent_prefill(**dict(dict(q=q, k_nope=kn, k_rope=kr, v=v), **bad))
    for bad in (dict(v=v.float()), dict(q=q.double()), dict(cu_seqlens=z(2, dtype=torch.int64)), dict(lse=z(1, 4, 2)), dict(out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            kda.latent_prefill(**dict(dict(q=q, k_nope=kn, k_rope=kr, v=v), **bad))
    with pytest.raises(kda.KDAError):
        kda.latent_prefill(z(1, 4, 2, 208), z(1, 4, 2, 208), None, v)
    with pytest.raises(ValueError):
        kda.rotary(q, f, positions=z(5, dtype=i32))
    with pytest.raises(ValueError):
        kda.rotary(q, f, positions=z(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        kda.rotary(q, f.float())
    with pytest.raises(kda.KDAError):
        kda.rotary(q, f, offset=80)
    with pytest.raises(kda.KDAError):  # part of its own memory
        kda.rotary(q[:, :3], f, out=q[:, 1:])
    cache, table, lens = z(6, 4, 96), z(2, 3, dtype=i32), z(2, dtype=i32)
    kv, qd = z(2, 1, 96), z(2, 1, 3, 96)
    for bad in (dict(kv=z(2, 1, 88)), dict(cache=cache.float()), dict(cache=z(6, 4, 88)), dict(table=z(3, 3, dtype=i32)), dict(table=z(2, 3)), dict(lens=z(3, dtype=i32)),
                dict(lens=z(2, dtype=torch.int64)), dict(d=0), dict(d=97), dict(norm_weight=z(63, dtype=FP32)), dict(freqs=f[:5]), dict(rows=z(2, 1, 96, dtype=FP32))):
        x = dict(dict(kv=kv, cache=cache, table=table, lens=lens, d=64), **bad)
        with pytest.raises((ValueError, TypeError)):
            kda.latent_append(x.pop("kv"), x.pop("cache"), x.pop("table"), x.pop("lens"), x.pop("d"), **x)
    for bad in (dict(q=z(2, 3, 96)), dict(cache=cache.float()), dict(table=z(3, 3, dtype=i32)), dict(lens=z(3, dtype=i32)), dict(d=97), dict(o=z(2, 1, 3, 96)), dict(lse=z(2, 1, 3))):
        x = dict(dict(q=qd, cache=cache, table=table, lens=lens, d=64), **bad)
        with pytest.raises((ValueError, TypeError)):
            kda.latent_decode(x.pop("q"), x.pop("cache"), x.pop("table"), x.pop("lens"), x.pop("d"), 0.1, **x)
    with pytest.raises(kda.KDAError):
        kda.latent_decode(z(2, 1, 3, 600), z(6, 4, 600), table, lens, 520, 0.1)
