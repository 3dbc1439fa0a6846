"""The sublayer's operators together, as a layer runs them: the short
convolution, the state space scan on slices of its output, the gated norm with
the residual and the next norm; a prompt and then tokens; the gradients back
through all of them; on other streams, at once, and captured into graphs."""
import numpy as np
import pytest
import torch

import gated_delta_rule_49_amd as kda
from oracle import reference
from oracle import sublayer as R
from sublayer_testutil import TOL, TOL_SPLIT, check, rounded

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
H, G, P, N, W = 6, 2, 32, 64, 4
DIM, C = H * P, H * P + 2 * G * N


class Layer:
    """Inputs and weights of one layer: device tensors, and the fp64 values."""

    def __init__(self, seed, B, T, dtype, docs=None):
        rng = np.random.default_rng(seed)
        self.B, self.T = B, T
        self.docs = B if docs is None else docs
        self.dev, self.ref = {}, {}
        for name, shape, scale, t in (("mixed", (B, T, C), 1, dtype), ("dt", (B, T, H), .5, dtype), ("gate", (B, T, DIM), 1, dtype),
                                      ("residual", (B, T, DIM), 1, dtype), ("w", (C, W), .5, F32), ("bias", (C,), .1, F32),
                                      ("D", (H,), 1, F32), ("dt_bias", (H,), .1, F32), ("post", (DIM // G,), 1, F32),
                                      ("scale", (DIM,), 1, F32), ("pre", (DIM,), 1, F32), ("window", (self.docs, C, W - 1), 1, F32),
                                      ("state", (self.docs, H, N, P), 1, F32)):
            cpu, self.ref[name] = rounded(scale * rng.standard_normal(shape), t)
            self.dev[name] = cpu.cuda()
        cpu, self.ref["A"] = rounded(-rng.uniform(1, 8, H), F32)
        self.dev["A"] = cpu.cuda()


def cut(y):
    x, b, c = y[..., :DIM], y[..., DIM:DIM + G * N], y[..., DIM + G * N:]
    if isinstance(y, torch.Tensor):
        return x.unflatten(-1, (H, P)), b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N))
    return x.reshape(*x.shape[:-1], H, P), b.reshape(*b.shape[:-1], G, N), c.reshape(*c.shape[:-1], G, N)


def forward(d, cu=None):
    """(conv's output, its window, y, state, out, normed)"""
    a, window = kda.short_conv(d["mixed"], d["w"], d["window"], d["bias"], cu, silu=True)
    x, b, c = cut(a)
    y, state = kda.ssm_prefill(x, d["dt"], d["A"], b, c, D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True, initial_state=d["state"],
                               cu_seqlens=cu, check_seqlens=False)
    out, normed = kda.block_norm(y.flatten(2), residual=d["residual"], post_weight=d["post"], gate=d["gate"], scale=d["scale"],
                                 pre_weight=d["pre"], group_size=DIM // G, gate_activation="silu", gate_first=True)
    return a, window, y, state, out, normed


def norm_ref(r, y):
    return R.block_norm(y.reshape(*y.shape[:2], DIM), r["residual"], r["post"], r["gate"], r["scale"], r["pre"], DIM // G, "silu", True)


def conv_ref(r, cu=None):
    return reference.short_conv(r["mixed"], r["w"], cu, r["window"], r["bias"], silu=True)[0]


def forward_ref(r, cu=None):
    a = conv_ref(r, cu)
    x, b, c = cut(a)
    y, state, _, _ = R.ssm_scan(x, r["dt"], r["A"], b, c, r["D"], r["dt_bias"], True, r["state"], cu)
    return (a, y, state) + norm_ref(r, y)


def offsets(lens):
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, None if cu is None else torch.from_numpy(cu).cuda()


@pytest.mark.parametrize("lens", [None, [70, 1, 0, 129]])
def test_a_layer_in_32_bits(lens):
    # Stage after stage within 2^-17 each (TOL).  The stages after the scan are
    # products, sums and norms: a norm passes a relative error on at most
    # twofold (its numerator and its mean), so out is within 3 and normed
    # within 7 such bounds; out also holds the residual, which adds no error.
    cu, dcu = offsets(lens)
    L = Layer(11, 1 if lens else 2, 200 if lens else 150, F32, len(lens) if lens else None)
    a, _, y, state, out, normed = forward(L.dev, dcu)
    ra, ry, rs, ro, rn = forward_ref(L.ref, cu)
    check("conv", a, ra, TOL[F32])
    check("y", y, ry, 2 * TOL[F32])
    check("state", state, rs, 2 * TOL[F32])
    check("out", out, ro, 3 * TOL[F32])
    check("normed", normed, rn, 7 * TOL[F32])


@pytest.mark.parametrize("lens", [None, [70, 1, 0, 129]])
def test_a_layer_in_bf16(lens):
    # each stage against the oracle on what the stage before really gave it
    cu, dcu = offsets(lens)
    L = Layer(12, 1 if lens else 2, 200 if lens else 150, BF, len(lens) if lens else None)
    a, _, y, state, out, normed = forward(L.dev, dcu)
    r = L.ref
    check("conv", a, conv_ref(r, cu), TOL[BF])
    x, b, c = cut(a.double().cpu().numpy())
    ry, rs, _, _ = R.ssm_scan(x, r["dt"], r["A"], b, c, r["D"], r["dt_bias"], True, r["state"], cu)
    check("y", y, ry, TOL[BF])
    check("state", state, rs, TOL_SPLIT)
    ro, rn = norm_ref(r, y.double().cpu().numpy())
    check("out", out, ro, TOL[BF])
    check("normed", normed, rn, TOL[BF])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_tokens_after_a_prompt(dtype):
    """A prompt of 100 tokens, then 3 single ones and 2 at once through the
    windows and states that the prompt left, against the oracle of them all."""
    B, T, first = 2, 105, 100
    L = Layer(13, B, T, dtype)
    d = L.dev
    part = lambda t0, t1: {k: v[:, t0:t1].contiguous() if k in ("mixed", "dt", "gate", "residual") else v for k, v in d.items()}  # noqa: E731
    p = part(0, first)
    a, window, y, state, _, _ = forward(p)
    rows, convs = [y], [a]
    for t0, t1 in ((100, 101), (101, 102), (102, 103), (103, 105)):
        p = part(t0, t1)
        a, window = kda.short_conv(p["mixed"], d["w"], window, d["bias"], silu=True, update_state=True)
        x, b, c = cut(a)
        y, state, _ = kda.ssm_decode(x, p["dt"], d["A"], b, c, state, D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True)
        out, normed = kda.block_norm(y.flatten(2), residual=p["residual"], post_weight=d["post"], gate=p["gate"], scale=d["scale"],
                                     pre_weight=d["pre"], group_size=DIM // G, gate_activation="silu", gate_first=True)
        rows.append(y)
        convs.append(a)
    a, y = torch.cat(convs, 1), torch.cat(rows, 1)
    r = L.ref
    check("conv", a, conv_ref(r), TOL[dtype])
    x, b, c = cut(a.double().cpu().numpy())
    ry, rs, _, _ = R.ssm_scan(x, r["dt"], r["A"], b, c, r["D"], r["dt_bias"], True, r["state"])
    check("y", y, ry, TOL[dtype])
    check("state", state, rs, TOL_SPLIT if dtype == BF else TOL[F32])
    last = {k: v[:, 103:] if k in ("gate", "residual") else v for k, v in r.items()}
    ro, rn = norm_ref(last, y[:, 103:].double().cpu().numpy())
    check("out", out, ro, TOL[dtype])
    check("normed", normed, rn, TOL[dtype])


def backward(d, fwd, d_out, d_normed, d_state, cu=None):
    """Gradients of everything the layer reads, by name."""
    a, _, y, _, _, _ = fwd
    dy, dres, dpost, dgate, dscale, dpre = kda.block_norm_backward(
        y.flatten(2), d_out, d_normed, residual=d["residual"], post_weight=d["post"], gate=d["gate"], scale=d["scale"],
        pre_weight=d["pre"], group_size=DIM // G, gate_activation="silu", gate_first=True)
    x, b, c = cut(a)
    dx, ddt, dA, dB, dC, dD, dbias, dstate = kda.ssm_backward(x, d["dt"], d["A"], b, c, dy.unflatten(-1, (H, P)), D=d["D"],
                                                              dt_bias=d["dt_bias"], dt_softplus=True, initial_state=d["state"],
                                                              d_final_state=d_state, cu_seqlens=cu)
    da = torch.cat([dx.flatten(2), dB.flatten(2), dC.flatten(2)], -1)
    dmixed, dw, dcb, dwindow = kda.short_conv_backward(d["mixed"], d["w"], da, d["window"], d["bias"], cu, silu=True)
    return dict(mixed=dmixed, dt=ddt, gate=dgate, residual=dres, w=dw, bias=dcb, D=dD, dt_bias=dbias, post=dpost, scale=dscale,
                pre=dpre, window=dwindow, state=dstate, A=dA)


@pytest.mark.parametrize("lens", [None, [70, 1, 0, 33]])
def test_a_layer_gradients_against_differences(lens):
    # Along one direction per argument: <gradient, direction> against central
    # differences of the fp64 chain, h = 1e-5: the difference's own error is
    # h^2 times a third derivative, some 1e-9 relative to the gradient.  The
    # gradient's: seven stages of 2^-17 (TOL), of the gradient's norm times the
    # direction's.
    cu, dcu = offsets(lens)
    L = Layer(14, 1 if lens else 2, 104 if lens else 90, F32, len(lens) if lens else None)
    rng = np.random.default_rng(5)
    fwd = forward(L.dev, dcu)
    grads = []
    for like in (fwd[4], fwd[5], fwd[3]):
        cpu, v = rounded(rng.standard_normal(like.shape), F32)
        grads.append((cpu.cuda(), v))
    got = backward(L.dev, fwd, grads[0][0], grads[1][0], grads[2][0], dcu)

    def loss(r):
        _, _, state, out, normed = forward_ref(r, cu)
        return (out * grads[0][1]).sum() + (normed * grads[1][1]).sum() + (state * grads[2][1]).sum()

    h = 1e-5
    for name, v in got.items():
        u = rng.standard_normal(v.shape)
        want = (loss({**L.ref, name: L.ref[name] + h * u}) - loss({**L.ref, name: L.ref[name] - h * u})) / (2 * h)
        g = v.double().cpu().numpy()
        bound = 7 * TOL[F32] * np.linalg.norm(g) * np.linalg.norm(u)
        print(f"[parity] d{name}: {(g * u).sum():.9g} {want:.9g} (<= {bound:.3g})", flush=True)
        assert abs((g * u).sum() - want) <= bound


def train(d, g, cu=None):
    fwd = forward(d, cu)
    return [*fwd, *backward(d, fwd, *g, cu).values()]


def seeds_of(L, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda shape, t: torch.randn(shape, generator=gen).to(t).cuda()  # noqa: E731
    return [mk((L.B, L.T, DIM), dtype), mk((L.B, L.T, DIM), dtype), mk((L.docs, H, N, P), F32)]


@pytest.mark.parametrize("dtype", [F32, BF])
def test_other_streams_at_once(dtype):
    """Two layers on two streams, neither the default, launched in turn."""
    layers = [Layer(20 + k, 2, 130 + 70 * k, dtype) for k in range(2)]
    grads = [seeds_of(L, k, dtype) for k, L in enumerate(layers)]
    want = [train(L.dev, g) for L, g in zip(layers, grads)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(train(layers[k].dev, grads[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            for a, b in zip(run, want[k]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [None, [70, 1, 0, 129]])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_and_replayed(dtype, lens):
    """Two layers' forward and gradients captured into a graph each; replayed
    in turn on changing inputs, with eager calls and waits between, every
    replay against the eager result."""
    cu, dcu = offsets(lens)
    n = len(lens) if lens else None
    shape = (1, 200) if lens else (2, 150)
    layers = [Layer(30 + k, *shape, dtype, n) for k in range(2)]
    grads = [seeds_of(L, k, dtype) for k, L in enumerate(layers)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for L, g in zip(layers, grads):
            train(L.dev, g, dcu)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for L, g in zip(layers, grads):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(train(L.dev, g, dcu))
        graphs.append(graph)
    for turn in range(4):
        for k, L in enumerate(layers):
            for name in ("mixed", "dt", "state", "gate"):
                L.dev[name].copy_(torch.roll(L.dev[name], 1 + turn + k, 1))
        for graph in graphs:
            graph.replay()
        eager = [train(L.dev, g, dcu) for L, g in zip(layers, grads)]
        torch.cuda.synchronize()
        for k in range(2):
            for a, b in zip(outs[k], eager[k]):
                assert torch.equal(a, b), (turn, k)


def test_tokens_captured_and_replayed():
    """A token step that updates its window and state in place."""
    L = Layer(40, 3, 8, BF)
    d = L.dev

    def step(t, window, state):
        a, _ = kda.short_conv(t["mixed"], d["w"], window, d["bias"], silu=True, update_state=True)
        x, b, c = cut(a)
        y, _, _ = kda.ssm_decode(x, t["dt"], d["A"], b, c, state, D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True)
        return kda.block_norm(y.flatten(2), residual=t["residual"], post_weight=d["post"], gate=t["gate"], pre_weight=d["pre"],
                              group_size=DIM // G, gate_activation="silu", gate_first=True)

    names = ("mixed", "dt", "residual", "gate")
    token = lambda i: {k: d[k][:, i:i + 1].contiguous() for k in names}  # noqa: E731
    held = token(0)
    window, state = d["window"].clone(), d["state"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held, window, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, normed = step(held, window, state)
    window.copy_(d["window"])
    state.copy_(d["state"])
    w2, s2 = d["window"].clone(), d["state"].clone()
    for i in range(8):
        now = token(i)
        for k in names:
            held[k].copy_(now[k])
        graph.replay()
        o2, n2 = step(now, w2, s2)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(normed, n2) and torch.equal(window, w2) and torch.equal(state, s2), i


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_document_of_bad_values_stays_alone(dtype, bad):
    """Every input of the middle document is NaN or infinite, its window and
    state too: the documents beside it in the same chunk's rows keep their
    results and gradients bit for bit."""
    lens = [70, 45, 33]
    cu, dcu = offsets(lens)
    L = Layer(50, 1, sum(lens), dtype, 3)
    g = seeds_of(L, 1, dtype)
    want = train(L.dev, g, dcu)
    lo, hi = int(cu[1]), int(cu[2])
    dirty = {k: v.clone() for k, v in L.dev.items()}
    for k in ("mixed", "dt", "gate", "residual"):
        dirty[k][:, lo:hi] = bad
    for k in ("window", "state"):
        dirty[k][1] = bad
    gd = [t.clone() for t in g]
    gd[0][:, lo:hi] = bad
    gd[1][:, lo:hi] = bad
    gd[2][1] = bad
    fwd = forward(dirty, dcu)
    grads = backward(dirty, fwd, *gd, dcu)
    got = [*fwd, *grads.values()]
    per_row = [i for i, t in enumerate(want) if t.dim() >= 3 and t.shape[:2] == (1, sum(lens))]
    per_doc = [i for i, t in enumerate(want) if t.dim() >= 3 and t.shape[0] == 3]
    assert len(per_row) == 8 and len(per_doc) == 4
    for i in per_row:
        assert torch.equal(got[i][:, :lo], want[i][:, :lo]) and torch.equal(got[i][:, hi:], want[i][:, hi:]), i
    for i in per_doc:
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][2], want[i][2]), i


@pytest.mark.parametrize("dtype", [F32, BF])
def test_broadcast_inputs(dtype):
    """B and C shared by the batch, x by the tokens (strides of zero), against
    the same values laid out: the same results, and gradients per element."""
    B, T = 3, 140
    L = Layer(60, B, T, dtype)
    d = L.dev
    x, b, c = cut(d["mixed"])
    xs, bs, cs = x[:, :1].expand(B, T, H, P), b[:1].expand(B, T, G, N), c[:1].expand(B, T, G, N)
    kw = dict(D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True, initial_state=d["state"])
    dy = seeds_of(L, 3, dtype)[0].unflatten(-1, (H, P))
    got = [*kda.ssm_prefill(xs, d["dt"], d["A"], bs, cs, **kw), *kda.ssm_backward(xs, d["dt"], d["A"], bs, cs, dy, **kw)]
    xs, bs, cs = xs.contiguous(), bs.contiguous(), cs.contiguous()
    want = [*kda.ssm_prefill(xs, d["dt"], d["A"], bs, cs, **kw), *kda.ssm_backward(xs, d["dt"], d["A"], bs, cs, dy, **kw)]
    for a, e in zip(got, want):
        assert torch.equal(a, e)


def test_refusals_of_the_binding():
    L = Layer(70, 2, 8, BF)
    d = L.dev
    x, b, c = cut(d["mixed"])
    ok = (x, d["dt"], d["A"], b, c)
    bad = [((x.float(), *ok[1:]), TypeError), ((x, d["dt"].float(), *ok[2:]), (TypeError, ValueError)),
           ((x, d["dt"], d["A"].double(), b, c), (TypeError, ValueError)), ((x, d["dt"], d["A"][:3], b, c), (TypeError, ValueError)),
           ((x.transpose(2, 3), *ok[1:]), ValueError), ((x, d["dt"], d["A"], b[:, :4], c), ValueError),
           ((x.cpu(), *ok[1:]), ValueError), ((x, d["dt"].cpu(), *ok[2:]), (TypeError, ValueError))]
    for args, error in bad:
        for fn, rest in ((kda.ssm_prefill, ()), (kda.ssm_decode, (d["state"],)), (kda.ssm_backward, (torch.zeros_like(x).contiguous(),))):
            with pytest.raises(error):
                fn(*args, *rest)
    with pytest.raises((TypeError, ValueError)):
        kda.ssm_prefill(*ok, initial_state=d["state"].to(BF))
    with pytest.raises((TypeError, ValueError)):
        kda.ssm_prefill(*ok, cu_seqlens=torch.tensor([0, 8], device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.ssm_prefill(x[..., :24].contiguous(), d["dt"], d["A"], b, c)  # d_head 24
    with pytest.raises(ValueError):
        kda.ssm_decode(*ok, d["state"], final_state=torch.empty_like(d["state"]))
    with pytest.raises((TypeError, ValueError)):
        kda.block_norm(d["gate"], residual=d["residual"].float())
    with pytest.raises((TypeError, ValueError)):
        kda.block_norm(d["gate"], post_weight=d["post"], group_size=7)
    with pytest.raises((TypeError, ValueError)):
        kda.short_conv_backward(d["mixed"], d["w"], d["gate"])
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Slices of tokens so wide that the last ones lie past 2^31 elements: the
    same results, bit for bit, as from dense copies."""
    B, T, width, h, g, p, n = 2, 140000, 8192, 2, 1, 64, 64
    base = torch.empty(B, T, width, dtype=BF, device="cuda")
    assert base.numel() > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(9)
    used = h * p + 2 * g * n
    base[..., -used:] = torch.randn(B, T, used, generator=gen, device="cuda").to(BF)
    cols = base[..., -used:]
    x, b, c = cols[..., :h * p].unflatten(-1, (h, p)), cols[..., h * p:h * p + g * n].unflatten(-1, (g, n)), cols[..., h * p + g * n:].unflatten(-1, (g, n))
    dt = torch.randn(B, T, h, generator=gen, device="cuda").to(BF)
    A, bias = torch.tensor([-1.0, -4.0], device="cuda"), torch.full((h,), -3.0, device="cuda")
    kw = dict(dt_bias=bias, dt_softplus=True)
    y, S = kda.ssm_prefill(x, dt, A, b, c, **kw)
    grads = kda.ssm_backward(x, dt, A, b, c, y, **kw)
    dense = [v.contiguous() for v in (x, b, c)]
    y2, S2 = kda.ssm_prefill(dense[0], dt, A, *dense[1:], **kw)
    grads2 = kda.ssm_backward(dense[0], dt, A, *dense[1:], y, **kw)
    for a, e in zip((y, S, *grads), (y2, S2, *grads2)):
        assert a is e is None or torch.equal(a, e)
    w = torch.rand(used, generator=gen, device="cuda")
    out, normed = kda.block_norm(cols, post_weight=w, pre_weight=w, group_size=64)
    out2, normed2 = kda.block_norm(cols.contiguous(), post_weight=w, pre_weight=w, group_size=64)
    assert torch.equal(out, out2) and torch.equal(normed, normed2)


@pytest.mark.parametrize("lens", [None, [70, 1, 0, 129]])
def test_the_gradients_report_their_status(lens):
    _, dcu = offsets(lens)
    L = Layer(80, 1 if lens else 2, 200 if lens else 150, F32, len(lens) if lens else None)
    d = L.dev
    x, b, c = cut(d["mixed"])
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    dy = torch.ones(L.B, L.T, H, P, device="cuda")
    kda.ssm_backward(x, d["dt"], d["A"], b, c, dy, initial_state=d["state"], cu_seqlens=dcu, device_status=status)
    assert int(status) == 0
