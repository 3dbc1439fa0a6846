"""Latent attention with its positions and its cache, in plain form and as the package's calls.

The full-attention layer of a hybrid language model keeps one latent vector a
token for all of its heads, and beside it one key that carries the position:

  rotary    rotary positions on part of each head: with p the token's position
            and f_i the frequency of pair i, the pair (a, b) becomes
            m (a cos p f_i - b sin p f_i, a sin p f_i + b cos p f_i); pairs are
            neighbours (``interleaved``) or half the rotated part apart.
            ``rotary_grad`` is the gradient, the rotation back.
  append    a token's latent c, normed, and its key's position part, rotated,
            written to the sequence's page of the cache.
  prefill   the expanded form: keys [k_nope_h, k_rope] and values v_h for each
            head h, k_rope shared by the heads,
                s = scale (q . k),  o = softmax(s) v,  lse = log sum exp s
            over the keys up to the query's own place (queries stand at the
            end of their sequence's keys).  A query without a key has o = 0
            and lse = -inf.  ``prefill_grad``: the gradients of q, k_nope,
            k_rope and v from those of o, with o and lse of the forward.
  decode    the absorbed form for a few tokens of many sequences: the queries
            live in the latent space, a cache row [c, k_rope] is the key of
            every head and c its value.

Where ``own`` is false everything is computed with elementary torch operations
in 32 bits (angles in 64)."""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # the queries of a long prompt that continues a context stretched to 131072 tokens, position part behind the plain part
        dict(name="rotary_long", op="rotary", dtype="bf16", batch=1, length=32768, heads=32, dim=192, rotated=64, offset=128, start=98304, interleaved=True, stretch=32.0),
        # a training batch's gradients, the first half of each head rotated, pairs half of it apart
        dict(name="rotary_grad", op="rotary_grad", dtype="fp32", batch=2, length=4096, heads=32, dim=128, rotated=64, offset=0, start=0, interleaved=False, stretch=1.0),
        # one new token for each of 256 running sequences
        dict(name="append_step", op="append", dtype="bf16", lens=",".join(["1"] * 256), before_lo=0, before_hi=1000, latent=512, rope=64, page=64, interleaved=True),
        # eight packed prompts written to the cache, two of them behind a cached beginning
        dict(name="append_prompts", op="append", dtype="bf16", lens="512,7001,1,2900,64,5333,0,1777", before_lo=0, before_hi=300, latent=512, rope=64, page=16, interleaved=False),
        # one user's short prompt, where latency counts
        dict(name="prefill_short", op="prefill", dtype="fp32", lens="600", before="0", batch=1, heads=8, nope=128, rope=64, dim_v=128, causal=True),
        # a long document
        dict(name="prefill_long", op="prefill", dtype="bf16", lens="8192", before="0", batch=1, heads=32, nope=128, rope=64, dim_v=128, causal=True),
        # ragged prompts packed along one axis, most of them behind a beginning that is in the cache already, one without a new token
        dict(name="prefill_packed", op="prefill", dtype="bf16", lens="512,3001,1,900,64,2333,0,777", before="0,1000,4097,0,63,500,129,0", batch=0, heads=32, nope=128, rope=64, dim_v=128, causal=True),
        # a training step's gradients over two rows of a batch
        dict(name="grad_train", op="prefill_grad", dtype="bf16", lens="4096", before="0", batch=2, heads=32, nope=128, rope=64, dim_v=128, causal=True),
        # packed documents in 32 bits
        dict(name="grad_packed", op="prefill_grad", dtype="fp32", lens="700,1,333,0,1201", before="0,0,0,0,0", batch=0, heads=8, nope=128, rope=64, dim_v=128, causal=True),
        # four sequences of a few hundred tokens in 32 bits: the smallest step
        dict(name="decode_small", op="decode", dtype="fp32", batch=4, tokens=1, heads=8, latent=512, rope=64, page=64, lo=1, hi=700, empty=0),
        # one token for each of 128 running sequences of up to 16384 tokens
        dict(name="decode_batch", op="decode", dtype="bf16", batch=128, tokens=1, heads=32, latent=512, rope=64, page=64, lo=1, hi=16384, empty=2),
        # four drafted tokens for three sequences with long contexts
        dict(name="decode_drafted", op="decode", dtype="bf16", batch=3, tokens=4, heads=64, latent=512, rope=64, page=64, lo=5000, hi=131072, empty=0),
    ]


def _between(rng, lo, hi):
    """A whole number spread evenly over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(lens):
    return ",".join(str(n) for n in lens)


def _cut(rng, total, count):
    """`count` ragged lengths of `total` in all, an empty one among them now and then."""
    cuts = sorted(rng.randrange(total + 1) for _ in range(count - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if count > 2 and rng.random() < 0.5:
        lens[rng.randrange(count)] = 0
    return lens if sum(lens) else [1] * count


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "append", "prefill", "prefill", "prefill_grad", "prefill_grad", "decode", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("rotary", "rotary_grad"):
        dim = rng.choice([32, 64, 80, 128, 192])
        rotated = rng.choice([n for n in (16, 32, 64, 80, 128) if n <= dim])
        return dict(op=op, dtype=dtype, batch=rng.choice([1, 1, 2, 5]), length=_between(rng, 1, 2500), heads=rng.choice([1, 3, 8, 32, 40]), dim=dim, rotated=rotated,
                    offset=rng.choice([0, dim - rotated]), start=_between(rng, 1, 1000000) - 1, interleaved=rng.random() < 0.5, stretch=rng.choice([1.0, 4.0, 32.0]))
    if op == "append":
        latent, rope = rng.choice([(512, 64), (256, 32), (512, 0), (384, 64), (128, 64)])
        lens = _cut(rng, _between(rng, 1, 12000), rng.choice([1, 2, 5, 17])) if rng.random() < 0.5 else [1] * _between(rng, 1, 300)
        return dict(op=op, dtype=dtype, lens=_text(lens), before_lo=0, before_hi=_between(rng, 1, 1000), latent=latent, rope=rope, page=rng.choice([1, 16, 48, 64, 256]),
                    interleaved=rng.random() < 0.5)
    if op == "decode":
        latent, rope = rng.choice([(512, 64), (512, 64), (256, 32), (512, 0), (384, 64), (128, 64)])
        batch, tokens = _between(rng, 1, 200), rng.choice([1, 1, 1, 2, 4, 7])
        heads = rng.choice([1, 4, 8, 20, 32, 64, 128])
        hi = _between(rng, 8, min(100000, max(16, int(2.5e9 // (2000 * batch)) * 32 // max(32, heads * tokens))))
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, heads=heads, latent=latent, rope=rope, page=rng.choice([1, 16, 48, 64, 256]), lo=1, hi=hi,
                    empty=rng.choice([0, 0, 1]) if batch > 1 else 0)
    nope, rope, dim_v = rng.choice([(128, 64, 128), (128, 64, 128), (64, 32, 64), (128, 0, 128), (64, 64, 128), (96, 32, 80), (48, 16, 40)])
    case = dict(op=op, dtype=dtype, heads=rng.choice([1, 3, 8, 20, 32]), nope=nope, rope=rope, dim_v=dim_v, causal=rng.random() < 0.8)
    total = _between(rng, 1, 4000 if dtype == "bf16" else 2000)
    if rng.random() < 0.5:
        lens = _cut(rng, total, rng.choice([2, 3, 6]))
        before = [rng.choice([0, 0, 1, 63, 64, 500, 1000]) for _ in lens]
        return dict(case, lens=_text(lens), before=_text(before), batch=0)
    batch = rng.choice([1, 1, 2, 3])
    return dict(case, lens=str(max(1, total // batch)), before=str(rng.choice([0, 0, 1, 70, 777])), batch=batch)


def _numbers(text):
    return [int(n) for n in text.split(",")]


def _spread(count, lo, hi, empty=0):
    """`count` lengths spread over [lo, hi] in no order, the longest first; the last `empty` of them 0."""
    lens = [hi] + [lo + int((hi - lo) * (k * 0.6180339887498949 % 1)) for k in range(1, count)]
    return lens[: count - empty] + [0] * empty


def _before(case):
    """Tokens that the sequences of an append have in the cache already."""
    return _spread(len(_numbers(case["lens"])), case["before_lo"], case["before_hi"])


def _pairs(case):
    """(query tokens, key tokens, visible pairs) of a prefill in all, for one head."""
    queries = keys = pairs = 0
    for n, b in zip(_numbers(case["lens"]), _numbers(case["before"])):
        queries, keys = queries + n, keys + n + b
        pairs += n * b + (n * (n + 1) // 2 if case["causal"] else n * n)
    return tuple(v * max(1, case["batch"]) for v in (queries, keys, pairs))


# ----------------------------------------------------------------- inputs ----
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _frequencies(rotated, stretch):
    """Radians a position of each pair, base 10000; a context `stretch` times as long turns slow pairs as much slower and leaves fast ones."""
    f = 10000.0 ** (-torch.arange(0, rotated, 2, dtype=torch.float64) / rotated)
    turns = 4096 * f / (2 * math.pi)  # over a context of 4096
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (f * keep + f / stretch * (1 - keep)).cuda()


def _pages(g, lens, page):
    """A pool a little larger than needed and each sequence's pages of it, in no order; -1 behind them."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)
    at = torch.arange(width, device="cuda")
    table = order[(first[:-1, None] + at).clamp(max=pool - 1)]
    return pool, torch.where(at < (first[1:] - first[:-1])[:, None], table, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": case, "op": case["op"]}
    if case["op"] in ("rotary", "rotary_grad"):
        b, t, h, d = case["batch"], case["length"], case["heads"], case["dim"]
        s["x"] = normal(b, t, h, d).to(dt)
        s["freqs"] = _frequencies(case["rotated"], case["stretch"])
        s["magnitude"] = 1 + 0.1 * math.log(case["stretch"])
        row = 7 * int(seed) % 50 + torch.arange(b, device="cuda") * 13  # rows of a batch stand at places of their own
        s["positions"] = (case["start"] + row[:, None] + torch.arange(t, device="cuda")).to(torch.int32)
        return s
    if case["op"] == "append":
        lens, before, c, r = _numbers(case["lens"]), _before(case), case["latent"], case["rope"]
        # a slice of the projection that makes the queries' latent too
        s["kv"] = (normal(1, sum(lens), c + r + 64) * 2).to(dt)[..., 64:]
        pool, s["table"] = _pages(g, [n + b for n, b in zip(lens, before)], case["page"])
        s["cache"] = normal(pool, case["page"], c + r).to(dt)
        s["lengths"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["weight"] = 1 + 0.2 * normal(c)
        s["freqs"] = _frequencies(r, 1.0) if r else None
        return s
    if case["op"] == "decode":
        c, r, m = case["latent"], case["rope"], case["tokens"]
        lens = _spread(case["batch"], case["lo"], case["hi"], case["empty"])
        pool, s["table"] = _pages(g, lens, case["page"])
        s["cache"] = torch.empty(pool, case["page"], c + r, dtype=dt, device="cuda")
        for part in s["cache"].split(max(1, 2 ** 28 // (case["page"] * (c + r)))):
            part.copy_(normal(*part.shape))
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = (1.5 * normal(case["batch"], m, case["heads"], c + r)).to(dt)
        s["scale"] = 1 / math.sqrt(192)
        return s
    lens, before = _numbers(case["lens"]), _numbers(case["before"])
    h, n, r, v = case["heads"], case["nope"], case["rope"], case["dim_v"]
    s["lens"], s["lens_k"] = lens, [a + b for a, b in zip(lens, before)]
    if case["batch"]:
        lead_q, lead_k = (case["batch"], lens[0]), (case["batch"], s["lens_k"][0])
        s["cu"] = s["cu_k"] = None
    else:
        lead_q, lead_k = (1, sum(lens)), (1, sum(s["lens_k"]))
        s["cu"], s["cu_k"] = (torch.tensor([0] + k, device="cuda").cumsum(0).to(torch.int32) for k in (lens, s["lens_k"]))
    s["q"] = (1.5 * normal(*lead_q, h, n + r)).to(dt)
    # keys and values as one up-projection gives them, the shared key as a slice of the down-projection
    up = normal(*lead_k, h, n + v).to(dt)
    s["k_nope"], s["v"] = up[..., :n], up[..., n:]
    s["k_rope"] = normal(*lead_k, 64 + r).to(dt)[..., 64:] if r else None
    s["scale"] = 1 / math.sqrt(n + r)
    if case["op"] == "prefill_grad":
        o, s["lse"] = _attend(s)
        s["o"] = o.to(dt)
        s["d_o"] = normal(*lead_q, h, v).to(dt)
    return s


# ------------------------------------------------------------ plain forms ----
def _turned(x, angle, magnitude, interleaved, offset):
    """Pairs of the channels from `offset` turned by `angle` [..., pairs], in 32 bits."""
    pairs = angle.shape[-1]
    cos, sin = (magnitude * angle.cos()).float(), (magnitude * angle.sin()).float()
    part = x[..., offset: offset + 2 * pairs]
    part = part.unflatten(-1, (pairs, 2)) if interleaved else part.unflatten(-1, (2, pairs)).transpose(-1, -2)
    a, b = part[..., 0], part[..., 1]
    part = torch.stack([a * cos - b * sin, a * sin + b * cos], -1)
    part = part.flatten(-2) if interleaved else part.transpose(-1, -2).flatten(-2)
    return torch.cat([x[..., :offset], part, x[..., offset + 2 * pairs:]], -1)


def _plain_rotary(s):
    case = s["case"]
    angle = s["positions"].double()[..., None, None] * s["freqs"]
    y = _turned(s["x"].float(), angle if case["op"] == "rotary" else -angle, s["magnitude"], case["interleaved"], case["offset"])
    return y.to(s["x"].dtype)


def _plain_append(s):
    case, c = s["case"], s["case"]["latent"]
    kv, cu, page = s["kv"][0].float(), s["cu"].long(), case["page"]
    token = torch.arange(kv.shape[0], device="cuda")
    seq = (token[:, None] >= cu[1:]).sum(-1)
    pos = s["lengths"].long()[seq] + token - cu[seq]
    latent = kv[:, :c]
    row = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if case["rope"]:
        row = torch.cat([row, _turned(kv[:, c:], pos.double()[:, None] * s["freqs"], 1.0, case["interleaved"], 0)], -1)
    row = row.to(s["kv"].dtype)
    s["cache"][s["table"][seq, pos // page].long(), pos % page] = row
    return s["cache"], row[None]


def _padded(v, cu, lens):
    """Packed sequences [1, T, ...] as a batch [N, longest, ...]; zeros behind each end."""
    if cu is None:
        return v
    at = cu[:-1, None].long() + torch.arange(max(lens), device=v.device)
    rows = v[0][at.clamp(max=max(v.shape[1] - 1, 0))]
    return rows * (at < cu[1:, None]).view(*at.shape, *[1] * (v.dim() - 2))


def _packed(v, cu):
    """The sequences' own tokens of a batch [N, longest, ...], packed as [1, T, ...]."""
    if cu is None:
        return v
    return v[torch.arange(v.shape[1], device=v.device) < (cu[1:] - cu[:-1])[:, None]][None]


def _heads(s, kind):
    """q, k and v as [N, H, tokens, channels] of `kind`, and which keys each query sees."""
    q = _padded(s["q"].to(kind), s["cu"], s["lens"]).transpose(1, 2)
    k, v = (_padded(s[m].to(kind), s["cu_k"], s["lens_k"]).transpose(1, 2) for m in ("k_nope", "v"))
    if s["k_rope"] is not None:
        shared = _padded(s["k_rope"].to(kind), s["cu_k"], s["lens_k"])[:, None]
        k = torch.cat([k, shared.expand(-1, k.shape[1], -1, -1)], -1)
    tq, tk = (torch.tensor(s[m], device="cuda")[:, None, None] for m in ("lens", "lens_k"))
    i, j = torch.arange(q.shape[2], device="cuda")[:, None], torch.arange(k.shape[2], device="cuda")
    seen = (i < tq) & (j < tk) & ((j <= i + tk - tq) if s["case"]["causal"] else torch.ones_like(j, dtype=torch.bool))
    return q, k, v, seen[:, None]


def _attend(s):
    """o in 32 bits and lse, packed as q is."""
    q, k, v, seen = _heads(s, torch.float32)
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~seen, -torch.inf)
    top = score.amax(-1, keepdim=True) if k.shape[2] else score.new_full((*score.shape[:3], 1), -torch.inf)
    top = top.masked_fill(top == -torch.inf, 0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ v / total.masked_fill(total == 0, 1)
    lse = (total.log() + top)[..., 0]
    return _packed(o.transpose(1, 2), s["cu"]), _packed(lse.transpose(1, 2), s["cu"])


def _plain_prefill(s):
    o, lse = _attend(s)
    return o.to(s["q"].dtype), lse


def _plain_prefill_grad(s):
    n, kind = s["case"]["nope"], s["q"].dtype
    q, k, v, seen = _heads(s, torch.float32)
    o, do = (_padded(s[m].float(), s["cu"], s["lens"]).transpose(1, 2) for m in ("o", "d_o"))
    lse = _padded(s["lse"].masked_fill(s["lse"] == -torch.inf, 0), s["cu"], s["lens"]).transpose(1, 2)
    p = (q @ k.transpose(-1, -2)).mul_(s["scale"]).sub_(lse[..., None]).masked_fill_(~seen, -torch.inf).exp_()
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    got = {"q": _packed(dq.transpose(1, 2), s["cu"]), "k_nope": _packed(dk[..., :n].transpose(1, 2), s["cu_k"]), "v": _packed(dv.transpose(1, 2), s["cu_k"])}
    if s["k_rope"] is not None:
        got["k_rope"] = _packed(dk[..., n:].sum(1), s["cu_k"])
    return {m: w.to(kind) for m, w in got.items()}


def _plain_decode(s):
    case, c = s["case"], s["case"]["latent"]
    b, m, h, d = s["q"].shape
    rows = s["cache"][s["table"].clamp(min=0).long()].flatten(1, 2).float()  # [b, places, d]
    place, length = torch.arange(rows.shape[1], device="cuda"), s["lengths"].long()[:, None]
    rows = rows * (place < length)[..., None]
    score = (s["q"].float().reshape(b, m * h, d) @ rows.transpose(-1, -2)).mul_(s["scale"]).view(b, m, h, -1)
    seen = place <= (length - m + torch.arange(m, device="cuda"))[..., None]  # the last token sees all
    score = score.masked_fill_(~seen[:, :, None], -torch.inf)
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -torch.inf, 0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(1, 2) @ rows[..., :c]).view(b, m, h, c) / total.masked_fill(total == 0, 1)
    return o.to(s["q"].dtype), (total.log() + top)[..., 0]


_PLAIN = {"rotary": _plain_rotary, "rotary_grad": _plain_rotary, "append": _plain_append, "prefill": _plain_prefill, "prefill_grad": _plain_prefill_grad,
          "decode": _plain_decode}


# ------------------------------------------------------ the package's calls ----
def _own(s):
    import gated_delta_rule_49_amd as kda
    op, case = s["op"], s["case"]
    if op in ("rotary", "rotary_grad"):
        call = kda.rotary if op == "rotary" else kda.rotary_backward
        return call(s["x"], s["freqs"], positions=s["positions"], offset=case["offset"], interleaved=case["interleaved"], magnitude=s["magnitude"])
    if op == "append":
        row = kda.latent_append(s["kv"], s["cache"], s["table"], s["lengths"], case["latent"], norm_weight=s["weight"], eps=EPS, freqs=s["freqs"],
                                interleaved=case["interleaved"], cu_seqlens=s["cu"], output_rows=True)
        return s["cache"], row
    if op == "decode":
        return kda.latent_decode(s["q"], s["cache"], s["table"], s["lengths"], case["latent"], s["scale"])
    if op == "prefill":
        return kda.latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], scale=s["scale"], causal=case["causal"], cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"],
                                  check_seqlens=False)
    dq, dk_nope, dk_rope, dv = kda.latent_backward(s["q"], s["k_nope"], s["k_rope"], s["v"], s["o"], s["lse"], s["d_o"], scale=s["scale"], causal=case["causal"],
                                                   cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"])
    got = {"q": dq, "k_nope": dk_nope, "v": dv}
    return got if dk_rope is None else dict(got, k_rope=dk_rope)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("rotary", "rotary_grad"):
        tokens = case["batch"] * case["length"]
        return {"bytes": tokens * (2 * case["heads"] * case["dim"] * e + 4), "flops": tokens * case["heads"] * case["rotated"] * 3}
    if op == "append":  # a row read, written to the cache and returned
        tokens, d = sum(_numbers(case["lens"])), case["latent"] + case["rope"]
        return {"bytes": tokens * 3 * d * e + 4 * case["latent"], "flops": tokens * 4 * d}
    if op == "decode":
        lens = _spread(case["batch"], case["lo"], case["hi"], case["empty"])
        c, d, each = case["latent"], case["latent"] + case["rope"], case["heads"] * case["tokens"]
        return {"bytes": sum(lens) * d * e + case["batch"] * each * ((c + d) * e + 4), "flops": sum(lens) * each * 2 * (c + d)}
    queries, keys, pairs = _pairs(case)
    h, n, r, v = case["heads"], case["nope"], case["rope"], case["dim_v"]
    q, k = queries * h * (n + r) * e, keys * (h * n + r) * e
    o, val = queries * h * v * e, keys * h * v * e
    if op == "prefill":
        return {"bytes": q + k + val + o + queries * h * 4, "flops": pairs * h * 2 * (n + r + v)}
    # q, k, v, o, lse and the gradient of o read, the gradients of q, k and v written
    return {"bytes": 2 * (q + k + val + o) + queries * h * 4, "flops": pairs * h * 2 * (3 * (n + r) + 2 * v)}


# ------------------------------------------------------------------ exact ----
def _exact_turned(x, angle, back, magnitude, interleaved):
    """The channels as complex numbers times e^(i angle), or e^(-i angle)."""
    pairs = x.shape[-1] // 2
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, pairs), slice(pairs, None))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * torch.polar(torch.full_like(angle, magnitude), -angle if back else angle)
    y = torch.empty_like(x)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_softmax(score, seen):
    """Probabilities and lse of 64-bit scores [rows, keys]; rows that see nothing are 0 and -inf."""
    lse = torch.logsumexp(torch.where(seen, score, -torch.inf), -1)
    return torch.where(seen, torch.exp(score - torch.where(lse.isfinite(), lse, 0.0)[:, None]), 0.0), lse


def _exact_append(s):
    case, c, at = s["case"], s["case"]["latent"], 0
    cache, rows = s["cache"].double(), s["kv"][0].double()
    for k, n in enumerate(_numbers(case["lens"])):
        x = rows[at: at + n]
        pos = int(s["lengths"][k]) + torch.arange(n, device="cuda")
        new = x.clone()
        new[:, :c] = x[:, :c] / torch.sqrt((x[:, :c] ** 2).sum(-1, keepdim=True) / c + EPS) * s["weight"].double()
        if case["rope"]:
            new[:, c:] = _exact_turned(x[:, c:], pos[:, None] * s["freqs"], False, 1.0, case["interleaved"])
        cache.view(-1, x.shape[1])[s["table"][k].long()[pos // case["page"]] * case["page"] + pos % case["page"]] = new
        rows[at: at + n] = new
        at += n
    return cache, rows[None]


def _exact_decode(s):
    case, c = s["case"], s["case"]["latent"]
    b, m, h, d = s["q"].shape
    o, lse = torch.zeros(b, m, h, c, dtype=torch.float64, device="cuda"), torch.full((b, m, h), -torch.inf, dtype=torch.float64, device="cuda")
    for k in range(b):
        n = int(s["lengths"][k])
        if n == 0:
            continue
        rows = s["cache"][s["table"][k, : -(-n // case["page"])].long()].reshape(-1, d)[:n].double()
        for t in range(m):
            sees = n - m + 1 + t
            if sees > 0:
                score = s["q"][k, t].double() @ rows[:sees].T * s["scale"]
                lse[k, t] = torch.logsumexp(score, -1)
                o[k, t] = torch.softmax(score, -1) @ rows[:sees, :c]
    return o, lse


def _exact_attention(s):
    """Sequence by sequence and head by head."""
    case, h, n = s["case"], s["case"]["heads"], s["case"]["nope"]
    grad = case["op"] == "prefill_grad"
    flat = {m: s[m].double().flatten(0, 1) for m in ("q", "k_nope", "k_rope", "v", "d_o") if s.get(m) is not None}
    o, lse = torch.zeros(flat["q"].shape[0], h, case["dim_v"], dtype=torch.float64, device="cuda"), flat["q"].new_zeros(flat["q"].shape[0], h)
    got = {m: torch.zeros_like(w) for m, w in flat.items() if m != "d_o"} if grad else {}
    repeat = max(1, case["batch"])
    at = at_k = 0
    for tq, tk in zip(s["lens"] * repeat, s["lens_k"] * repeat):
        rq, rk = slice(at, at + tq), slice(at_k, at_k + tk)
        at, at_k = at + tq, at_k + tk
        if tq == 0:
            continue
        seen = torch.ones(tq, tk, dtype=torch.bool, device="cuda")
        if case["causal"]:
            seen = seen.tril(tk - tq)
        for head in range(h):
            q, v = flat["q"][rq, head], flat["v"][rk, head]
            k = flat["k_nope"][rk, head]
            if "k_rope" in flat:
                k = torch.cat([k, flat["k_rope"][rk]], -1)
            p, lse[rq, head] = _exact_softmax(q @ k.T * s["scale"], seen)
            o[rq, head] = p @ v
            if grad:
                do = flat["d_o"][rq, head]
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
                got["q"][rq, head] = ds @ k
                got["v"][rk, head] = p.T @ do
                dk = ds.T @ q
                got["k_nope"][rk, head] = dk[:, :n]
                if "k_rope" in flat:
                    got["k_rope"][rk] += dk[:, n:]
    if grad:
        return {m: w.view(s[m].shape) for m, w in got.items()}
    return o.view(*s["q"].shape[:3], -1), lse.view(s["q"].shape[:3])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotary", "rotary_grad"):
        x, a, w = s["x"].double(), case["offset"], case["rotated"]
        y = x.clone()
        y[..., a: a + w] = _exact_turned(x[..., a: a + w], (s["positions"].double()[..., None] * s["freqs"])[:, :, None].expand(-1, -1, x.shape[2], -1),
                                         case["op"] == "rotary_grad", s["magnitude"], case["interleaved"])
        return y
    return {"append": _exact_append, "decode": _exact_decode}.get(case["op"], _exact_attention)(s)
