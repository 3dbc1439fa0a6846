"""Shared by the tests of the sublayer's stages and of the state space scan:
seeded inputs, and the error measure with tolerances counted in roundings.

A result is compared by the 2-norm of its error over the 2-norm of the fp64
value, per tensor.  A value rounded to bf16 is off by at most half a step,
2^-8 of itself; uniformly spread roundings give an rms of about 0.41 of that.
The bounds below leave room for TWO such roundings at their worst in bf16
(the result's own, and the state's or a product's operand), 2 * 2^-8.  In fp32
the operations' own roundings are 2^-24 each; sums of up to some thousand
terms and exponents of accumulated logs (a log of magnitude up to 64 carries
2^-19 absolute) stay below 2^-17."""
import numpy as np
import torch

TOL = {torch.bfloat16: 2 * 2.0 ** -8, torch.float32: 2.0 ** -17}
# fp32 results of bf16 inputs on the matrix cores: operands split in two bf16
# parts are exact to 2^-16 (half a step of the second part)
TOL_SPLIT = 2.0 ** -16


def err(got, want):
    g = got.detach().double().cpu().numpy()
    w = np.asarray(want, dtype=np.float64)
    assert g.shape == w.shape, (g.shape, w.shape)
    if w.size == 0:
        return 0.0
    assert np.isfinite(g).all(), "non-finite values"
    n = np.linalg.norm(w)
    return float(np.linalg.norm(g - w) / n) if n else float(np.linalg.norm(g))


def check(name, got, want, tol):
    e = err(got, want)
    print(f"[parity] {name}: {e:.3e} (<= {tol:.3e})", flush=True)
    assert e <= tol, f"{name}: {e:.3e} > {tol:.3e}"


def rounded(a, dtype):
    """A tensor of `dtype` on the CPU and the fp64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype)
    return t, t.double().numpy()


def scan_inputs(seed, lead, H, G, P, N, dtype, steps=(0.001, 0.1), decay=(1.0, 16.0)):
    """x, B, C as slices of one activated tensor, dt before its softplus;
    (device tensors, fp64 values)."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((*lead, H * P + 2 * G * N))
    mixed, m64 = rounded(z / (1 + np.exp(-z)), dtype)
    dt, dt64 = rounded(0.5 * rng.standard_normal((*lead, H)), dtype)
    step = np.exp(rng.uniform(np.log(steps[0]), np.log(steps[1]), H))
    bias, b64 = rounded(step + np.log(-np.expm1(-step)), torch.float32)
    A, a64 = rounded(-rng.uniform(*decay, H), torch.float32)
    D, d64 = rounded(1 + 0.1 * rng.standard_normal(H), torch.float32)
    dev = mixed.cuda()

    def cut(v):
        x, B, C = v[..., :H * P], v[..., H * P:H * P + G * N], v[..., H * P + G * N:]
        return x.reshape(*lead, H, P), B.reshape(*lead, G, N), C.reshape(*lead, G, N)

    x = dev[..., :H * P].unflatten(-1, (H, P))
    B = dev[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    C = dev[..., H * P + G * N:].unflatten(-1, (G, N))
    t = dict(x=x, dt=dt.cuda(), A=A.cuda(), B=B, C=C, D=D.cuda(), dt_bias=bias.cuda())
    x64, B64, C64 = cut(m64)
    return t, dict(x=x64, dt=dt64, A=a64, B=B64, C=C64, D=d64, dt_bias=b64)
