"""The selective state update token by token in 64 bits on the CPU, what an
error of its pieces can amount to, and random prompts."""
import math

import torch


def gates(dt, A, dt_bias, softplus=True):
    """(dt', A dt') in 64 bits [rows, H]."""
    v = dt.double() + dt_bias.double()
    d = torch.nn.functional.softplus(v) if softplus else v
    return d, A.double() * d


def run(S, x, B, C, d, g, D):
    """S [H, 64, 128]; x [n, H, 64], B, C [n, G, 128], d, g [n, H], D [H]: (final
    state, outputs [n, H, 64]) in 64 bits."""
    S = S.double().clone()
    r = x.shape[1] // B.shape[1]
    out = torch.zeros(x.shape, dtype=torch.float64)
    x, B, C = x.double(), B.double().repeat_interleave(r, 1), C.double().repeat_interleave(r, 1)
    for t in range(x.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S + (d[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
        out[t] = (S * C[t][:, None, :]).sum(-1) + D.double()[:, None] * x[t]
    return S, out


def gate(y, z):
    z = z.double()
    return y * z * torch.sigmoid(z)


def inputs(gen, rows, H, G, wide=0, decay=True):
    """x, B, C as slices of rows `wide` values wider, z likewise; dt, A, D, dt_bias (decay False: hardly any)."""
    r = torch.randn(rows, H * 64 + 2 * G * 128 + wide, generator=gen).bfloat16()
    z = torch.randn(rows, H * 64 + wide, generator=gen).bfloat16()
    return dict(x=r[:, :H * 64].unflatten(1, (H, 64)), B=r[:, H * 64:H * 64 + G * 128].unflatten(1, (G, 128)),
                C=r[:, H * 64 + G * 128:H * 64 + 2 * G * 128].unflatten(1, (G, 128)), z=z[:, :H * 64].unflatten(1, (H, 64)),
                dt=0.5 * torch.randn(rows, H, generator=gen),
                A=-torch.exp(math.log(16.0) * torch.rand(H, generator=gen)) * (1.0 if decay else 1e-4),
                D=torch.randn(H, generator=gen), dt_bias=-4 + 2 * torch.rand(H, generator=gen))


# Tolerances, of single values.  With every operand taken by its absolute value
# the rule gives y_abs and S_abs, which bound what any partial sum of a value can
# reach (A dt' <= 0).  A sum of n products in fp32 is off by at most n 2^-24 of
# that; operands in three parts make it 3 n sums.  A chunk of 64 tokens adds
# (3 x 64 + 8) 2^-24 S_abs to a state's error (its update, its decay, dt' and the
# weights, a few roundings each), which later decays only make smaller; the
# joining of segments adds no more than a chunk.  An output is the readout (3 x
# 128), the chunk's tokens (3 x 64) and as many roundings again as a chunk's gates;
# dt' itself, through softplus, is within 2^-21 (8 half steps).  Towards bf16 outputs the
# state and the weights keep two parts, off by at most 2^-17 together, and the result is rounded once: 2^-8 of it.
def tol_state(tokens):
    return (math.ceil(tokens / 64) + 1) * (3 * 64 + 16) * 2.0 ** -24


def tol_out(tokens, out):
    t = tol_state(tokens) + (3 * 128 + 3 * 64 + 32) * 2.0 ** -24
    return (2.0 ** -8, t + 2.0 ** -17) if out == "bf16" else (2.0 ** -24, t)


def check(got, want, size, limits, what):
    """|got - want| <= limits[0] |want| + limits[1] size, value by value."""
    got, want = got.cpu().double(), want.double()
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), what + ": not finite"
    if got.numel() == 0:
        return
    off, allowed = (got - want).abs(), limits[0] * want.abs() + limits[1] * size + 1e-37
    worst = float((off / allowed).max())
    assert worst <= 1.0, "%s: %.3g times what is allowed" % (what, worst)
