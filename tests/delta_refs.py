"""The gated delta rule token by token in 64 bits on the CPU, and host-side
caches in the layout of include/ssu_delta.h: what the tests compare with."""
import math

import torch

EPS = 1e-6


def gates(dt, beta, A, dt_bias, softplus=True, sigmoid=True):
    """g, b in 64 bits [rows, hv]."""
    z = dt.double() + dt_bias.double()
    z = torch.nn.functional.softplus(z) if softplus else z
    return A.double() * z, torch.sigmoid(beta.double()) if sigmoid else beta.double()


def unit(x, norm=True):
    x = x.double()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) if norm else x


def run(S, q, k, v, g, b, scale, norm=True):
    """S [hv, dv, dk]; q, k [n, hk, dk], v [n, hv, dv], g, b [n, hv]: (final
    state, outputs [n, hv, dv]), everything in 64 bits; q may be None."""
    S = S.double().clone()
    r = v.shape[1] // k.shape[1]
    out = torch.zeros(v.shape, dtype=torch.float64)
    for t in range(v.shape[0]):
        kt = unit(k[t], norm).repeat_interleave(r, 0)
        S = torch.exp(g[t])[:, None, None] * S
        u = b[t][:, None] * (v[t].double() - (S * kt[:, None, :]).sum(-1))
        S = S + u[:, :, None] * kt[:, None, :]
        if q is not None:
            out[t] = scale * (S * unit(q[t], norm).repeat_interleave(r, 0)[:, None, :]).sum(-1)
    return S, out


def tile_index(dv, dk, e):
    """Flat place, in a head's tiled checkpoint of e-byte values, of value (p, n)."""
    p, n = torch.meshgrid(torch.arange(dv), torch.arange(dk), indexing="ij")
    t, q, r = n // 16, n // 4 % 4, n % 4
    i, lane, per = 4 * t + r, 16 * q + p % 16, 16 // e
    return (p // 16) * 16 * dk + (i // per * 64 + lane) * per + i % per


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Cache:
    """A random cache on the CPU; `pad` bytes behind every slot page hold 0xA5."""

    def __init__(self, gen, slots, hk, hv, dk, dv, L, state, pad=0):
        self.slots, self.hk, self.hv, self.dk, self.dv, self.L, self.state_dtype, self.pad = slots, hk, hv, dk, dv, L, state, pad
        rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        g = -torch.exp(math.log(0.004) + (math.log(2.0) - math.log(0.004)) * torch.rand(slots, hv, L, generator=gen))
        b = torch.rand(slots, hv, L, generator=gen)
        self.t = dict(state=(0.3 * rnd(slots, hv * dv * dk)).to(TYPES[state]),
                      k_cache=rnd(slots, hk * L * dk).bfloat16(), v_cache=rnd(slots, hv * L * dv).bfloat16(),
                      gate_cache=torch.stack([g, b], -1).reshape(slots, -1).contiguous())
        self.ring_start = torch.randint(0, L, (slots,), generator=gen, dtype=torch.int32)
        self.place = tile_index(dv, dk, TYPES[state].itemsize).reshape(-1)

    def states(self, slot):
        """[hv, dv, dk] in the checkpoint's type."""
        return self.t["state"][slot].view(self.hv, -1)[:, self.place].view(self.hv, self.dv, self.dk)

    def ring(self, slot, first, count):
        """k, v, g, b of `count` tokens from live token `first` on."""
        at = (int(self.ring_start[slot]) + first + torch.arange(count)) % self.L
        k = self.t["k_cache"][slot].view(self.hk, self.L, self.dk)[:, at].transpose(0, 1)
        v = self.t["v_cache"][slot].view(self.hv, self.L, self.dv)[:, at].transpose(0, 1)
        g = self.t["gate_cache"][slot].view(self.hv, self.L, 2)[:, at].transpose(0, 1).double()
        return k, v, g[..., 0], g[..., 1]

    def upload(self, ssu, dev, norm=True):
        """Device tensors (bytes, with the padding) and the DeltaCache."""
        d = {}
        for name, t in self.t.items():
            raw = t.contiguous().view(torch.uint8).view(self.slots, -1)
            d[name] = torch.nn.functional.pad(raw, (0, self.pad), value=0xA5).to(dev)
        d["ring_start"] = self.ring_start.to(dev)
        d["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        dc = ssu.DeltaCache(self.slots, self.hk, self.hv, self.L, self.state_dtype, d["state"], d["k_cache"], d["v_cache"],
                            d["gate_cache"], d["ring_start"], d["status"], dim_k=self.dk, dim_v=self.dv, qk_norm=norm)
        return d, dc

    def download(self, d):
        """The device bytes as host tensors, the padding checked."""
        out = {}
        for name, t in self.t.items():
            raw = d[name].cpu()
            if self.pad:
                assert bool((raw[:, -self.pad:] == 0xA5).all()), name + ": padding written"
                raw = raw[:, :-self.pad]
            out[name] = raw.contiguous().view(t.dtype).view(t.shape)
        out["ring_start"] = d["ring_start"].cpu()
        return out


def inputs(gen, rows, hk, hv, dk, dv, wide=0):
    """q, k, v (slices of rows `wide` values wider), dt, beta, A, dt_bias."""
    x = torch.randn(rows, 2 * hk * dk + hv * dv + wide, generator=gen).bfloat16()
    q = x[:, :hk * dk].view(rows, hk, dk) if not wide else x[:, :hk * dk].unflatten(1, (hk, dk))
    k = x[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
    v = x[:, 2 * hk * dk:2 * hk * dk + hv * dv].unflatten(1, (hv, dv))
    return dict(q=q, k=k, v=v, dt=0.5 * torch.randn(rows, hv, generator=gen), beta=torch.randn(rows, hv, generator=gen),
                A=-torch.exp(math.log(16.0) * torch.rand(hv, generator=gen)), dt_bias=-4 + 2 * torch.rand(hv, generator=gen))


# Tolerances, of 2-norms over one (entry, head): a kernel's value is a chain of
# three products (keys with the state, T with the residuals, the update or the
# readout) of depths up to dim_k and w, each summed in fp32 from operands that
# keep 24 bits, so it is off by at most 3 (dim_k + w) 2^-24 of the norms it is
# made of; the update with unit keys and b <= 1 never makes an earlier error
# larger, so errors of later windows add.  The norms: the result's own and, as
# the products may cancel, that of what went in (states and values).  Results
# rounded to a type add half a step of it; operands towards bf16 outputs and
# 16-bit checkpoints keep 16 bits, two parts on either side of a product: 3 x 2
# x 2^-17.  (A prompt's and a flush's products with an fp32 state take it in two
# parts as well, off by at most 2^-18 a value and at random: over the 64 and
# more values of a row less than a fifth of 3 (dim_k + w) 2^-24, which counts
# every addition of the sums at its worst.)
def tol(dk, w, windows, dtype, state=None):
    """(part of the result's norm: its rounding, part of every norm)."""
    t = 3 * (dk + w) * 2.0 ** -24 * windows
    if "bf16" in (dtype, state) or "f16" in (dtype, state):
        t += 6 * 2.0 ** -17 * windows
    return {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}[dtype], t


def check(got, want, went_in, limits, what):
    """||got - want|| within the limits for every leading index; went_in: the
    norm of what the products were made of, a number or one per index."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), what + ": not finite"
    if got.numel() == 0:
        return
    off = (got - want).flatten(1).norm(dim=1)
    size = want.flatten(1).norm(dim=1)
    allowed = limits[0] * size + limits[1] * (size + went_in)
    at = int((off / allowed.clamp(min=1e-30)).argmax())
    assert bool((off <= allowed).all()), "%s: [%d] off by %.3g, %.3g allowed (norm %.3g)" % (
        what, at, off[at], allowed[at], size[at])
