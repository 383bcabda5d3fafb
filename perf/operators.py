"""Cases and plain forms of the gated delta rule and of draft verification.

Three groups of operators of speculative decode, each in its plain form (elementary torch operations in 32 bits) and,
with `own`, as calls of speculative_replay_state_amd:

  prefill  the gated delta rule over whole prompts (varlen), from given or zero states to outputs and final states
  step     the rule for a few new tokens of every request, read out from a checkpoint that is replayed through the
           tokens of a ring, the checkpoint unchanged
  flush    accepted tokens of the ring folded into the checkpoint
  verify   drafted tokens accepted or rejected against the target's probabilities from given uniform numbers, one
           more token drawn, and the ring bookkeeping that follows from the count

The rule, per value head with state S [dim_v, dim_k], g_t = A softplus(dt_t + dt_bias) and b_t = sigmoid(beta_t), k and
q scaled to unit length (k / sqrt(sum k^2 + 1e-6)), q also by dim_k^-1/2:

  S <- exp(g_t) S;  u_t = b_t (v_t - S k_t);  S <- S + u_t k_t^T;  o_t = S q_t.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
PAD = 1  # slot 0 of a cache is the padding slot


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a few short prompts arriving together: launch and chain latency
        dict(name="prefill_short", op="prefill", seqs=4, max_len=48, hk=8, hv=16, dk=128, dv=128, init=False),
        # a ragged batch of prompts with narrow heads
        dict(name="prefill_ragged", op="prefill", seqs=16, max_len=701, hk=16, hv=32, dk=64, dv=64, init=False),
        # one long document continued from a state: few independent chains, each of them long
        dict(name="prefill_long", op="prefill", seqs=1, max_len=16384, hk=8, hv=32, dk=128, dv=128, init=True),
        # a full batch of prompts of a layer with 64 heads
        dict(name="prefill_batch", op="prefill", seqs=8, max_len=4096, hk=8, hv=64, dk=128, dv=128, init=False),
        # one request, one token: the latency of the smallest decode
        dict(name="step_one", op="step", batch=1, T=1, varlen=False, hk=8, hv=16, dk=128, dv=128, ring=16, live=4,
             state="bf16", out="bf16"),
        # a decode batch with three drafts a request
        dict(name="step_drafts", op="step", batch=64, T=4, varlen=False, hk=8, hv=64, dk=128, dv=128, ring=16, live=4,
             state="bf16", out="bf16"),
        # a large ragged decode batch with fp32 checkpoints and fp32 outputs
        dict(name="step_large", op="step", batch=256, T=8, varlen=True, hk=8, hv=64, dk=128, dv=128, ring=16, live=8,
             state="f32", out="f32"),
        # accepted tokens of a decode batch folded, bf16 and fp32 checkpoints
        dict(name="flush_batch", op="flush", batch=64, hk=8, hv=64, dk=128, dv=128, ring=16, fold=8, state="bf16"),
        dict(name="flush_large", op="flush", batch=128, hk=8, hv=64, dk=128, dv=128, ring=32, fold=17, state="f32"),
        # one request's drafts: latency of the row's scan
        dict(name="verify_one", op="verify", batch=1, T=4, vocab=32000, ring=16, probs="f32", onehot=False),
        # a decode batch, an odd vocabulary, drafts without a distribution of their own
        dict(name="verify_batch", op="verify", batch=64, T=4, vocab=100003, ring=16, probs="f32", onehot=True),
        # a large decode batch with both distributions in bf16
        dict(name="verify_large", op="verify", batch=256, T=8, vocab=131072, ring=16, probs="bf16", onehot=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    hk = rng.choice([1, 2, 4, 8, 16])
    r = rng.choice([1, 2, 3, 4, 8])
    while hk * r > most:
        hk = max(1, hk // 2)
        r = max(1, r - 1)
    return hk, hk * r


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "step", "flush", "verify"])
    if op == "prefill":
        seqs = _log(rng, 1, 32)
        hk, hv = _heads(rng, 64)
        # at most the tokens x heads of the largest listed case, and no longer a chain
        max_len = _log(rng, 1, max(2, min(12000, 1500000 // (seqs * hv))))
        return dict(op=op, seqs=seqs, max_len=max_len, hk=hk, hv=hv, dk=rng.choice([64, 128]),
                    dv=rng.choice([64, 128]), init=rng.random() < 0.5)
    if op == "step":
        hk, hv = _heads(rng, 64)
        ring = rng.choice([5, 8, 16, 16, 23, 32])
        T = rng.randint(1, min(16, ring))
        return dict(op=op, batch=_log(rng, 1, 200), T=T, varlen=rng.random() < 0.5, hk=hk, hv=hv,
                    dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), ring=ring, live=rng.randint(0, ring - T),
                    state=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16"]))
    if op == "flush":
        hk, hv = _heads(rng, 64)
        ring = rng.choice([5, 8, 16, 16, 23, 32])
        return dict(op=op, batch=_log(rng, 1, 128), hk=hk, hv=hv, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    ring=ring, fold=rng.randint(1, ring), state=rng.choice(["f32", "bf16", "f16"]))
    return dict(op=op, batch=_log(rng, 1, 250), T=rng.randint(1, 8), vocab=_log(rng, 200, 130001), ring=16,
                probs=rng.choice(["f32", "bf16", "f16"]), onehot=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _lengths(g, n, most):
    """Between half and the whole of `most`, evenly, one of them whole: the same lengths for every seed (outputs keep
    their shapes), in an order of the seed's."""
    lo = (most + 1) // 2
    v = torch.tensor([most - (most - lo) * i // max(1, n - 1) for i in range(n)], device=DEV)
    return v[torch.randperm(n, generator=g, device=DEV)]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(g, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(*shape, generator=g, device=DEV)


def _qkv(g, rows, c):
    """q, k and v as a projection leaves them: slices of one tensor's rows."""
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    x = _randn(g, rows, 2 * hk * dk + hv * dv).to(torch.bfloat16)
    q = x[:, :hk * dk].view(rows, hk, dk)
    k = x[:, hk * dk:2 * hk * dk].view(rows, hk, dk)
    v = x[:, 2 * hk * dk:].view(rows, hv, dv)
    return q, k, v


def _gates(g, rows, hv):
    return dict(dt=0.5 * _randn(g, rows, hv), beta=_randn(g, rows, hv), A=-torch.exp(_uniform(g, 0.0, math.log(16.0), hv)),
                dt_bias=_uniform(g, -4.0, -2.0, hv))


def _cu(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), lens.cumsum(0)]).to(torch.int32)


def _cache(g, c, slots):
    """A cache of random requests: checkpoints, ring entries (live and dead) and ring starts."""
    hk, hv, dk, dv, L = c["hk"], c["hv"], c["dk"], c["dv"], c["ring"]
    gates = torch.stack([-torch.exp(_uniform(g, math.log(0.004), math.log(2.0), slots, hv, L)),
                         torch.rand(slots, hv, L, generator=g, device=DEV)], dim=-1)
    return dict(state=(0.1 * _randn(g, slots, hv * dv * dk)).to(_TYPES[c["state"]]),
                k_cache=_randn(g, slots, hk, L, dk).to(torch.bfloat16), v_cache=_randn(g, slots, hv, L, dv).to(torch.bfloat16),
                gate_cache=gates, ring_start=torch.randint(0, L, (slots,), generator=g, device=DEV, dtype=torch.int32))


def _slots(g, batch):
    """Distinct slots in no order; a quarter of the cache is other requests'."""
    n = PAD + batch + (batch + 3) // 4
    ids = PAD + torch.randperm(n - PAD, generator=g, device=DEV)[:batch]
    return n, ids.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, op = dict(case), case["op"]
    s = dict(c=c)
    if op == "prefill":
        lens = _lengths(g, c["seqs"], c["max_len"])
        s["lens"] = lens.tolist()
        s["rows"] = rows = sum(s["lens"])
        s["cu"] = _cu(lens)
        s["q"], s["k"], s["v"] = _qkv(g, rows, c)
        s.update(_gates(g, rows, c["hv"]))
        shape = (c["seqs"], c["hv"], c["dv"], c["dk"])
        s["initial"] = 0.1 * _randn(g, *shape) if c["init"] else None
        s["out"] = torch.zeros(rows, c["hv"], c["dv"], dtype=torch.bfloat16, device=DEV)
        s["final"] = torch.zeros(shape, device=DEV)
    elif op == "step":
        n, s["ids"] = _slots(g, c["batch"])
        s["cache"] = _cache(g, c, n)
        lens = _lengths(g, c["batch"], c["T"]) if c["varlen"] else torch.full((c["batch"],), c["T"], device=DEV)
        rows = int(lens.sum())
        s["lens"], s["cu"], s["rows"] = lens, _cu(lens), rows
        s["live"] = torch.randint(0, c["live"] + 1, (c["batch"],), generator=g, device=DEV, dtype=torch.int32)
        s["q"], s["k"], s["v"] = _qkv(g, rows, c)
        s.update(_gates(g, rows, c["hv"]))
        s["out"] = torch.zeros(rows, c["hv"], c["dv"], dtype=_TYPES[c["out"]], device=DEV)
    elif op == "flush":
        n, s["ids"] = _slots(g, c["batch"])
        s["cache"] = _cache(g, c, n)
        s["fold"] = _lengths(g, c["batch"], c["fold"]).to(torch.int32)
    else:
        b, T, V = c["batch"], c["T"], c["vocab"]
        logits = 3.0 * _randn(g, b * T, V)
        draft = torch.softmax(logits + 0.7 * _randn(g, b * T, V), dim=-1)
        s["target"] = torch.softmax(logits, dim=-1).to(_TYPES[c["probs"]])
        picked = torch.multinomial(draft, 1, generator=g)[:, 0].view(b, T)
        # row t of a request is the token that was fed; the draft of row t is fed in row t + 1
        s["tokens"] = torch.cat([torch.randint(0, V, (b, 1), generator=g, device=DEV), picked[:, :-1]],
                                dim=1).reshape(-1).to(torch.int32)
        s["draft"] = None if c["onehot"] else draft.to(_TYPES[c["probs"]])
        s["u"] = torch.rand(b * T, generator=g, device=DEV)
        if c["onehot"]:  # drafts of a lookup: accepted about half of the time
            s["u"] = s["u"] * 2.0 * s["target"].float().gather(1, picked.view(-1, 1))[:, 0]
        s["u_final"] = torch.rand(b, generator=g, device=DEV)
        s["live"] = torch.randint(0, c["ring"] - T + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        s["fold"] = (torch.rand(b, generator=g, device=DEV) * (s["live"] + 1)).to(torch.int32)
        s["out_tokens"] = torch.zeros(b, T, dtype=torch.int32, device=DEV)
        s["accepted"], s["next_live"], s["next_fold"] = (torch.zeros(b, dtype=torch.int32, device=DEV) for _ in range(3))
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors and workspaces that a program keeps beside its tensors."""
    import speculative_replay_state_amd as ssu
    c, op = s["c"], s["c"]["op"]
    s["ssu"] = ssu
    if op == "prefill":
        ws = torch.empty(max(ssu.delta_prefill_workspace_size(s["rows"], c["seqs"], c["hv"]), 16), dtype=torch.uint8, device=DEV)
        s["call"] = ssu.make_delta_prefill(s["cu"], s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["dt_bias"], s["out"],
                                           initial_states=s["initial"], final_states=s["final"], workspace=ws)
    elif op in ("step", "flush"):
        t = s["cache"]
        s["dc"] = ssu.DeltaCache(t["state"].shape[0], c["hk"], c["hv"], c["ring"], c["state"], t["state"], t["k_cache"],
                                 t["v_cache"], t["gate_cache"], t["ring_start"], dim_k=c["dk"], dim_v=c["dv"])
        if op == "step":
            s["call"] = ssu.make_delta_step(s["dc"], c["T"], s["ids"], s["live"], s["cu"] if c["varlen"] else None, s["q"],
                                            s["k"], s["v"], s["dt"], s["beta"], s["A"], s["dt_bias"], s["out"])
    else:
        ws = torch.empty(max(ssu.verify_workspace_size(c["batch"], c["vocab"]), 16), dtype=torch.uint8, device=DEV)
        s["call"] = ssu.make_verify(s["tokens"], s["target"], s["draft"], s["u"], s["u_final"], s["out_tokens"], s["accepted"],
                                    workspace=ws, live=s["live"], fold=s["fold"], ring_len=c["ring"],
                                    next_live=s["next_live"], next_fold=s["next_fold"])


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------

def run(state):
    s, op = state, state["c"]["op"]
    if own:
        return _own(s, op)
    return dict(prefill=_plain_prefill, step=_plain_step, flush=_plain_flush, verify=_plain_verify)[op](s)


def _own(s, op):
    ssu = s["ssu"]
    if op == "prefill":
        ssu.delta_prefill(s["call"])
        return dict(out=s["out"], final=s["final"])
    if op == "step":
        ssu.delta_replay_step(s["dc"], s["call"])
        return dict(out=s["out"], k_cache=s["cache"]["k_cache"], v_cache=s["cache"]["v_cache"], gate_cache=s["cache"]["gate_cache"])
    if op == "flush":
        ssu.delta_flush(s["dc"], s["ids"], s["fold"])
        return dict(state=s["cache"]["state"], ring_start=s["cache"]["ring_start"])
    ssu.verify(s["call"])
    return dict(tokens=s["out_tokens"], accepted=s["accepted"], live=s["next_live"], fold=s["next_fold"])


def _tile(h, dv, dk):
    """[..., dv, dk] -> the checkpoint's order: rows in blocks of 16, lane 16 q + m of a block holds row m's values
    n = 16 t + 4 q + r, in 16-byte chunks, chunk u of all lanes side by side."""
    e = 16 // h.element_size()
    x = h.reshape(*h.shape[:-2], dv // 16, 16, dk // 16, 4, 4)     # block, m, t, q, r
    x = x.movedim(-2, -4)                                          # block, q, m, t, r
    lead = x.dim() - 5
    x = x.transpose(lead + 1, lead + 1).reshape(*h.shape[:-2], dv // 16, 4, 16, dk // 4 // e, e)
    return x.movedim(-2, -4).reshape(*h.shape[:-2], dv * dk)       # block, u, q, m, e


def _untile(x, dv, dk):
    e = 16 // x.element_size()
    y = x.reshape(*x.shape[:-1], dv // 16, dk // 4 // e, 4, 16, e).movedim(-4, -2)  # block, q, m, u, e
    y = y.reshape(*x.shape[:-1], dv // 16, 4, 16, dk // 16, 4).movedim(-4, -2)      # block, m, t, q, r
    return y.reshape(*x.shape[:-1], dv, dk)


def _unit(x):
    x = x.float()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _gate(s):
    """(g, b) of the new rows, f32 [rows, hv]."""
    return s["A"] * _softplus(s["dt"] + s["dt_bias"]), 1 / (1 + torch.exp(-s["beta"]))


def _window(k, G, b):
    """For windows of tokens [..., w, dk] (unit keys, running decays G in 64 bits, b 0 where there is no token): the decay
    matrix exp(G_i - G_j) for j <= i and (I + A)^-1, A_ij = b_i exp(G_i - G_j) k_i.k_j for j < i."""
    w = k.shape[-2]
    low = torch.ones(w, w, dtype=torch.bool, device=k.device).tril()
    decay = torch.where(low, torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], 0.0)).float(), 0.0)
    power = -(b[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    inverse = torch.eye(w, device=k.device) + power
    for _ in range(max(0, (w - 1).bit_length() - 1)):
        power = power @ power
        inverse = inverse + inverse @ power
    return decay, inverse


def _plain_prefill(s):
    c, C = s["c"], 64
    n, hk, hv, dk, dv = c["seqs"], c["hk"], c["hv"], c["dk"], c["dv"]
    nc = -(-c["max_len"] // C)
    at = s["cu"][:-1, None] + torch.arange(nc * C, device=DEV)[None]
    there = at < s["cu"][1:, None]
    at = torch.where(there, at, 0).long()

    def chunks(x):  # [rows, h, d] -> [n, h, nc, C, d]
        return x[at].transpose(1, 2).reshape(n, x.shape[1], nc, C, x.shape[2])

    def wide(x):  # key heads -> value heads
        return x.repeat_interleave(hv // hk, dim=1)

    gt, bt = _gate(s)
    q, k, v = wide(chunks(_unit(s["q"]) * dk ** -0.5)), wide(chunks(_unit(s["k"]))), chunks(s["v"].float())
    here = there.view(n, 1, nc, C)
    G = torch.where(here, chunks(gt[..., None])[..., 0], 0.0).double().cumsum(-1)
    b = torch.where(here, chunks(bt[..., None])[..., 0], 0.0)
    decay, inverse = _window(k, G, b)
    e = torch.exp(G).float()[..., None]
    W, U = inverse @ (b[..., None] * e * k), inverse @ (b[..., None] * v)
    P = decay * (q @ k.transpose(-1, -2))
    q = q * e
    rest = torch.exp(G[..., -1:] - G).float()[..., None] * k
    last = torch.exp(G[..., -1]).float()[..., None, None]
    h = s["initial"].transpose(-1, -2).contiguous() if s["initial"] is not None else torch.zeros(n, hv, dk, dv, device=DEV)
    o = torch.empty(n, hv, nc, C, dv, device=DEV)
    for i in range(nc):
        u = U[:, :, i] - W[:, :, i] @ h
        o[:, :, i] = q[:, :, i] @ h + P[:, :, i] @ u
        h = last[:, :, i] * h + rest[:, :, i].transpose(-1, -2) @ u
    o = o.reshape(n, hv, nc * C, dv).transpose(1, 2)[there]
    s["out"].copy_(o)
    s["final"].copy_(h.transpose(-1, -2))
    return dict(out=s["out"], final=s["final"])


def _ring(s, first, count):
    """Ring positions of `count` tokens after the ring start: [batch, count] and the slots."""
    slot = s["ids"].long()
    return slot, (s["cache"]["ring_start"][slot].long()[:, None] + first + torch.arange(count, device=DEV)) % s["c"]["ring"]


def _plain_step(s):
    c, t = s["c"], s["cache"]
    hk, hv, dk, dv, T = c["hk"], c["hv"], c["dk"], c["dv"], c["T"]
    slot = s["ids"].long()
    live = s["live"].long()[:, None]
    gt, bt = _gate(s)
    # append the new tokens
    off = torch.arange(T, device=DEV)[None]
    new = off < s["lens"][:, None]
    row = torch.where(new, s["cu"][:-1, None] + off, 0).long()
    at = (t["ring_start"][slot].long()[:, None] + live + off) % c["ring"]
    si, pi, ri = slot[:, None].expand(-1, T)[new], at[new], row[new]
    t["k_cache"][si, :, pi] = s["k"][ri]
    t["v_cache"][si, :, pi] = s["v"][ri]
    t["gate_cache"][si, :, pi] = torch.stack([gt, bt], dim=-1)[ri]
    # the window: live tokens, then new ones
    w = c["live"] + T
    _, pos = _ring(s, 0, w)
    here = (torch.arange(w, device=DEV)[None] < live + s["lens"][:, None])[:, None]  # [batch, 1, w]

    def win(x):  # ring tensor -> [batch, h, w, ...]
        return x[slot[:, None], :, pos].transpose(1, 2)

    gates = win(t["gate_cache"])
    G = torch.where(here, gates[..., 0], 0.0).double().cumsum(-1)
    b = torch.where(here, gates[..., 1], 0.0)
    k = _unit(win(t["k_cache"])).repeat_interleave(hv // hk, dim=1)
    v = win(t["v_cache"]).float()
    decay, inverse = _window(k, G, b)
    h = _untile(t["state"][slot].view(-1, hv, dv * dk), dv, dk).float()
    e = torch.exp(G).float()[..., None]
    u = inverse @ (b[..., None] * (v - e * (k @ h.transpose(-1, -2))))
    q = (_unit(s["q"]) * dk ** -0.5).repeat_interleave(hv // hk, dim=1)[row].transpose(1, 2)  # [batch, hv, T, dk]
    mine = (live + off).clamp(max=w - 1)[:, None, :, None].expand(-1, hv, -1, -1)
    P = decay.gather(2, mine.expand(-1, -1, -1, w)) * (q @ k.transpose(-1, -2))
    o = e.gather(2, mine) * (q @ h.transpose(-1, -2)) + P @ u
    s["out"].copy_(o.transpose(1, 2)[new])
    return dict(out=s["out"], k_cache=t["k_cache"], v_cache=t["v_cache"], gate_cache=t["gate_cache"])


def _plain_flush(s):
    c, t = s["c"], s["cache"]
    hk, hv, dk, dv, w = c["hk"], c["hv"], c["dk"], c["dv"], c["fold"]
    slot, pos = _ring(s, 0, w)
    here = (torch.arange(w, device=DEV)[None] < s["fold"][:, None])[:, None]

    def win(x):
        return x[slot[:, None], :, pos].transpose(1, 2)

    gates = win(t["gate_cache"])
    G = torch.where(here, gates[..., 0], 0.0).double().cumsum(-1)
    b = torch.where(here, gates[..., 1], 0.0)
    k = _unit(win(t["k_cache"])).repeat_interleave(hv // hk, dim=1)
    v = win(t["v_cache"]).float()
    _, inverse = _window(k, G, b)
    h = _untile(t["state"][slot].view(-1, hv, dv * dk), dv, dk).float()
    e = torch.exp(G).float()[..., None]
    u = inverse @ (b[..., None] * (v - e * (k @ h.transpose(-1, -2))))
    u = u * torch.exp(G[..., -1:] - G).float()[..., None]
    h = torch.exp(G[..., -1]).float()[..., None, None] * h + u.transpose(-1, -2) @ k
    t["state"][slot] = _tile(h.to(t["state"].dtype), dv, dk).view(len(slot), -1)
    t["ring_start"][slot] = ((t["ring_start"][slot] + s["fold"]) % c["ring"]).to(torch.int32)
    return dict(state=t["state"], ring_start=t["ring_start"])


def _plain_verify(s):
    c = s["c"]
    b, T, V = c["batch"], c["T"], c["vocab"]
    target = s["target"].view(b, T, V)
    drafted = s["tokens"].view(b, T)[:, 1:].long()
    p = target[:, :-1].gather(2, drafted[..., None])[..., 0].double()
    q = s["draft"].view(b, T, V)[:, :-1].gather(2, drafted[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p)
    n = (s["u"].view(b, T)[:, :-1].double() * q < p).to(torch.int32).cumprod(1).sum(1)
    i = torch.arange(b, device=DEV)
    r = target[i, n].float()
    if s["draft"] is not None:
        less = s["draft"].view(b, T, V)[i, n].float()
    else:
        tok = torch.cat([drafted, torch.zeros(b, 1, dtype=torch.int64, device=DEV)], dim=1)[i, n]
        less = (torch.arange(V, device=DEV)[None] == tok[:, None]).float()
    r = torch.where((n < T - 1)[:, None], (r - less).clamp(min=0), r)
    total = r.double().cumsum(1)
    drawn = torch.searchsorted(total, s["u_final"].double()[:, None] * total[:, -1:], right=True)[:, 0]
    off = torch.arange(T, device=DEV)[None]
    fed = torch.cat([drafted, torch.zeros(b, 1, dtype=torch.int64, device=DEV)], dim=1)
    s["out_tokens"].copy_(torch.where(off < n[:, None], fed, torch.where(off == n[:, None], drawn[:, None], -1)))
    s["accepted"].copy_(n + 1)
    s["next_live"].copy_(s["live"] - s["fold"] + n + 1)
    s["next_fold"].copy_(torch.where(s["next_live"] + T > c["ring"], s["next_live"], 0))
    return dict(tokens=s["out_tokens"], accepted=s["accepted"], live=s["next_live"], fold=s["next_fold"])


# ---------------------------------------------------------------------------
# what a pass needs
# ---------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op == "verify":
        # the row that is drawn from (both distributions unless every draft was accepted), and a few words
        row = c["vocab"] * (4 if c["probs"] == "f32" else 2)
        return dict(bytes=c["batch"] * (row * (1 if c["onehot"] else 2) + c["T"] * 16 + 24), flops=c["batch"] * c["vocab"] * 3)
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    if op == "prefill":
        rows = c["max_len"] if c["seqs"] == 1 else int(0.75 * c["seqs"] * c["max_len"])
        states = c["seqs"] * hv * dk * dv * 4
        return dict(bytes=rows * (2 * hk * dk * 2 + 2 * hv * dv * 2 + hv * 8) + states * (2 if c["init"] else 1),
                    flops=rows * hv * (6 * dk * dv + 4 * dk))
    size = 4 if c["state"] == "f32" else 2
    token = hk * dk * 2 + hv * dv * 2 + hv * 8
    state = c["batch"] * hv * dk * dv * size
    if op == "step":
        T = c["T"] * (0.75 if c["varlen"] else 1.0)
        new, live = c["batch"] * T, c["batch"] * c["live"] / 2
        return dict(bytes=state + live * token + new * (2 * token + hk * dk * 2 + hv * dv * (4 if c["out"] == "f32" else 2)),
                    flops=hv * dk * dv * (2 * new + 4 * (new + live)))
    k = c["batch"] * c["fold"] * 0.75
    return dict(bytes=2 * state + k * token, flops=k * hv * 6 * dk * dv)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token
# ---------------------------------------------------------------------------

def _recur(h, q, k, v, g, b):
    """One token for every row of `h` [..., dv, dk] in 64 bits; returns (state, output or None)."""
    h = torch.exp(g)[..., None, None] * h
    u = b[..., None] * (v - (h * k[..., None, :]).sum(-1))
    h = h + u[..., :, None] * k[..., None, :]
    return h, None if q is None else (h * q[..., None, :]).sum(-1)


def _gate64(s):
    z = s["dt"].double() + s["dt_bias"].double()
    return s["A"].double() * (torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))), torch.sigmoid(s["beta"].double())


def _unit64(x, times=1.0):
    x = x.double()
    return times * x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return dict(prefill=_exact_prefill, step=_exact_step, flush=_exact_flush, verify=_exact_verify)[case["op"]](s)


def _exact_prefill(s):
    c = s["c"]
    r = c["hv"] // c["hk"]
    order = sorted(range(c["seqs"]), key=lambda i: -s["lens"][i])  # longest first: the first m are still running
    cu = s["cu"].tolist()
    g, b = _gate64(s)
    start = torch.tensor([cu[i] for i in order], device=DEV)
    h = s["initial"].double()[order] if s["initial"] is not None else torch.zeros(c["seqs"], c["hv"], c["dv"], c["dk"], dtype=torch.float64, device=DEV)
    out = torch.empty(s["rows"], c["hv"], c["dv"], dtype=torch.float64, device=DEV)
    if c["max_len"] * (1 + c["seqs"] * c["hv"] * c["dk"] * c["dv"] * 40 / 3e9) > 60000:
        return None
    for t in range(c["max_len"]):
        m = sum(1 for i in order if s["lens"][i] > t)
        at = start[:m] + t
        q = _unit64(s["q"][at], c["dk"] ** -0.5).repeat_interleave(r, dim=1)
        k = _unit64(s["k"][at]).repeat_interleave(r, dim=1)
        new, o = _recur(h[:m], q, k, s["v"][at].double(), g[at], b[at])
        h[:m] = new
        out[at] = o
    back = torch.empty_like(h)
    back[order] = h
    return dict(out=out, final=back)


def _exact_step(s):
    c, t = s["c"], {k: v.clone() for k, v in s["cache"].items()}
    r, L = c["hv"] // c["hk"], c["ring"]
    g, b = _gate64(s)
    live, lens, cu = s["live"].tolist(), s["lens"].tolist(), s["cu"].tolist()
    slots, ring = s["ids"].tolist(), t["ring_start"].tolist()
    gates = t["gate_cache"].double()
    k_cache, v_cache = t["k_cache"].double(), t["v_cache"].double()
    for j, slot in enumerate(slots):
        for i in range(lens[j]):
            at, row = (ring[slot] + live[j] + i) % L, cu[j] + i
            k_cache[slot, :, at], v_cache[slot, :, at] = s["k"][row].double(), s["v"][row].double()
            gates[slot, :, at, 0], gates[slot, :, at, 1] = g[row], b[row]
    h = _untile(t["state"][s["ids"].long()].view(-1, c["hv"], c["dv"] * c["dk"]), c["dv"], c["dk"]).double()
    out = torch.empty(s["rows"], c["hv"], c["dv"], dtype=torch.float64, device=DEV)
    for i in range(c["live"] + c["T"]):
        on = [j for j in range(len(slots)) if i < live[j] + lens[j]]
        if not on:
            break
        sl, at = [slots[j] for j in on], [(ring[slots[j]] + i) % L for j in on]
        sl, at = torch.tensor(sl, device=DEV), torch.tensor(at, device=DEV)
        row = torch.tensor([max(0, cu[j] + i - live[j]) for j in on], device=DEV)
        q = _unit64(s["q"][row], c["dk"] ** -0.5).repeat_interleave(r, dim=1)
        k = _unit64(k_cache[sl, :, at]).repeat_interleave(r, dim=1)
        h[on], o = _recur(h[on], q, k, v_cache[sl, :, at], gates[sl, :, at, 0], gates[sl, :, at, 1])
        new = torch.tensor([i >= live[j] for j in on], device=DEV)
        out[row[new]] = o[new]
    return dict(out=out, k_cache=k_cache, v_cache=v_cache, gate_cache=gates)


def _exact_flush(s):
    c, t = s["c"], s["cache"]
    r, L = c["hv"] // c["hk"], c["ring"]
    slots, ring, fold = s["ids"].tolist(), t["ring_start"].tolist(), s["fold"].tolist()
    h = _untile(t["state"][s["ids"].long()].view(-1, c["hv"], c["dv"] * c["dk"]), c["dv"], c["dk"]).double()
    for i in range(c["fold"]):
        on = [j for j in range(len(slots)) if i < fold[j]]
        sl = torch.tensor([slots[j] for j in on], device=DEV)
        at = torch.tensor([(ring[slots[j]] + i) % L for j in on], device=DEV)
        gates = t["gate_cache"][sl, :, at].double()
        k = _unit64(t["k_cache"][sl, :, at]).repeat_interleave(r, dim=1)
        h[on], _ = _recur(h[on], None, k, t["v_cache"][sl, :, at].double(), gates[..., 0], gates[..., 1])
    # the order of the checkpoint, by the index of each value
    dv, dk, e = c["dv"], c["dk"], 16 // t["state"].element_size()
    p, n = torch.meshgrid(torch.arange(dv, device=DEV), torch.arange(dk, device=DEV), indexing="ij")
    lane, held = 16 * (n // 4 % 4) + p % 16, n // 16 * 4 + n % 4
    place = p // 16 * 16 * dk + (held // e * 64 + lane) * e + held % e
    flat = torch.empty(len(slots), c["hv"], dv * dk, dtype=torch.float64, device=DEV)
    flat[:, :, place.reshape(-1)] = h.reshape(len(slots), c["hv"], dv * dk)
    state = t["state"].double()
    state[s["ids"].long()] = flat.view(len(slots), -1)
    starts = t["ring_start"].clone()
    for j, slot in enumerate(slots):
        starts[slot] = (ring[slot] + fold[j]) % L
    return dict(state=state, ring_start=starts)


def _exact_verify(s):
    c = s["c"]
    b, T, V = c["batch"], c["T"], c["vocab"]
    tokens, accepted, live, fold = [], [], [], []
    fed, u = s["tokens"].tolist(), s["u"].tolist()
    for j in range(b):
        n = 0
        while n < T - 1:
            row, d = j * T + n, fed[j * T + n + 1]
            chance = 1.0 if s["draft"] is None else float(s["draft"][row, d])
            if not u[row] * chance < float(s["target"][row, d]):
                break
            n += 1
        row = j * T + n
        r = s["target"][row].double()
        if n < T - 1:
            less = torch.zeros_like(r)
            if s["draft"] is None:
                less[fed[row + 1]] = 1.0
            else:
                less = s["draft"][row].double()
            # the difference is rounded to 32 bits, as the definition says
            r = torch.clamp(r - less, min=0).float().double()
        sums = torch.cumsum(r, 0)
        drawn = int((sums <= float(s["u_final"][j]) * sums[-1]).sum())
        tokens.append(fed[j * T + 1:j * T + 1 + n] + [drawn] + [-1] * (T - 1 - n))
        accepted.append(n + 1)
        live.append(int(s["live"][j]) - int(s["fold"][j]) + n + 1)
        fold.append(live[-1] if live[-1] + T > c["ring"] else 0)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(tokens=as_int(tokens), accepted=as_int(accepted), live=as_int(live), fold=as_int(fold))
