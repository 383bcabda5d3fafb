"""Cases and plain forms of the selective state update over prompts, of checkpoints read back, and of logits turned
into the probabilities that verification takes.

Four operators around the decode loop of speculative_replay_state_amd, each in its plain form (elementary torch
operations in 32 bits) and, with `own`, as calls of the package:

  prefill  the selective state update over whole prompts (varlen), from given or zero states to outputs and final states
  read     the checkpoints of cache slots, in any of their encodings, as fp32 states
  count    tokens of requests counted in their history pages (prompts, or what a verification accepted)
  logits   penalties by those counts and by the drafts before a row, biases, grammar masks, temperature and softmax

The rule of a prompt, per head with state h [64, 128], dt'_t = softplus(dt_t + dt_bias):

  h <- exp(A dt'_t) h + dt'_t x_t B_t^T;  y_t = h C_t + D x_t  (times z_t sigmoid(z_t) where there is a gate).

A history page holds a word 2 n + p for each value of the vocabulary (n times generated, p = 1 if in the prompt), valid
where the value's bit among the page's `seen` words is set.  A row of logits l becomes

  x = l + bias;  seen: x = x / r if x > 0 else x r;  x -= f n + c [n > 0];  masked: none;  p = softmax(x / temperature)

with the tokens fed before the row's, from the entry's second one on, counted too; temperature 0 is 1 at the largest x.
"""
import math

import torch

own = False

DEV = "cuda"
PAD = 1  # slot 0 of a cache and of a history is the padding slot
P, N = 64, 128  # values of a head, of its state's rows


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a few short prompts arriving together: launch and latency
        dict(name="prefill_short", op="prefill", seqs=4, max_len=48, heads=16, groups=2, init=False, gate=False, out="bf16"),
        # a ragged batch of prompts, one group of B and C, fp32 outputs
        dict(name="prefill_ragged", op="prefill", seqs=16, max_len=701, heads=32, groups=1, init=False, gate=False, out="f32"),
        # one long document continued from a state, gated: few chains, each of them long
        dict(name="prefill_long", op="prefill", seqs=1, max_len=16384, heads=64, groups=8, init=True, gate=True, out="bf16"),
        # a full batch of prompts of a layer with 128 heads
        dict(name="prefill_batch", op="prefill", seqs=8, max_len=4096, heads=128, groups=8, init=False, gate=False, out="bf16"),
        # one request's checkpoint taken out of the cache
        dict(name="read_one", op="read", batch=1, heads=16, state="bf16", recur=False),
        # a batch of fp8 checkpoints read back to continue their prompts
        dict(name="read_batch", op="read", batch=64, heads=128, state="fp8", recur=False),
        # what a verification accepted of a decode batch
        dict(name="count_step", op="count", batch=256, T=8, vocab=131072, prompt=False),
        # prompts of new requests counted in cleared pages
        dict(name="count_prompts", op="count", batch=32, T=4096, vocab=100003, prompt=True),
        # one request, one token: the latency of a row
        dict(name="logits_one", op="logits", batch=1, T=1, varlen=False, vocab=32000, logits="f32", out="f32", penalty=True,
             bias=0, mask=False, softmax=True),
        # a batch in plain decode whose sampler is the caller's own: logits in, logits out
        dict(name="logits_plain", op="logits", batch=64, T=1, varlen=False, vocab=65537, logits="bf16", out="f32", penalty=True,
             bias=300, mask=True, softmax=False),
        # a decode batch with three drafts a request, an odd vocabulary
        dict(name="logits_batch", op="logits", batch=64, T=4, varlen=False, vocab=100003, logits="f32", out="f32", penalty=True,
             bias=20, mask=True, softmax=True),
        # a large ragged decode batch, 16-bit values in and out
        dict(name="logits_large", op="logits", batch=256, T=8, varlen=True, vocab=131072, logits="bf16", out="bf16",
             penalty=True, bias=8, mask=True, softmax=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "read", "count", "logits", "logits", "logits"])
    if op == "prefill":
        seqs, groups = _log(rng, 1, 32), rng.choice([1, 1, 2, 4, 8])
        heads = groups * rng.choice([1, 2, 3, 5, 8, 12, 16])
        # at most the tokens x heads of the largest listed case, and no longer a chain than its longest
        max_len = _log(rng, 1, max(2, min(16000, 2500000 // (seqs * heads))))
        return dict(op=op, seqs=seqs, max_len=max_len, heads=heads, groups=groups, init=rng.random() < 0.5,
                    gate=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "read":
        state = rng.choice(["f32", "bf16", "f16", "fp8", "nvfp4"])
        heads = rng.choice([1, 3, 8, 16, 24, 64, 128])
        return dict(op=op, batch=_log(rng, 1, 8000 // heads), heads=heads, state=state,
                    recur=state in ("fp8", "nvfp4") and rng.random() < 0.4)
    if op == "count":
        prompt = rng.random() < 0.5
        return dict(op=op, batch=_log(rng, 1, 200), T=_log(rng, 1, 3000) if prompt else rng.randint(1, 8),
                    vocab=_log(rng, 200, 130001), prompt=prompt)
    b, T, vocab = _log(rng, 1, 200), rng.randint(1, 8), _log(rng, 200, 130001)
    soft = rng.random() < 0.75
    return dict(op=op, batch=b, T=T, varlen=rng.random() < 0.5, vocab=vocab, logits=rng.choice(["f32", "bf16", "f16"]),
                out=rng.choice(["f32", "bf16", "f16"]) if soft else "f32", penalty=rng.random() < 0.8,
                bias=rng.choice([0, 0, 7, 150]), mask=rng.random() < 0.5, softmax=soft)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_PAGE = {"f32": P * N * 4, "bf16": P * N * 2, "f16": P * N * 2, "fp8": P * N, "nvfp4": P * N // 2}  # bytes of a head


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


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV)


def _cu(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), lens.cumsum(0)]).to(torch.int32)


def _slots(g, batch):
    """Distinct slots in no order; a quarter of the cache is other requests'."""
    n = PAD + batch + (batch + 3) // 4
    ids = PAD + torch.randperm(n - PAD, generator=g, device=DEV)[:batch]
    return n, ids.to(torch.int32)


def _words(bits):
    """[..., vocab] truth values -> [..., ceil(vocab / 32)] words, value i in bit i % 32 of word i / 32."""
    pad = -bits.shape[-1] % 32
    w = torch.nn.functional.pad(bits, (0, pad)).unflatten(-1, (-1, 32))
    out = torch.zeros(w.shape[:-1], dtype=torch.int32, device=DEV)
    for i in range(32):
        out |= w[..., i].to(torch.int32) << i
    return out


def _history(g, slots, vocab, most=600):
    """Pages of requests under way: words of counted values, and what an earlier request left in the others."""
    counts = _randint(g, 0, 9, slots, vocab).to(torch.int32)
    seen = torch.zeros(slots, vocab, dtype=torch.bool, device=DEV)
    seen.scatter_(1, _randint(g, 0, vocab, slots, min(most, vocab)), True)
    counts = torch.where(seen, counts.clamp(min=1), counts)
    return counts, _words(seen)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, op = dict(case), case["op"]
    s = dict(c=c)
    if op == "prefill":
        H, G = c["heads"], c["groups"]
        lens = _lengths(g, c["seqs"], c["max_len"])
        s["lens"] = lens.tolist()
        s["rows"] = rows = sum(s["lens"])
        s["cu"] = _cu(lens)
        # x, B and C as a convolution leaves them, and the gate as a projection does: slices of one tensor's rows
        xbc = torch.nn.functional.silu(_randn(g, rows, H * P + 2 * G * N)).to(torch.bfloat16)
        s["x"] = xbc[:, :H * P].view(rows, H, P)
        s["B"] = xbc[:, H * P:H * P + G * N].view(rows, G, N)
        s["C"] = xbc[:, H * P + G * N:].view(rows, G, N)
        s["z"] = _randn(g, rows, 2 * H * P).to(torch.bfloat16)[:, :H * P].view(rows, H, P) if c["gate"] else None
        s["dt"] = 0.5 * _randn(g, rows, H)
        s["A"] = -torch.exp(_uniform(g, 0.0, math.log(16.0), H))
        s["D"], s["dt_bias"] = _uniform(g, 0.5, 1.5, H), _uniform(g, -4.0, -2.0, H)
        s["initial"] = 0.1 * _randn(g, c["seqs"], H, P, N) if c["init"] else None
        s["out"] = torch.zeros(rows, H, P, dtype=_TYPES[c["out"]], device=DEV)
        s["final"] = torch.zeros(c["seqs"], H, P, N, device=DEV)
    elif op == "read":
        H, st = c["heads"], c["state"]
        n, s["ids"] = _slots(g, c["batch"])
        if st in _TYPES:
            s["state"] = (0.1 * _randn(g, n, H * P * N)).to(_TYPES[st]).view(torch.uint8)
        else:
            s["state"] = _randint(g, 0, 256, n, H * _PAGE[st]).to(torch.uint8)
            if st == "fp8":  # no code is NaN
                s["state"] = torch.where((s["state"] & 127) == 127, s["state"] - 1, s["state"])
        s["scale"] = s["gscale"] = s["recur"] = None
        if st == "fp8":
            s["scale"] = _uniform(g, 1e-4, 1e-2, n, H * P).view(torch.uint8)
        if st == "nvfp4":
            s["scale"] = _randint(g, 0, 127, n, H * P * N // 16).to(torch.uint8)
            words = torch.zeros(n, (1 + H + 3) // 4 * 4, device=DEV)
            words[:, 0] = _uniform(g, 1e-5, 1e-4, n)
            s["gscale"] = words.view(torch.uint8)
        if c["recur"] or st == "nvfp4":
            s["recur"] = (0.1 * _randn(g, n, H * P * N)).half().view(torch.uint8)
        s["states"] = torch.zeros(c["batch"], H, P, N, device=DEV)
    elif op == "count":
        b, T, V = c["batch"], c["T"], c["vocab"]
        n, s["ids"] = _slots(g, b)
        s["counts"], s["seen"] = _history(g, n, V)
        lens = _lengths(g, b, T)
        # a few of the values come again and again, as in a text
        if c["prompt"]:
            s["cu"], total = _cu(lens), int(lens.sum())
            s["tokens"] = (V * torch.rand(total, generator=g, device=DEV) ** 4).to(torch.int32)
        else:
            s["num"] = lens.to(torch.int32)
            tokens = (V * torch.rand(b, T, generator=g, device=DEV) ** 4).to(torch.int32)
            s["tokens"] = torch.where(torch.arange(T, device=DEV)[None] < lens[:, None], tokens, -1)
    else:
        b, T, V = c["batch"], c["T"], c["vocab"]
        lens = _lengths(g, b, T) if c["varlen"] else torch.full((b,), T, device=DEV)
        s["lens"], s["cu"], s["rows"] = lens, _cu(lens), int(lens.sum())
        rows = s["rows"]
        s["logits"] = (3.0 * _randn(g, rows, V)).to(_TYPES[c["logits"]])
        s["out"] = torch.zeros(rows, V, dtype=_TYPES[c["out"]], device=DEV)
        if c["penalty"]:
            n, s["ids"] = _slots(g, b)
            s["counts"], s["seen"] = _history(g, n, V)
            s["tokens"] = (V * torch.rand(rows, generator=g, device=DEV) ** 4).to(torch.int32)
            s["repetition"] = _uniform(g, 1.0, 1.3, b)
            s["frequency"], s["presence"] = _uniform(g, 0.0, 0.5, b), _uniform(g, -0.2, 0.8, b)
        # one request in eight is greedy
        s["temperature"] = torch.where(torch.arange(b, device=DEV) % 8 == 5, 0.0, _uniform(g, 0.5, 1.2, b))
        if c["bias"]:
            many = _randint(g, 0, c["bias"] + 1, b).clamp(max=V)
            s["bias_offsets"] = _cu(many)
            order = torch.rand(b, V, generator=g, device=DEV).topk(min(c["bias"], V), dim=1).indices  # distinct tokens
            mine = torch.arange(order.shape[1], device=DEV)[None] < many[:, None]
            s["bias_tokens"] = order[mine].to(torch.int32)
            s["bias_values"] = 4.0 * _randn(g, s["bias_tokens"].numel())
        if c["mask"]:  # a grammar leaves nearly everything, some of it, or a few values
            share = torch.tensor([0.99, 0.3, 0.002], device=DEV)[_randint(g, 0, 3, rows)]
            allowed = torch.rand(rows, V, generator=g, device=DEV) < share[:, None]
            allowed.scatter_(1, _randint(g, 0, V, rows, 2), True)
            s["mask"] = _words(allowed)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors and workspaces that a program keeps beside its tensors."""
    import speculative_replay_state_amd as ssu
    c, op = s["c"], s["c"]["op"]
    s["ssu"] = ssu
    page = lambda slots, nbytes: torch.zeros(slots, nbytes, dtype=torch.uint8, device=DEV)  # noqa: E731
    if op == "prefill":
        ws = torch.empty(max(ssu.prefill_workspace_size(s["rows"], c["seqs"], c["heads"]), 16), dtype=torch.uint8, device=DEV)
        s["call"] = ssu.make_prefill(s["cu"], s["x"], s["B"], s["C"], s["dt"], s["A"], s["D"], s["dt_bias"], s["out"], z=s["z"],
                                     initial_states=s["initial"], final_states=s["final"], workspace=ws)
    elif op == "read":
        n, H, L = s["state"].shape[0], c["heads"], 16
        s["cache"] = ssu.DeviceCache(n, H, 1, L, c["state"], s["state"], s["scale"], page(n, H * L * P * 2), page(n, L * N * 2),
                                     page(n, H * L * 4), torch.zeros(n, dtype=torch.int32, device=DEV), recur=s["recur"],
                                     gscale=s["gscale"])
    elif op == "count":
        s["history"] = ssu.TokenHistory(s["counts"].shape[0], c["vocab"], s["counts"], s["seen"])
        if c["prompt"]:
            s["call"] = ssu.make_count(s["history"], s["ids"], s["tokens"], cu_seqlens=s["cu"], prompt=True, reset=True)
        else:
            s["call"] = ssu.make_count(s["history"], s["ids"], s["tokens"], num_tokens=s["num"])
    else:
        ws = torch.empty(max(ssu.logits_workspace_size(c["batch"], c["T"], c["vocab"]), 16), dtype=torch.uint8, device=DEV)
        more = {}
        if c["penalty"]:
            more.update(history=ssu.TokenHistory(s["counts"].shape[0], c["vocab"], s["counts"], s["seen"]), slot_idx=s["ids"],
                        tokens=s["tokens"], repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"])
        if c["bias"]:
            more.update(bias_offsets=s["bias_offsets"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"])
        if c["mask"]:
            more.update(mask=s["mask"])
        s["call"] = ssu.make_logits(s["logits"], s["out"], c["batch"], c["T"], cu_seqlens=s["cu"] if c["varlen"] else None,
                                    temperature=s["temperature"], softmax=c["softmax"], workspace=ws, **more)


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------

def run(state):
    s, op = state, state["c"]["op"]
    if own:
        return _own(s, op)
    return dict(prefill=_plain_prefill, read=_plain_read, count=_plain_count, logits=_plain_logits)[op](s)


def _own(s, op):
    ssu = s["ssu"]
    if op == "prefill":
        ssu.prefill(s["call"])
        return dict(out=s["out"], final=s["final"])
    if op == "read":
        ssu.read_state(s["cache"], s["states"], s["ids"], recur=s["c"]["recur"])
        return dict(states=s["states"])
    if op == "count":
        ssu.count(s["call"])
        return dict(counts=s["counts"], seen=s["seen"])
    ssu.logits(s["call"])
    return dict(out=s["out"])


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _plain_prefill(s):
    c, C = s["c"], 64
    n, H, G = c["seqs"], c["heads"], c["groups"]
    nc = -(-c["max_len"] // C)
    at = s["cu"][:-1, None] + torch.arange(nc * C, device=DEV)[None]
    there = at < s["cu"][1:, None]
    at = torch.where(there, at, 0).long()

    def chunks(x):  # [rows, h, d] -> [n, h, nc, C, d]
        return x[at].transpose(1, 2).reshape(n, x.shape[1], nc, C, x.shape[2])

    def wide(x):  # groups -> heads
        return x.repeat_interleave(H // G, dim=1)

    here = there.view(n, 1, nc, C)
    dt = torch.where(here, chunks(_softplus(s["dt"] + s["dt_bias"])[..., None])[..., 0], 0.0)
    decays = (s["A"].view(1, H, 1, 1) * dt).double().cumsum(-1)
    x, B, Cm = chunks(s["x"].float()), chunks(s["B"].float()), chunks(s["C"].float())
    low = torch.ones(C, C, dtype=torch.bool, device=DEV).tril()
    W = wide(Cm @ B.transpose(-1, -2)) * dt[..., None, :]
    W *= torch.where(low, torch.exp(torch.where(low, decays[..., :, None] - decays[..., None, :], 0.0).float()), 0.0)
    y = W @ x
    x = x * (torch.exp(decays[..., -1:] - decays).float() * dt)[..., None]
    last = torch.exp(decays[..., -1]).float()[..., None, None]
    h = s["initial"].clone() if s["initial"] is not None else torch.zeros(n, H, P, N, device=DEV)
    e = torch.exp(decays).float()[..., None]
    for i in range(nc):
        y[:, :, i] += e[:, :, i] * (wide(Cm[:, :, i]) @ h.transpose(-1, -2))
        h = last[:, :, i] * h + x[:, :, i].transpose(-1, -2) @ wide(B[:, :, i])
    y = y.reshape(n, H, nc * C, P).transpose(1, 2)[there] + s["D"].view(1, H, 1) * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    s["out"].copy_(y)
    s["final"].copy_(h)
    return dict(out=s["out"], final=s["final"])


def _untile(x):
    """[..., 64 * 128] values in a checkpoint's order -> [..., 64, 128]: rows in blocks of 16, lane 16 q + m of a block
    holds values 32 q .. of row m, in 16-byte chunks, chunk u of all lanes side by side."""
    e = 16 // x.element_size()
    y = x.unflatten(-1, (4, 32 // e, 4, 16, e))          # block, u, q, m, i
    return y.movedim(-2, -4).movedim(-2, -3).reshape(*x.shape[:-1], P, N)  # block, m, q, u, i


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_read(s):
    c, slot = s["c"], s["ids"].long()
    b, H, st = c["batch"], c["heads"], "f16" if c["recur"] else c["state"]
    page = (s["recur"] if c["recur"] else s["state"])[slot]
    if st in _TYPES:
        h = _untile(page.view(_TYPES[st]).view(b, H, P * N)).float()
    elif st == "fp8":
        h = _untile(page.view(b, H, P * N)).view(torch.float8_e4m3fn).float()
        h = h * s["scale"][slot].view(torch.float32).view(b, H, P, 1)
    else:
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=DEV)
        code = torch.stack([page & 15, page >> 4], dim=-1)                     # value t in byte t / 2, even t below
        h = table[code.long()].view(b, H, 4, 4, 16, 32).transpose(3, 4)        # block, q, m, t -> block, m, q, t
        sf = s["scale"][slot].view(torch.float8_e4m3fn).float().view(b, H, 4, 16, 4, 2)  # q, m, block, half
        sf = sf.permute(0, 1, 4, 3, 2, 5).repeat_interleave(16, dim=-1)        # block, m, q, t
        h = (h * sf).reshape(b, H, P, N) * s["gscale"][slot].view(torch.float32)[:, :1, None, None]
    s["states"].copy_(h)
    return dict(states=s["states"])


def _plain_count(s):
    c, V = s["c"], s["c"]["vocab"]
    if c["prompt"]:
        entry = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), s["cu"].diff().long())
        token = s["tokens"].long()
        s["seen"][s["ids"].long()] = 0
    else:
        mine = torch.arange(c["T"], device=DEV)[None] < s["num"][:, None]
        entry = torch.arange(c["batch"], device=DEV)[:, None].expand(-1, c["T"])[mine]
        token = s["tokens"][mine].long()
    key, times = torch.unique(s["ids"].long()[entry] * V + token, return_counts=True)
    slot, token = key // V, key % V
    words, bit = s["seen"].shape[1], token % 32
    word = slot * words + token // 32
    was = (s["seen"].view(-1)[word] >> bit.to(torch.int32)) & 1
    old = torch.where(was == 1, s["counts"].view(-1)[key], 0)
    s["counts"].view(-1)[key] = (old | 1) if c["prompt"] else old + 2 * times.to(torch.int32)
    new = torch.zeros(s["seen"].numel(), dtype=torch.int64, device=DEV)
    new.scatter_add_(0, word, torch.where(was == 1, 0, 1 << bit))
    new = torch.where(new >= 2 ** 31, new - 2 ** 32, new).to(torch.int32)
    s["seen"] |= new.view_as(s["seen"])
    return dict(counts=s["counts"], seen=s["seen"])


def _bits(words, vocab):
    return ((words[..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).flatten(-2)[..., :vocab].bool()


def _plain_logits(s):
    c, V, rows = s["c"], s["c"]["vocab"], s["rows"]
    entry = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), s["lens"])
    x = s["logits"].float()
    if c["bias"]:
        bias = torch.zeros(c["batch"], V, device=DEV)
        of = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), s["bias_offsets"].diff().long())
        bias[of, s["bias_tokens"].long()] = s["bias_values"]
        x = x + bias[entry]
    if c["penalty"]:
        slot = s["ids"].long()[entry]
        seen = _bits(s["seen"], V)[slot]
        n = torch.where(seen, s["counts"][slot] >> 1, 0)
        # the tokens fed before a row's own end, from the entry's second one on
        first = s["cu"].long()[entry]
        t = torch.arange(rows, device=DEV) - first
        j = torch.arange(1, c["T"] + 1, device=DEV)[None]
        fed = j <= t[:, None]
        token = s["tokens"].long()[torch.where(fed, first[:, None] + j, 0)]
        at = (torch.arange(rows, device=DEV)[:, None] * V + token)[fed]
        n.view(-1).index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
        seen.view(-1)[at] = True
        r = s["repetition"][entry][:, None]
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - (s["frequency"][entry][:, None] * n + torch.where(n > 0, s["presence"][entry][:, None], 0.0))
    if c["mask"]:
        x = torch.where(_bits(s["mask"], V), x, -math.inf)
    temperature = s["temperature"][entry][:, None]
    greedy = temperature <= 0
    if not c["softmax"]:
        s["out"].copy_(torch.where(greedy, x, x / torch.where(greedy, 1.0, temperature)))
        return dict(out=s["out"])
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(greedy, 1.0, temperature))
    p = e / e.sum(-1, keepdim=True)
    i = torch.arange(V, device=DEV)
    best = torch.where(x == top, i, V).amin(-1, keepdim=True)
    s["out"].copy_(torch.where(greedy, (i == best).float(), p))
    return dict(out=s["out"])


# ---------------------------------------------------------------------------
# what a pass needs
# ---------------------------------------------------------------------------

def _mean(c, n, most):
    """Mean of the lengths."""
    lo = (most + 1) // 2
    return sum(most - (most - lo) * i // max(1, n - 1) for i in range(n)) / n


def work(case):
    c, op = case, case["op"]
    if op == "prefill":
        H, G = c["heads"], c["groups"]
        rows = c["seqs"] * _mean(c, c["seqs"], c["max_len"])
        row = H * P * (2 + (2 if c["gate"] else 0) + (4 if c["out"] == "f32" else 2)) + H * 4 + 2 * G * N * 2
        states = c["seqs"] * H * P * N * 4
        return dict(bytes=rows * row + states * (2 if c["init"] else 1), flops=rows * H * (4 * P * N + 4 * P))
    if op == "read":
        st = "f16" if c["recur"] else c["state"]
        scales = {"fp8": P * 4, "nvfp4": P * N // 16}.get(st, 0)
        heads = c["batch"] * c["heads"]
        return dict(bytes=heads * (_PAGE[st] + scales + P * N * 4), flops=heads * P * N)
    if op == "count":
        tokens, words = c["batch"] * _mean(c, c["batch"], c["T"]), (c["vocab"] + 31) // 32
        # each token, its bit and its word; a cleared page's bits
        return dict(bytes=tokens * 20 + (c["batch"] * words * 4 if c["prompt"] else 0), flops=tokens)
    rows = c["batch"] * (_mean(c, c["batch"], c["T"]) if c["varlen"] else c["T"])
    size = {"f32": 4, "bf16": 2, "f16": 2}
    bits = c["vocab"] / 8
    return dict(bytes=rows * (c["vocab"] * (size[c["logits"]] + size[c["out"]]) + (bits if c["mask"] else 0)) +
                (c["batch"] * bits if c["penalty"] else 0) + c["batch"] * c["bias"] * 4, flops=rows * c["vocab"] * 5)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return dict(prefill=_exact_prefill, read=_exact_read, count=_exact_count, logits=_exact_logits)[case["op"]](s)


def _exact_prefill(s):
    """Token by token."""
    c, H = s["c"], s["c"]["heads"]
    r = H // c["groups"]
    if c["max_len"] * (1e-4 + c["seqs"] * H * P * N * 80 / 3e12) > 15:
        return None
    order = sorted(range(c["seqs"]), key=lambda i: -s["lens"][i])  # longest first: the first m are still running
    cu = s["cu"].tolist()
    v = s["dt"].double() + s["dt_bias"].double()
    dt = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    g = torch.exp(s["A"].double() * dt)
    start = torch.tensor([cu[i] for i in order], device=DEV)
    h = torch.zeros(c["seqs"], H, P, N, dtype=torch.float64, device=DEV)
    if s["initial"] is not None:
        h += s["initial"].double()[order]
    out = torch.empty(s["rows"], H, P, dtype=torch.float64, device=DEV)
    for t in range(c["max_len"]):
        m = sum(1 for i in order if s["lens"][i] > t)
        at = start[:m] + t
        x = s["x"][at].double()
        B, C = (s[k][at].double().repeat_interleave(r, dim=1) for k in "BC")
        h[:m] *= g[at][..., None, None]
        h[:m] += (dt[at][..., None] * x)[..., None] * B[:, :, None]
        out[at] = (h[:m] * C[:, :, None]).sum(-1) + s["D"].double()[:, None] * x
    if s["z"] is not None:
        z = s["z"].double()
        out *= z * torch.sigmoid(z)
    back = torch.empty_like(h)
    back[order] = h
    return dict(out=out, final=back)


def _exact_read(s):
    """Each value by the place that the layout gives it."""
    c, H, slot = s["c"], s["c"]["heads"], s["ids"].long()
    st = "f16" if c["recur"] else c["state"]
    p, n = torch.meshgrid(torch.arange(P, device=DEV), torch.arange(N, device=DEV), indexing="ij")
    lane, t = 16 * (n // 32) + p % 16, n % 32
    head = torch.arange(H, device=DEV)[:, None, None]
    page = (s["recur"] if c["recur"] else s["state"])[slot]
    if st == "nvfp4":
        byte = page[:, head * 4096 + p // 16 * 1024 + lane * 16 + t // 2].long()
        code = torch.where(t % 2 == 0, byte % 16, byte // 16)
        value = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)[code % 8] * torch.where(code >= 8, -1.0, 1.0)
        sf = s["scale"][slot][:, head * 512 + lane * 8 + p // 16 * 2 + t // 16].long()
        e, m = sf // 8 % 16, (sf % 8).double()
        scale = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.double() - 10))
        return dict(states=value * scale * s["gscale"][slot].view(torch.float32)[:, 0].double()[:, None, None, None])
    eb = _PAGE[st] // (P * N)
    value = p // 16 * 2048 + (t // (16 // eb) * 64 + lane) * (16 // eb) + t % (16 // eb)
    value = head * (P * N) + value
    if st != "fp8":
        return dict(states=page.view(_TYPES[st])[:, value].double())
    code = page[:, value].long()
    e, m = code // 8 % 16, (code % 8).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.double() - 10)) * torch.where(code >= 128, -1.0, 1.0)
    return dict(states=v * s["scale"][slot].view(torch.float32).double()[:, head * P + p])


def _exact_count(s):
    c = s["c"]
    slots = s["ids"].tolist()
    if c["prompt"]:
        cu, tokens = s["cu"].tolist(), s["tokens"].tolist()
        fed = [tokens[cu[j]:cu[j + 1]] for j in range(c["batch"])]
    else:
        fed = [row[:n] for row, n in zip(s["tokens"].tolist(), s["num"].tolist())]
    counts, seen = s["counts"].cpu().numpy().copy(), s["seen"].cpu().numpy().copy().view("uint32")
    for slot, row in zip(slots, fed):
        if c["prompt"]:
            seen[slot] = 0
        for token in row:
            w, bit = token // 32, 1 << (token % 32)
            if not int(seen[slot, w]) & bit:
                counts[slot, token] = 0
                seen[slot, w] = int(seen[slot, w]) | bit
            counts[slot, token] = counts[slot, token] | 1 if c["prompt"] else counts[slot, token] + 2
    return dict(counts=torch.from_numpy(counts).to(DEV), seen=torch.from_numpy(seen.view("int32")).to(DEV))


def _exact_logits(s):
    """Row by row."""
    c, V = s["c"], s["c"]["vocab"]
    cu, temperature = s["cu"].tolist(), s["temperature"].tolist()
    out = torch.empty(s["rows"], V, dtype=torch.float64, device=DEV)
    tokens = s["tokens"].tolist() if c["penalty"] else None
    i = torch.arange(V, device=DEV)
    for b in range(c["batch"]):
        if c["penalty"]:
            slot = int(s["ids"][b])
            bit = (s["seen"][slot].long()[i // 32] >> (i % 32)) & 1
            n0, seen0 = torch.where(bit == 1, s["counts"][slot].double().div(2).floor(), 0.0), bit == 1
            rep, freq, pres = (s[k][b].double() for k in ("repetition", "frequency", "presence"))
        for row in range(cu[b], cu[b + 1]):
            x = s["logits"][row].double()
            if c["bias"]:
                lo, hi = s["bias_offsets"][b], s["bias_offsets"][b + 1]
                x[s["bias_tokens"][lo:hi].long()] += s["bias_values"][lo:hi].double()
            if c["penalty"]:
                n, seen = n0.clone(), seen0.clone()
                for token in tokens[cu[b] + 1:row + 1]:
                    n[token] += 1
                    seen[token] = True
                x = torch.where(seen, x * torch.where(x > 0, 1 / rep, rep), x) - freq * n - pres * (n > 0)
            if c["mask"]:
                x[((s["mask"][row].long()[i // 32] >> (i % 32)) & 1) == 0] = -math.inf
            if not c["softmax"]:
                out[row] = x / temperature[b] if temperature[b] > 0 else x
            elif temperature[b] > 0:
                p = torch.exp((x - x.max()) / s["temperature"][b].double())
                out[row] = p / p.sum()
            else:
                out[row] = 0.0
                out[row, int((x == x.max()).nonzero()[0])] = 1.0
    return dict(out=out)
