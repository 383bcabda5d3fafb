"""The gated delta rule on the GPU (step, flush, init, read, prompts) against
the rule token by token in 64 bits (delta_refs), through the C ABI.

Tolerances are delta_refs.tol, derived there; copies (ring appends, untouched
slots, rows behind the last sequence, checkpoints a step must not change) are
compared bit for bit.
"""
import pytest
import torch

from tests import delta_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def up(x):
    return {k: v.to(DEV) for k, v in x.items()}


def call_step(dc, T, ids, pnat, cu, x, out, **kw):
    d = ssu.make_delta_step(dc, T, i32(ids), i32(pnat), None if cu is None else i32(cu), x["q"], x["k"], x["v"], x["dt"],
                            x["beta"], x["A"], x["dt_bias"], out, **kw)
    ssu.delta_replay_step(dc, d)
    return d


def check_step(c, before, got, out, x, ids, pnat, rows, out_name, scale, norm=True, softplus=True, sigmoid=True):
    """Outputs and every cache byte after a step; rows[b] = (first row, count)."""
    g, b = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"], softplus, sigmoid)
    hk, hv, L = c.hk, c.hv, c.L
    k_want, v_want, gate_want = (before[n].clone() for n in ("k_cache", "v_cache", "gate_cache"))
    for j, slot in enumerate(ids):
        first, n = rows[j]
        if slot <= 0 or slot >= c.slots:
            assert bool((out[first:first + n] == 0).all()), "padding entry %d" % j
            continue
        k, v, gr, br = c.ring(slot, 0, pnat[j])
        at = slice(first, first + n)
        S, _ = R.run(c.states(slot), None, k, v, gr, br, scale, norm)
        _, o = R.run(S, x["q"][at], x["k"][at], x["v"][at], g[at], b[at], scale, norm)
        # what went in, through a unit query: the checkpoint and the window's values
        went = scale * (c.states(slot).double().flatten(1).norm(dim=1) +
                        torch.cat([v, x["v"][at]]).double().transpose(0, 1).flatten(1).norm(dim=1))
        if not norm:
            went = went * x["q"][at].double().norm(dim=-1).max() if n else went
        R.check(out[at].transpose(0, 1), o.transpose(0, 1), went, R.tol(c.dk, pnat[j] + n, 1, out_name, c.state_dtype), "entry %d" % j)
        pos = (int(c.ring_start[slot]) + pnat[j] + torch.arange(n)) % L
        k_want[slot].view(hk, L, c.dk)[:, pos] = x["k"][at].transpose(0, 1)
        v_want[slot].view(hv, L, c.dv)[:, pos] = x["v"][at].transpose(0, 1)
        new = torch.stack([g[at], b[at]], -1).transpose(0, 1)
        # softplus, sigmoid and a product in fp32: 8 roundings at most
        have = got["gate_cache"][slot].view(hv, L, 2)[:, pos].double()
        assert float(((have - new).abs() - 8 * 2.0 ** -24 * new.abs()).max()) <= 1e-30 if n else True, "gates"
        gate_want[slot].view(hv, L, 2)[:, pos] = got["gate_cache"][slot].view(hv, L, 2)[:, pos]
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(got["state"], before["state"]), "a step changed a checkpoint"
    assert same(got["k_cache"], k_want) and same(got["v_cache"], v_want) and same(got["gate_cache"], gate_want)
    assert torch.equal(got["ring_start"], before["ring_start"])


# batch, T, live, hk, hv, dk, dv, L, state, out: every checkpoint and output type at both windows (rings to 16 and to 32)
# and both widths of k; heads alone, in groups and in odd groups; dim_v that fills a wave's rows, less and more
STEPS = [
    (1, 1, 0, 1, 1, 128, 128, 16, "bf16", "bf16"),
    (1, 1, 15, 1, 1, 128, 128, 16, "f32", "f32"),
    (5, 4, 4, 2, 4, 128, 128, 16, "bf16", "f32"),
    (5, 4, 4, 2, 6, 64, 64, 16, "bf16", "bf16"),
    (4, 3, 2, 1, 3, 128, 48, 5, "f16", "f32"),
    (4, 5, 11, 2, 2, 64, 16, 16, "f16", "bf16"),
    (3, 16, 0, 1, 8, 128, 256, 16, "f32", "f32"),
    (3, 16, 16, 2, 4, 128, 128, 32, "f32", "f32"),
    (3, 16, 16, 2, 2, 64, 80, 32, "bf16", "f32"),
    (3, 7, 16, 4, 4, 128, 64, 23, "f16", "bf16"),
    (3, 1, 16, 1, 5, 64, 128, 17, "f32", "bf16"),
    (2, 9, 7, 2, 2, 64, 208, 16, "f32", "f32"),
    (2, 2, 1, 1, 1, 64, 64, 3, "bf16", "f32"),
    (2, 12, 20, 1, 2, 128, 144, 32, "bf16", "bf16"),
]


@pytest.mark.parametrize("case", STEPS)
@pytest.mark.parametrize("varlen", [False, True])
def test_step(case, varlen):
    batch, T, live, hk, hv, dk, dv, L, state, out_name = case
    g = gen(STEPS.index(case) + 50 * varlen)
    c = R.Cache(g, batch + 4, hk, hv, dk, dv, L, state, pad=32 if varlen else 0)
    ids = (1 + torch.randperm(batch + 3, generator=g)[:batch]).tolist()
    if batch > 2:
        ids[1] = 0  # padding
    lens = torch.randint(0, T + 1, (batch,), generator=g).tolist() if varlen else [T] * batch
    lens[0] = T
    pnat = [int(torch.randint(0, live + 1, (1,), generator=g)) for _ in range(batch)]
    pnat[0] = live
    cu = [3 if varlen else 0]  # varlen: rows before and behind the sequences belong to nobody
    for n in lens:
        cu.append(cu[-1] + n)
    rows = cu[-1] + (5 if varlen else 0)
    x = R.inputs(g, rows, hk, hv, dk, dv, wide=8 if varlen else 0)
    if varlen:
        for name in ("q", "k", "v"):  # rows that no entry owns
            x[name][:3] = float("nan")
            x[name][cu[-1]:] = float("inf")
    # ring entries that are not live hold anything
    for slot, p in zip(ids, pnat):
        if slot > 0:
            dead = (int(c.ring_start[slot]) + p + torch.arange(L - p)) % L
            c.t["k_cache"][slot].view(hk, L, dk)[:, dead] = float("nan")
            c.t["v_cache"][slot].view(hv, L, dv)[:, dead] = float("inf")
            c.t["gate_cache"][slot].view(hv, L, 2)[:, dead] = float("nan")
    d, dc = c.upload(ssu, DEV)
    before = c.download(d)
    print("step", case, "varlen", varlen, flush=True)
    out = torch.full((rows, hv, dv), 7.0, dtype=R.TYPES[out_name], device=DEV)
    desc = call_step(dc, T, ids, pnat, cu if varlen else None, up(x), out)
    torch.cuda.synchronize()
    assert int(d["status"]) == 0
    got, o = c.download(d), out.cpu()
    check_step(c, before, got, o, x, ids, pnat, [(cu[j], lens[j]) for j in range(batch)], out_name, dk ** -0.5)
    if varlen:
        assert bool((o[:3] == 7).all()) and bool((o[cu[-1]:] == 7).all())
    # again: the same outputs and the same cache
    ssu.delta_replay_step(dc, desc)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), o)
    again = c.download(d)
    assert all(torch.equal(again[n].view(torch.uint8), got[n].view(torch.uint8)) for n in again)


@pytest.mark.parametrize("norm,softplus,sigmoid,scale", [(False, True, True, None), (True, False, False, 0.5), (False, False, False, 2.0)])
def test_step_flags(norm, softplus, sigmoid, scale):
    g = gen(5)
    c = R.Cache(g, 4, 2, 4, 64, 64, 16, "f32")
    c.t["k_cache"] *= 0.1  # not scaled by the kernel: as short as a model's would be
    x = R.inputs(g, 8, 2, 4, 64, 64)
    x["k"] *= 0.1
    if not softplus:
        x["dt"], x["dt_bias"] = x["dt"].abs() * 0.2, torch.full((4,), 0.01)
    if not sigmoid:
        x["beta"] = torch.rand(8, 4, generator=g)
    d, dc = c.upload(ssu, DEV, norm=norm)
    before = c.download(d)
    out = torch.empty(8, 4, 64, dtype=torch.float32, device=DEV)
    call_step(dc, 4, [3, 1], [5, 2], None, up(x), out, scale=scale, dt_softplus=softplus, beta_sigmoid=sigmoid)
    check_step(c, before, c.download(d), out.cpu(), x, [3, 1], [5, 2], [(0, 4), (4, 4)], "f32", 64 ** -0.5 if scale is None else scale,
               norm, softplus, sigmoid)


def test_step_bad_entries_are_skipped_and_named():
    g = gen(6)
    c = R.Cache(g, 8, 1, 2, 64, 64, 8, "bf16")
    c.ring_start[3], c.ring_start[4] = 8, -1
    x = R.inputs(g, 20, 1, 2, 64, 64)
    cases = [([1, 2], [6, -1], None, ssu.SSU_STATUS_BAD_PNAT), ([3, 4], [0, 0], None, ssu.SSU_STATUS_BAD_RING),
             ([5, 6], [0, 0], [4, 0, 5], ssu.SSU_STATUS_BAD_SEQLEN),
             ([5, 6], [0, 0], [2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1], ssu.SSU_STATUS_BAD_SEQLEN), ([5, 6], [0, 2 ** 31 - 1], None, ssu.SSU_STATUS_BAD_PNAT),
             ([-1, 8], [0, 0], None, 0), ([-2 ** 31, 2 ** 31 - 1], [9, 9], None, 0)]
    for ids, pnat, cu, bit in cases:
        d, dc = c.upload(ssu, DEV)
        before = c.download(d)
        out = torch.full((20, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        call_step(dc, 4, ids, pnat, cu, up(x), out)
        torch.cuda.synchronize()
        assert int(d["status"]) == bit, (ids, pnat, cu)
        after = c.download(d)
        # 5 has pnat 0 in the last case but two: a good entry beside a bad one
        others = [sl for sl in range(8) if not (sl == 5 and pnat == [0, 2 ** 31 - 1])]
        assert all(torch.equal(after[n][others].view(torch.uint8), before[n][others].view(torch.uint8)) for n in after)
        o = out.cpu()
        if bit == ssu.SSU_STATUS_BAD_SEQLEN:
            assert bool((o == 7).all())
        else:
            good = {0} if pnat == [0, 2 ** 31 - 1] else set()
            for j in range(2):
                assert (j in good) or bool((o[4 * j:4 * j + 4] == 0).all())
            assert bool((o[8:] == 7).all())


def test_step_bad_pnat_leaves_a_good_entry_alone():
    g = gen(7)
    c = R.Cache(g, 4, 1, 1, 64, 64, 8, "f32")
    x = R.inputs(g, 8, 1, 1, 64, 64)
    d, dc = c.upload(ssu, DEV)
    out = torch.empty(8, 1, 64, device=DEV)
    call_step(dc, 4, [2, 1], [5, 4], None, up(x), out)
    torch.cuda.synchronize()
    assert int(d["status"]) == ssu.SSU_STATUS_BAD_PNAT
    d2, dc2 = c.upload(ssu, DEV)
    out2 = torch.empty(8, 1, 64, device=DEV)
    call_step(dc2, 4, [0, 1], [0, 4], None, up(x), out2)
    assert torch.equal(out[4:], out2[4:]) and bool((out[:4] == 0).all())


def test_nan_stays_in_its_request_and_head():
    """(Within them it may reach the call's earlier tokens: their weights for it are zeros, and 0 x NaN is NaN.)"""
    g = gen(8)
    c = R.Cache(g, 4, 1, 2, 64, 64, 16, "bf16")
    x = R.inputs(g, 9, 1, 2, 64, 64)
    d, dc = c.upload(ssu, DEV)
    want = torch.empty(9, 2, 64, device=DEV)
    call_step(dc, 3, [1, 2, 3], [4, 4, 4], None, up(x), want)
    x["v"][4, 1, 5] = float("nan")   # entry 1, token 1, head 1
    x["dt"][8, 0] = float("inf")     # entry 2, token 2, head 0
    d, dc = c.upload(ssu, DEV)
    got = torch.empty(9, 2, 64, device=DEV)
    call_step(dc, 3, [1, 2, 3], [4, 4, 4], None, up(x), got)
    assert torch.equal(got[:3], want[:3]) and torch.equal(got[3:6, 0], want[3:6, 0])
    assert torch.equal(got[6:, 1], want[6:, 1])
    assert bool(torch.isnan(got[4, 1, 5])) and bool(torch.isnan(got[5, 1, 5]))


FLUSHES = [(1, 1, 1, 128, 128, 16, "f32", 1), (4, 2, 4, 128, 64, 16, "f32", 16), (4, 2, 4, 128, 128, 32, "f32", 32),
           (4, 1, 3, 64, 48, 16, "bf16", 9), (4, 2, 2, 64, 128, 32, "bf16", 30), (3, 1, 2, 128, 256, 5, "bf16", 5),
           (4, 2, 6, 64, 16, 16, "f16", 7), (4, 1, 1, 128, 144, 23, "f16", 20)]


@pytest.mark.parametrize("case", FLUSHES)
def test_flush(case):
    batch, hk, hv, dk, dv, L, state, most = case
    g = gen(FLUSHES.index(case))
    c = R.Cache(g, batch + 4, hk, hv, dk, dv, L, state, pad=16)
    ids = (1 + torch.randperm(batch + 3, generator=g)[:batch]).tolist()
    fold = [most] + [int(torch.randint(0, most + 1, (1,), generator=g)) for _ in range(batch - 1)]
    if batch > 3:
        fold[1], fold[2], ids[3] = 0, 1, 0
    for slot, k in zip(ids, fold):  # what is not folded may be anything
        dead = (int(c.ring_start[slot]) + k + torch.arange(L - k)) % L
        c.t["v_cache"][slot].view(hv, L, dv)[:, dead] = float("nan")
        c.t["k_cache"][slot].view(hk, L, dk)[:, dead] = float("nan")
        c.t["gate_cache"][slot].view(hv, L, 2)[:, dead] = float("inf")
    d, dc = c.upload(ssu, DEV)
    before = c.download(d)
    print("flush", case, fold, flush=True)
    ssu.delta_flush(dc, i32(ids), i32(fold))
    torch.cuda.synchronize()
    assert int(d["status"]) == 0
    got = c.download(d)
    want_start = before["ring_start"].clone()
    for slot, k in zip(ids, fold):
        if slot <= 0 or k == 0:
            continue
        want_start[slot] = (int(c.ring_start[slot]) + k) % L
        kr, v, gr, br = c.ring(slot, 0, k)
        S, _ = R.run(c.states(slot), None, kr, v, gr, br, 1.0)
        have = got["state"][slot].view(hv, -1)[:, c.place].view(hv, dv, dk)
        went = c.states(slot).double().flatten(1).norm(dim=1) + v.double().transpose(0, 1).flatten(1).norm(dim=1)
        R.check(have, S, went, R.tol(dk, k, 1, state), "slot %d" % slot)
        before["state"][slot] = got["state"][slot]
    assert torch.equal(got["ring_start"], want_start)
    assert all(torch.equal(got[n].view(torch.uint8), before[n].view(torch.uint8)) for n in ("state", "k_cache", "v_cache", "gate_cache"))


def test_flush_bad_entries():
    g = gen(9)
    c = R.Cache(g, 6, 1, 2, 64, 64, 8, "f32")
    c.ring_start[5] = 99
    d, dc = c.upload(ssu, DEV)
    before = c.download(d)
    for ids, fold, bit in (([1, 2], [9, -1], ssu.SSU_STATUS_BAD_FOLD), ([5, 0], [2, 2], ssu.SSU_STATUS_BAD_RING), ([-3, 6], [2, 2], 0)):
        d["status"].zero_()
        ssu.delta_flush(dc, i32(ids), i32(fold))
        torch.cuda.synchronize()
        assert int(d["status"]) == bit
        after = c.download(d)
        assert all(torch.equal(after[n].view(torch.uint8), before[n].view(torch.uint8)) for n in after)


@pytest.mark.parametrize("state,dk,dv,hk,hv", [("f32", 128, 128, 2, 4), ("bf16", 64, 48, 1, 3), ("f16", 128, 256, 1, 1)])
def test_init_and_read_state(state, dk, dv, hk, hv):
    g = gen(10)
    c = R.Cache(g, 6, hk, hv, dk, dv, 8, state, pad=48)
    d, dc = c.upload(ssu, DEV)
    before = c.download(d)
    states = torch.randn(4, hv, dv, dk, generator=g)
    ids = [4, 0, 2, 6]
    ssu.delta_init_state(dc, states.to(DEV), i32(ids))
    got = c.download(d)
    for j, slot in enumerate(ids):
        if not 0 < slot < 6:
            continue
        want = torch.empty(hv, dv * dk, dtype=R.TYPES[state])
        want[:, c.place] = states[j].to(R.TYPES[state]).view(hv, -1)
        assert torch.equal(got["state"][slot], want.view(-1))
        assert all(not bool(got[n][slot].any()) for n in ("k_cache", "v_cache", "gate_cache")) and int(got["ring_start"][slot]) == 0
        for n in got:
            before[n][slot] = got[n][slot]
    assert all(torch.equal(got[n].view(torch.uint8), before[n].view(torch.uint8)) for n in got)
    back = torch.full((4, hv, dv, dk), 7.0, device=DEV)
    ssu.delta_read_state(dc, back, i32(ids))
    for j, slot in enumerate(ids):
        want = states[j].to(R.TYPES[state]).float() if 0 < slot < 6 else torch.full((hv, dv, dk), 7.0)
        assert torch.equal(back[j].cpu(), want)
    # one state for several slots
    ssu.delta_init_state(dc, states[:1].to(DEV).expand(3, -1, -1, -1), i32([1, 3, 5]))
    ssu.delta_read_state(dc, back[:3], i32([1, 3, 5]))
    assert all(torch.equal(back[j].cpu(), states[0].to(R.TYPES[state]).float()) for j in range(3))


def call_prefill(x, cu, out, h0=None, h1=None, status=None, ws=None, **kw):
    rows, hv = x["q"].shape[0], x["v"].shape[1]
    if ws is None:
        ws = torch.empty(max(16, ssu.delta_prefill_workspace_size(rows, len(cu) - 1, hv)), dtype=torch.uint8, device=DEV)
    d = ssu.make_delta_prefill(i32(cu), x["q"], x["k"], x["v"], x["dt"], x["beta"], x["A"], x["dt_bias"], out,
                               initial_states=h0, final_states=h1, workspace=ws, status=status, **kw)
    ssu.delta_prefill(d)
    return d


PREFILLS = [([1], 1, 1, 128, 128, False), ([0, 1, 31, 0], 1, 2, 64, 64, True), ([32], 2, 4, 128, 64, False),
            ([33, 64, 2], 1, 3, 128, 48, True), ([100, 0, 7, 65], 2, 2, 64, 256, True), ([257], 1, 2, 128, 144, False),
            ([5, 300, 31, 32, 1], 2, 6, 64, 16, False), ([96, 95, 97], 4, 4, 128, 128, True)]


@pytest.mark.parametrize("lens,hk,hv,dk,dv,init", PREFILLS)
@pytest.mark.parametrize("out_name", ["bf16", "f32"])
def test_prefill(lens, hk, hv, dk, dv, init, out_name):
    g = gen(sum(lens) + dv)
    cu = [2]
    for n in lens:
        cu.append(cu[-1] + n)
    rows = cu[-1] + 9
    x = R.inputs(g, rows, hk, hv, dk, dv, wide=16)
    for name in ("q", "k", "v"):
        x[name][:2], x[name][cu[-1]:] = float("nan"), float("inf")
    h0 = 0.3 * torch.randn(len(lens), hv, dv, dk, generator=g) if init else None
    h1 = torch.full((len(lens), hv, dv, dk), 7.0, device=DEV)
    out = torch.full((rows, hv, dv), 7.0, dtype=R.TYPES[out_name], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    print("prefill", lens, hk, hv, dk, dv, out_name, flush=True)
    call_prefill(up(x), cu, out, None if h0 is None else h0.to(DEV), h1, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    o, gt = out.cpu(), R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"])
    assert bool((o[:2] == 7).all()) and bool((o[cu[-1]:] == 7).all())
    for s, n in enumerate(lens):
        at = slice(cu[s], cu[s] + n)
        S0 = h0[s] if init else torch.zeros(hv, dv, dk)
        S, want = R.run(S0, x["q"][at], x["k"][at], x["v"][at], gt[0][at], gt[1][at], dk ** -0.5)
        went = S0.double().flatten(1).norm(dim=1) + x["v"][at].double().transpose(0, 1).flatten(1).norm(dim=1)
        windows = max(1, -(-n // 32))
        R.check(o[at].transpose(0, 1), want.transpose(0, 1), went * dk ** -0.5, R.tol(dk, 32, windows, out_name), "outputs %d" % s)
        R.check(h1[s].cpu(), S, went, R.tol(dk, 32, windows, "f32"), "state %d" % s)
    # in place: the final states over the initial ones; without them; the same again
    if init:
        both, out2 = h0.to(DEV), torch.full_like(out, 7.0)
        call_prefill(up(x), cu, out2, both, both)
        assert torch.equal(both, h1) and torch.equal(out2, out)
    out3 = torch.full_like(out, 7.0)
    call_prefill(up(x), cu, out3, None if h0 is None else h0.to(DEV), None)
    assert torch.equal(out3, out)


# the chains (sequence, value head) that each scan kernel takes: up to 256 blocks of 16 columns one kernel, more another,
# over 256 chains of more than 64 columns a third
@pytest.mark.parametrize("out_name", ["bf16", "f32"])
@pytest.mark.parametrize("n,most,hk,hv,dk,dv,init", [(9, 70, 2, 4, 128, 128, True), (20, 90, 4, 8, 64, 64, True),
                                                     (20, 100, 2, 8, 128, 48, False), (40, 100, 4, 8, 128, 128, True),
                                                     (33, 66, 2, 8, 64, 144, False), (64, 40, 1, 4, 64, 256, True)])
def test_prefill_of_many_chains(n, most, hk, hv, dk, dv, init, out_name):
    g = gen(n + dv)
    lens = torch.randint(0, most + 1, (n,), generator=g).tolist()
    lens[:3] = [most, 0, 33]
    cu = [0]
    for k in lens:
        cu.append(cu[-1] + k)
    x = R.inputs(g, cu[-1] + 3, hk, hv, dk, dv)
    x["k"][cu[-1]:] = float("nan")
    h0 = 0.3 * torch.randn(n, hv, dv, dk, generator=g) if init else None
    h1 = torch.empty(n, hv, dv, dk, device=DEV)
    out = torch.full((cu[-1] + 3, hv, dv), 7.0, dtype=R.TYPES[out_name], device=DEV)
    print("chains", n * hv, dk, dv, flush=True)
    call_prefill(up(x), cu, out, None if h0 is None else h0.to(DEV), h1)
    o, gt, h1 = out.cpu(), R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"]), h1.cpu()
    assert bool((o[cu[-1]:] == 7).all())
    for s in list(range(4)) + [n // 2, n - 1]:
        at = slice(cu[s], cu[s + 1])
        S0 = h0[s] if init else torch.zeros(hv, dv, dk)
        S, want = R.run(S0, x["q"][at], x["k"][at], x["v"][at], gt[0][at], gt[1][at], dk ** -0.5)
        went = S0.double().flatten(1).norm(dim=1) + x["v"][at].double().transpose(0, 1).flatten(1).norm(dim=1)
        windows = max(1, -(-lens[s] // 32))
        R.check(o[at].transpose(0, 1), want.transpose(0, 1), went * dk ** -0.5, R.tol(dk, 32, windows, out_name), "outputs %d" % s)
        R.check(h1[s], S, went, R.tol(dk, 32, windows, "f32"), "state %d" % s)


def test_prefill_without_rows():
    """Empty sequences only: the final states are the initial ones."""
    x = up(R.inputs(gen(11), 0, 1, 2, 64, 64))
    h0 = torch.randn(3, 2, 64, 64, device=DEV)
    h1 = torch.empty_like(h0)
    call_prefill(x, [0, 0, 0, 0], torch.empty(0, 2, 64, device=DEV), h0, h1)
    assert torch.equal(h0, h1)
    call_prefill(x, [0, 0, 0, 0], torch.empty(0, 2, 64, device=DEV), None, h1)
    assert not bool(h1.any())


def test_prefill_bad_sequences_are_skipped_and_named():
    x = up(R.inputs(gen(12), 64, 1, 1, 64, 64))
    for cu, good in (([0, 40, 30, 64], (0, 2)), ([-5, 20, 64, 64], (1, 2)), ([0, 20, 64, 70], (0, 1))):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        h1 = torch.full((3, 1, 64, 64), 7.0, device=DEV)
        out = torch.full((64, 1, 64), 7.0, device=DEV)
        call_prefill(x, cu, out, None, h1, status)
        torch.cuda.synchronize()
        assert int(status) == ssu.SSU_STATUS_BAD_SEQLEN
        for s in range(3):
            assert bool((h1[s] == 7).all()) == (s not in good)


@pytest.mark.parametrize("n,dv", [(150, 16), (150, 80)])
def test_many_short_sequences_find_their_chunks(n, dv):
    """More sequences than lanes look at once, empty ones among them."""
    g = gen(13)
    lens = torch.randint(0, 40, (n,), generator=g)
    lens[::7] = 0
    cu = [0] + lens.cumsum(0).tolist()
    x = R.inputs(g, cu[-1], 1, 1, 64, dv)
    out = torch.empty(cu[-1], 1, dv, device=DEV)
    call_prefill(up(x), cu, out)
    gt = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"])
    for s in range(n):
        at = slice(cu[s], cu[s + 1])
        _, want = R.run(torch.zeros(1, dv, 64), x["q"][at], x["k"][at], x["v"][at], gt[0][at], gt[1][at], 0.125)
        R.check(out[at].cpu().transpose(0, 1), want.transpose(0, 1), 0.125 * float(x["v"][at].double().norm()),
                R.tol(64, 32, 2, "f32"), "sequence %d" % s)


def test_far_decays_do_not_overflow():
    """Gates of -60 a token (a state forgotten at once) and of 0 (kept)."""
    g = gen(14)
    x = R.inputs(g, 70, 1, 2, 64, 64)
    x["A"] = torch.tensor([-60.0, 0.0])
    x["dt"], x["dt_bias"] = torch.ones(70, 2), torch.zeros(2)
    out = torch.empty(70, 2, 64, device=DEV)
    h1 = torch.empty(1, 2, 64, 64, device=DEV)
    call_prefill(up(x), [0, 70], out, None, h1, dt_softplus=False)
    gt = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"], softplus=False)
    S, want = R.run(torch.zeros(2, 64, 64), x["q"], x["k"], x["v"], *gt, 0.125)
    went = x["v"].double().transpose(0, 1).flatten(1).norm(dim=1)
    R.check(out.cpu().transpose(0, 1), want.transpose(0, 1), 0.125 * went, R.tol(64, 32, 3, "f32"), "outputs")
    R.check(h1[0].cpu(), S, went, R.tol(64, 32, 3, "f32"), "state")


@pytest.mark.parametrize("big", [1e8, 1e30, float("inf")])
def test_a_token_that_forgets_everything(big):
    """One gate of -1e8 and less (past fp32's range too) among ordinary ones: the state before it is gone, the decays
    between the tokens behind it are as exact as without it."""
    g = gen(17)
    x = R.inputs(g, 70, 1, 2, 64, 64)
    x["A"] = torch.tensor([-1.0, -1e10])
    x["dt"], x["dt_bias"] = 0.1 * torch.rand(70, 2, generator=g), torch.zeros(2)
    x["dt"][:, 1] *= 1e-10
    for t in (3, 40):
        x["dt"][t] = big
    gt = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"], softplus=False)
    out = torch.empty(70, 2, 64, device=DEV)
    h1 = torch.empty(1, 2, 64, 64, device=DEV)
    call_prefill(up(x), [0, 70], out, None, h1, dt_softplus=False)
    S, want = R.run(torch.zeros(2, 64, 64), x["q"], x["k"], x["v"], *gt, 0.125)
    went = x["v"].double().transpose(0, 1).flatten(1).norm(dim=1)
    R.check(out.cpu().transpose(0, 1), want.transpose(0, 1), 0.125 * went, R.tol(64, 32, 3, "f32"), "outputs")
    R.check(h1[0].cpu(), S, went, R.tol(64, 32, 3, "f32"), "state")
    # the same tokens through a ring of 16 after 5 of them, and folded
    c = R.Cache(g, 2, 1, 2, 64, 64, 16, "f32")
    d, dc = c.upload(ssu, DEV)
    got = torch.empty(70, 2, 64, device=DEV)
    call_step(dc, 10, [1], [4], None, up(x), got, dt_softplus=False)
    k, v, gr, br = c.ring(1, 0, 4)
    S0, _ = R.run(c.states(1), None, k, v, gr, br, 0.125)
    S, want = R.run(S0, x["q"][:10], x["k"][:10], x["v"][:10], gt[0][:10], gt[1][:10], 0.125)
    went = c.states(1).double().flatten(1).norm(dim=1) + torch.cat([v, x["v"][:10]]).double().transpose(0, 1).flatten(1).norm(dim=1)
    R.check(got[:10].cpu().transpose(0, 1), want.transpose(0, 1), 0.125 * went, R.tol(64, 14, 1, "f32"), "step")
    ssu.delta_flush(dc, i32([1]), i32([14]))
    back = torch.empty(1, 2, 64, 64, device=DEV)
    ssu.delta_read_state(dc, back, i32([1]))
    R.check(back[0].cpu(), S, went, R.tol(64, 14, 1, "f32"), "folded")


def test_repeated_keys():
    """The same key in every token with b near 1, where A is all ones below the
    diagonal and its powers would grow."""
    g = gen(15)
    x = R.inputs(g, 64, 1, 1, 64, 64)
    x["k"][:] = x["k"][0]
    x["beta"][:] = 9.0
    x["A"][:] = -0.001
    out = torch.empty(64, 1, 64, device=DEV)
    h1 = torch.empty(1, 1, 64, 64, device=DEV)
    call_prefill(up(x), [0, 64], out, None, h1)
    gt = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"])
    S, want = R.run(torch.zeros(1, 64, 64), x["q"], x["k"], x["v"], *gt, 0.125)
    went = float(x["v"].double().norm())
    R.check(out.cpu().transpose(0, 1), want.transpose(0, 1), 0.125 * went, R.tol(64, 32, 2, "f32"), "outputs")
    R.check(h1[0].cpu(), S, went, R.tol(64, 32, 2, "f32"), "state")


def test_slots_past_4_gib():
    """A cache whose last slots lie past 2^32 bytes and 2^31 values."""
    g = gen(16)
    slots, hv = 4100, 16
    small = R.Cache(g, 3, 1, hv, 128, 128, 8, "f32")
    stride = hv * 128 * 128 * 4
    state = torch.zeros(slots, stride, dtype=torch.uint8, device=DEV)
    tail = {n: torch.zeros(slots, small.t[n][0].numel() * small.t[n].element_size(), dtype=torch.uint8, device=DEV) for n in ("k_cache", "v_cache", "gate_cache")}
    start = torch.zeros(slots, dtype=torch.int32, device=DEV)
    ids = [slots - 1, slots - 2]
    for j, slot in enumerate(ids):
        state[slot] = small.t["state"][j + 1].view(torch.uint8).to(DEV)
        for n in tail:
            tail[n][slot] = small.t[n][j + 1].view(torch.uint8).to(DEV)
        start[slot] = int(small.ring_start[j + 1])
    dc = ssu.DeltaCache(slots, 1, hv, 8, "f32", state, tail["k_cache"], tail["v_cache"], tail["gate_cache"], start)
    d, dc2 = small.upload(ssu, DEV)
    x = up(R.inputs(g, 4, 1, hv, 128, 128))
    a, b = torch.empty(4, hv, 128, device=DEV), torch.empty(4, hv, 128, device=DEV)
    call_step(dc, 2, ids, [3, 5], None, x, a)
    call_step(dc2, 2, [1, 2], [3, 5], None, x, b)
    assert torch.equal(a, b) and bool(a.any())
    ssu.delta_flush(dc, i32(ids), i32([4, 7]))
    ssu.delta_flush(dc2, i32([1, 2]), i32([4, 7]))
    torch.cuda.synchronize()
    for j, slot in enumerate(ids):
        assert torch.equal(state[slot], d["state"][j + 1])
    assert not bool(state[:8].any()) and not bool(state[slots - 10:slots - 2].any())


def test_prompt_rows_past_4_gib():
    """Sequences whose rows of v, out and the scratch lie past 2^32 bytes, bit for bit as at the front."""
    g = gen(18)
    rows, hk, hv = 140000, 2, 128
    x = up(R.inputs(g, 300, hk, hv, 64, 128))
    far = {n: torch.zeros(rows, *x[n].shape[1:], dtype=x[n].dtype, device=DEV) for n in ("q", "k", "v", "dt", "beta")}
    for n in far:
        far[n][-300:] = x[n]
    far["A"], far["dt_bias"] = x["A"], x["dt_bias"]
    out, want = torch.zeros(rows, hv, 128, dtype=torch.bfloat16, device=DEV), torch.empty(300, hv, 128, dtype=torch.bfloat16, device=DEV)
    h1, w1 = torch.empty(2, hv, 128, 64, device=DEV), torch.empty(2, hv, 128, 64, device=DEV)
    print("prompt rows past 4 GiB", flush=True)
    call_prefill(far, [rows - 300, rows - 100, rows], out, None, h1)
    call_prefill(x, [0, 200, 300], want, None, w1)
    assert torch.equal(out[-300:], want) and torch.equal(h1, w1) and not bool(out[:100].any())
