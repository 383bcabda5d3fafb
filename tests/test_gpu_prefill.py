"""ssu_prefill on the GPU against the rule token by token in 64 bits."""
import pytest
import torch

from tests import prompt_refs as R

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


def call(a, lens, out_name, init=None, gate=False, softplus=True, final=True, rows=None, in_place=False, status=None, stream=None):
    """One prefill of host inputs `a`; (out, final states) on the host."""
    H, n = a["x"].shape[1], len(lens)
    rows = a["x"].shape[0] if rows is None else rows
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
    d = {}
    for k, t in a.items():  # slices stay slices
        if k in ("x", "B", "C", "z") and t.dim() == 3 and t.shape[0] > 1 and t.stride(0) != t.shape[1] * t.shape[2]:
            wide = torch.full((t.shape[0], t.stride(0)), float("nan"), dtype=t.dtype, device=DEV)
            wide[:, :t.shape[1] * t.shape[2]] = t.flatten(1).to(DEV)
            d[k] = wide[:, :t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])
        else:
            d[k] = t.to(DEV)
    out = torch.full((rows, H, 64), -7.0, dtype=torch.float32 if out_name == "f32" else torch.bfloat16, device=DEV)
    h0 = init.to(DEV) if init is not None else None
    h1 = h0 if in_place else (torch.full((n, H, 64, 128), -7.0, device=DEV) if final else None)
    size = ssu.prefill_workspace_size(rows, n, H)
    ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    p = ssu.make_prefill(cu, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], out, z=d["z"] if gate else None,
                         initial_states=h0, final_states=h1, workspace=ws[:size] if size else None, dt_softplus=softplus, status=status)
    ssu.prefill(p, stream=stream)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xA5).all()), "written behind the workspace"
    return out.cpu(), None if h1 is None else h1.cpu()


def want(a, lens, init=None, gate=False, softplus=True):
    """out, final states and, for tolerances, the same of absolute values."""
    H = a["x"].shape[1]
    d, g = R.gates(a["dt"], a["A"], a["dt_bias"], softplus)
    outs, states = [[], []], [[], []]
    at = 0
    for s, n in enumerate(lens):
        r = slice(at, at + n)
        at += n
        for k, f in enumerate((lambda t: t, torch.abs)):
            S0 = f(init[s]) if init is not None else torch.zeros(H, 64, 128)
            S, y = R.run(S0, f(a["x"][r]), f(a["B"][r]), f(a["C"][r]), f(d[r]), g[r], f(a["D"]))
            if gate:
                y = R.gate(y, a["z"][r]) if k == 0 else y * R.gate(torch.ones_like(y), a["z"][r]).abs()
            outs[k].append(y)
            states[k].append(S)
    return torch.cat(outs[0]), torch.stack(states[0]), torch.cat(outs[1]), torch.stack(states[1])


def compare(a, lens, out_name, what="", **kw):
    init, gate = kw.get("init"), kw.get("gate", False)
    out, final = call(a, lens, out_name, **kw)
    y, S, y_abs, S_abs = want(a, lens, init, gate, kw.get("softplus", True))
    most = max(lens + [1])
    n = sum(lens)
    R.check(out[:n], y, y_abs, R.tol_out(most, out_name), what + " out")
    if final is not None:
        R.check(final, S, S_abs, (2.0 ** -24, R.tol_state(most)), what + " final")
    return out, final


# one token, odd lengths, chunk borders; groups of 1, 2, 3, 4, 5 and 8 heads
@pytest.mark.parametrize("lens", [[1], [2, 1, 15], [16, 17, 63], [64, 65, 0, 127], [128, 129], [0, 0, 33], [200]])
@pytest.mark.parametrize("H,G", [(1, 1), (4, 2), (6, 2), (4, 1), (5, 1), (16, 2)])
@pytest.mark.parametrize("out_name", ["bf16", "f32"])
def test_short_prompts(lens, H, G, out_name):
    g = gen(1000 * sum(lens) + 10 * H + G)
    a = R.inputs(g, sum(lens), H, G)
    init = 0.3 * torch.randn(len(lens), H, 64, 128, generator=g)
    compare(a, lens, out_name, init=init, gate=H != 4)
    compare(a, lens, out_name)


# cut into segments (512 tokens and more): borders of segments and of chunks inside them
@pytest.mark.parametrize("lens", [[1500], [512, 513, 511], [1024, 1, 1025, 0, 700], [577, 3, 1281]])
@pytest.mark.parametrize("H,G,out_name", [(2, 1, "f32"), (4, 1, "bf16"), (5, 1, "bf16"), (2, 2, "bf16")])
@pytest.mark.parametrize("decay", [True, False])
def test_long_prompts(lens, H, G, out_name, decay):
    g = gen(17 * sum(lens) + H)
    a = R.inputs(g, sum(lens), H, G, decay=decay)
    init = 0.3 * torch.randn(len(lens), H, 64, 128, generator=g)
    compare(a, lens, out_name, init=init, gate=True)
    compare(a, lens, out_name, init=init.clone(), in_place=True)  # final states over the initial ones
    compare(a, lens, out_name, final=False)


def test_pieces_of_a_prompt_continue_it():
    g = gen(5)
    a = R.inputs(g, 300, 4, 2)
    whole, S = call(a, [300], "f32")
    state = torch.zeros(1, 4, 64, 128)
    parts = []
    for lo, hi in ((0, 1), (1, 70), (70, 128), (128, 300)):
        cut = {k: (t[lo:hi] if t.dim() > 1 else t) for k, t in a.items()}
        out, state = call(cut, [hi - lo], "f32", init=state)
        parts.append(out)
    _, _, y_abs, S_abs = want(a, [300])
    R.check(torch.cat(parts), whole.double(), y_abs, (2.0 ** -23, 2 * R.tol_out(300, "f32")[1]), "pieces")
    R.check(state, S.double(), S_abs, (2.0 ** -23, 2 * R.tol_state(300)), "state")


def test_slices_of_wider_rows_and_rows_nobody_owns():
    g = gen(6)
    rows, lens = 150, [40, 0, 65]
    a = R.inputs(g, rows, 6, 2, wide=24)
    for k in ("x", "B", "C", "z", "dt"):  # behind the last sequence: nothing that may reach a result
        a[k][105:] = float("nan")
    out, _ = compare(a, lens, "bf16", gate=True)
    assert bool((out[105:] == -7).all()), "rows behind the last sequence written"


def test_dt_as_it_is_and_gates_far_below():
    g = gen(7)
    a = R.inputs(g, 130, 4, 1)
    a["dt"] = torch.rand(130, 4, generator=g) * 0.5 - a["dt_bias"]
    compare(a, [130], "f32", softplus=False)
    a["dt"][40] = 1e30   # everything before it is forgotten; what comes after is not
    a["A"][0] = -1e10
    a["x"][40] = 0
    out, final = call(a, [130], "f32", softplus=False)
    b = {k: (t[41:] if t.dim() > 1 else t) for k, t in a.items()}
    y, S, y_abs, S_abs = want(b, [89], softplus=False)
    R.check(out[41:], y, y_abs, R.tol_out(130, "f32"), "after a gate far below")
    R.check(final, S, S_abs, (2.0 ** -24, R.tol_state(130)), "state after a gate far below")


def test_no_rows_and_no_sequences():
    init = torch.randn(3, 2, 64, 128, generator=gen(8))
    a = R.inputs(gen(9), 0, 2, 1)
    out, final = call(a, [0, 0, 0], "bf16", init=init)
    assert torch.equal(final, init) and out.numel() == 0
    out, final = call(a, [0, 0], "bf16")
    assert not final.any()
    call(a, [], "bf16")


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [-1, 20, 50, 100], [0, 20, 50, 101], [5, 2 ** 31 - 1, 7, 9], [0, -2 ** 31, 3, 100]])
@pytest.mark.parametrize("H,rows", [(2, 100), (64, 40000)])
def test_bad_cu_seqlens_are_said_and_write_nothing_outside(cu, H, rows):
    a = {k: t.to(DEV) for k, t in R.inputs(gen(10), rows, H, 1).items()}
    cu = [v if v != 100 else rows for v in cu]
    cu = [v if v != 101 else rows + 1 for v in cu]
    n = len(cu) - 1
    guard = 4
    out = torch.full((rows + guard, H, 64), -7.0, dtype=torch.bfloat16, device=DEV)
    final = torch.full((n + 1, H, 64, 128), -7.0, device=DEV)
    size = ssu.prefill_workspace_size(rows, n, H)
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = ssu.make_prefill(torch.tensor(cu, dtype=torch.int32, device=DEV), a["x"], a["B"], a["C"], a["dt"], a["A"], a["D"],
                         a["dt_bias"], out[:rows], final_states=final[:n], workspace=ws[:size] if size else None, status=status)
    ssu.prefill(p)
    torch.cuda.synchronize()
    assert int(status) == ssu.SSU_STATUS_BAD_SEQLEN
    assert bool((out[rows:] == -7).all()) and bool((final[n:] == -7).all()) and bool((ws[size:] == 0xA5).all())


def test_nan_stays_with_its_sequence_and_head():
    g = gen(11)
    a = R.inputs(g, 200, 4, 2)
    clean, S = call(a, [100, 100], "f32")
    a["x"][30, 1] = float("nan")
    a["dt"][150, 2] = float("inf")
    out, final = call(a, [100, 100], "f32")
    for s in range(2):
        for h in range(4):
            r = slice(100 * s, 100 * s + 100)
            if (s, h) in ((0, 1), (1, 2)):
                assert not torch.isfinite(out[r, h]).all()
            else:
                assert torch.equal(out[r, h], clean[r, h]) and torch.equal(final[s, h], S[s, h]), (s, h)


def test_the_same_call_again_gives_the_same_bits():
    g = gen(12)
    a = R.inputs(g, 2300, 8, 2)
    first = call(a, [1500, 800], "bf16", gate=True)
    again = call(a, [1500, 800], "bf16", gate=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_rows_past_4_GiB():
    """x in rows so far apart that their offsets pass 32 bits."""
    g = gen(13)
    rows, stride = 700, (1 << 23) - 8
    a = R.inputs(g, rows, 2, 1)
    x = torch.empty(rows * stride, dtype=torch.bfloat16, device=DEV).as_strided((rows, 2, 64), (stride, 64, 1))
    x.copy_(a["x"])
    d = {k: t.to(DEV) for k, t in a.items() if k not in ("x", "z")}
    out, final = torch.empty(rows, 2, 64, device=DEV), torch.empty(1, 2, 64, 128, device=DEV)
    size = ssu.prefill_workspace_size(rows, 1, 2)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    p = ssu.make_prefill(torch.tensor([0, rows], dtype=torch.int32, device=DEV), x, d["B"].contiguous(), d["C"].contiguous(), d["dt"],
                         d["A"], d["D"], d["dt_bias"], out, final_states=final, workspace=ws)
    ssu.prefill(p)
    y, S, y_abs, S_abs = want(a, [rows])
    R.check(out, y, y_abs, R.tol_out(rows, "f32"), "out")
    R.check(final, S, S_abs, (2.0 ** -24, R.tol_state(rows)), "final")


# Every value on the way to a result is rounded to fp32, off by at most half a step, 2^-24 of it; a result's way has up
# to 64 such roundings that are not averaged away (dt' 8, the decays 8, the weights 4, the sums over parts and depth of
# three products 3 x 6, the update of the state and its scaling through a few chunks 16, the readout's own scaling, the
# chunk's tokens and the joining of segments 10).  Independent, they add up to sqrt(64) = 8 half steps of the norm.  An
# operand cut to two parts (16 bits) is off by up to 2^-18 = 64 half steps by itself.
LIMIT = 8 * 2.0 ** -24


@pytest.mark.parametrize("lens,H,G", [([400], 2, 1), ([100, 300, 64], 4, 2), ([1300], 4, 1)])
@pytest.mark.parametrize("out_name", ["f32", "bf16"])
def test_fp32_results_are_near(lens, H, G, out_name):
    g = gen(14 + len(lens))
    a = R.inputs(g, sum(lens), H, G)
    init = 0.3 * torch.randn(len(lens), H, 64, 128, generator=g)
    out, final = call(a, lens, out_name, init=init)
    y, S, _, _ = want(a, lens, init)
    off = (final.double() - S).flatten(2).norm(dim=2) / S.flatten(2).norm(dim=2)
    print("states off by %.2g to %.2g" % (off.min(), off.max()), flush=True)
    assert float(off.max()) <= LIMIT
    if out_name == "f32":
        off = (out.double() - y).transpose(0, 1).flatten(1).norm(dim=1) / y.transpose(0, 1).flatten(1).norm(dim=1)
        print("outputs off by %.2g to %.2g" % (off.min(), off.max()), flush=True)
        assert float(off.max()) <= LIMIT
