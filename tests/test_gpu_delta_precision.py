"""How near the gated delta rule's fp32 results come to the rule in 64 bits, on
ordinary inputs: the figures the headers give, which the worst-case tolerances
of the other tests are far too wide to hold.

Every value on the way to a result is rounded to fp32, off by at most half a
step, 2^-24 of it.  A result's way has up to 64 such roundings that are not
averaged away: a key's and a query's unit length (sum, root, quotient, product:
4 each), the decays (exponent and exponential, 2 half steps each: 8 for a
token's own and its neighbours'), the residual (4), T's two levels of blocks
(12), the products' sums over parts and depth (3 x 6), the update (4), the
readout and its weights (10).  Independent, they add up to sqrt(64) = 8 half
steps, 8 x 2^-24 = 4.8e-7 of the norm.  An operand cut to 16 bits (two bf16
parts instead of three) is off by up to 2^-18 = 64 half steps of it by itself,
and ends past the limit.

The states of a prompt with bf16 outputs take three such operands (state, T - I,
residuals), each off by at most 2^-18 and, evenly spread, by 2^-18 / sqrt(3) in
the mean: 2^-18 together.
"""
import pytest
import torch

from tests import delta_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu

DEV = "cuda:0"
LIMIT = 8 * 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def near(got, want, what, limit=LIMIT):
    """Of every head (the leading index) the 2-norm of the difference, of the result's."""
    got, want = got.cpu().double().flatten(1), want.flatten(1)
    off = (got - want).norm(dim=1) / want.norm(dim=1)
    print("%s: off by %.2g to %.2g" % (what, off.min(), off.max()), flush=True)
    assert bool((off <= limit).all()), "%s: off by %.3g of its norm, %.3g allowed" % (what, off.max(), limit)


# sequences, tokens each, key and value heads, dims, with states: one case for each scan kernel and width of k
@pytest.mark.parametrize("n,tokens,hk,hv,dk,dv,init", [
    (1, 400, 1, 2, 128, 128, True), (1, 400, 2, 4, 64, 64, False),       # few chains
    (10, 200, 2, 4, 128, 128, False), (20, 200, 2, 4, 64, 64, True),     # more of them
    (33, 100, 2, 8, 128, 128, True), (33, 100, 2, 8, 64, 128, False)])   # whole heads
@pytest.mark.parametrize("out_name", ["f32", "bf16"])
@pytest.mark.parametrize("kept", [False, True])  # hardly any decay: an error stays
def test_prompt(n, tokens, hk, hv, dk, dv, init, out_name, kept):
    g = gen(n + dk)
    x = R.inputs(g, n * tokens, hk, hv, dk, dv)
    if kept:
        x["A"], x["beta"] = 0.01 * x["A"], x["beta"] + 2
    h0 = 0.3 * torch.randn(n, hv, dv, dk, generator=g) if init else torch.zeros(n, hv, dv, dk)
    d = {k: v.to(DEV) for k, v in x.items()}
    out, h1 = torch.empty(n * tokens, hv, dv, dtype=R.TYPES[out_name], device=DEV), torch.empty(n, hv, dv, dk, device=DEV)
    ws = torch.empty(ssu.delta_prefill_workspace_size(n * tokens, n, hv), dtype=torch.uint8, device=DEV)
    cu = torch.arange(0, n * tokens + 1, tokens, dtype=torch.int32, device=DEV)
    ssu.delta_prefill(ssu.make_delta_prefill(cu, d["q"], d["k"], d["v"], d["dt"], d["beta"], d["A"], d["dt_bias"], out,
                                             initial_states=h0.to(DEV) if init else None, final_states=h1, workspace=ws))
    gates = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"])
    for s in {0, n - 1}:
        at = slice(s * tokens, (s + 1) * tokens)
        S, want = R.run(h0[s], x["q"][at], x["k"][at], x["v"][at], gates[0][at], gates[1][at], dk ** -0.5)
        if out_name == "f32":
            near(out[at].transpose(0, 1), want.transpose(0, 1), "outputs of sequence %d" % s)
        near(h1[s], S, "state of sequence %d" % s, LIMIT if out_name == "f32" else LIMIT + 2.0 ** -18)


def cache_of(g, L, dk, dv, hv=4):
    """fp32 checkpoints of two slots, full rings, hardly any decay."""
    c = R.Cache(g, 3, 2, hv, dk, dv, L, "f32")
    gates = c.t["gate_cache"].view(3, hv, L, 2)
    gates[..., 0] = -0.02 * torch.rand(3, hv, L, generator=g)
    gates[..., 1] = 0.5 + 0.5 * torch.rand(3, hv, L, generator=g)
    return c


@pytest.mark.parametrize("L,fold,dk,dv", [(16, 1, 128, 128), (16, 4, 128, 64), (16, 16, 128, 128), (32, 32, 128, 128),
                                          (32, 20, 64, 64), (5, 5, 64, 128)])
def test_flush(L, fold, dk, dv):
    """The state, and what the fold leaves of it along the keys that it took out: there an operand's lost bits are not
    averaged over the whole state."""
    g = gen(L + fold + dk)
    c = cache_of(g, L, dk, dv)
    d, dc = c.upload(ssu, DEV)
    ids = torch.tensor([2, 1], dtype=torch.int32, device=DEV)
    ssu.delta_flush(dc, ids, torch.full_like(ids, fold))
    back = torch.empty(2, c.hv, dv, dk, device=DEV)
    ssu.delta_read_state(dc, back, ids)
    for j, slot in enumerate((2, 1)):
        k, v, gr, br = c.ring(slot, 0, fold)
        S, _ = R.run(c.states(slot), None, k, v, gr, br, 1.0)
        near(back[j], S, "state of slot %d" % slot)
        keys = R.unit(k).repeat_interleave(c.hv // c.hk, 1).permute(1, 2, 0)  # [hv, dk, fold]
        was = (c.states(slot).double() @ keys).flatten(1).norm(dim=1) + v.double().norm(dim=(0, 2))
        off = ((back[j].cpu().double() - S) @ keys).flatten(1).norm(dim=1) / was
        print("along the keys: %.2g to %.2g" % (off.min(), off.max()), flush=True)
        assert bool((off <= LIMIT).all()), "along the keys off by %.3g, %.3g allowed" % (off.max(), LIMIT)


@pytest.mark.parametrize("L,live,T,dk,dv", [(16, 0, 1, 128, 128), (16, 12, 4, 128, 64), (32, 16, 16, 128, 128), (32, 20, 7, 64, 64)])
def test_step(L, live, T, dk, dv):
    g = gen(L + live + dk)
    c = cache_of(g, L, dk, dv)
    d, dc = c.upload(ssu, DEV)
    x = R.inputs(g, 2 * T, 2, 4, dk, dv)
    dev = {n: t.to(DEV) for n, t in x.items()}
    ids, out = torch.tensor([2, 1], dtype=torch.int32, device=DEV), torch.empty(2 * T, 4, dv, device=DEV)
    ssu.delta_replay_step(dc, ssu.make_delta_step(dc, T, ids, torch.full_like(ids, live), None, dev["q"], dev["k"], dev["v"], dev["dt"],
                                                  dev["beta"], dev["A"], dev["dt_bias"], out))
    gates = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"])
    for j, slot in enumerate((2, 1)):
        at = slice(j * T, (j + 1) * T)
        k, v, gr, br = c.ring(slot, 0, live)
        S, _ = R.run(c.states(slot), None, k, v, gr, br, 1.0)
        _, want = R.run(S, x["q"][at], x["k"][at], x["v"][at], gates[0][at], gates[1][at], dk ** -0.5)
        near(out[at].transpose(0, 1), want.transpose(0, 1), "outputs of slot %d" % slot)
