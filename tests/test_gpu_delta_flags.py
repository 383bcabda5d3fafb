"""The flags of prompts and flushes (keys and queries as they are, dt and beta
as they are, a scale of the caller's) against the rule in 64 bits: each of those
kernels reads them for itself."""
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


FLAGS = [(False, True, True, None), (True, False, True, None), (True, True, False, 0.5), (False, False, False, 2.0)]


def flagged(g, rows, hk, hv, dk, dv, norm, softplus, sigmoid):
    """Inputs as a model with those flags would give them: keys not scaled by the kernel are short, gates taken as they
    are lie where the activations would put them."""
    x = R.inputs(g, rows, hk, hv, dk, dv)
    if not norm:
        x["k"] = 0.1 * x["k"]
    if not softplus:
        x["dt"], x["dt_bias"] = 0.2 * x["dt"].abs(), torch.full((hv,), 0.01)
    if not sigmoid:
        x["beta"] = torch.rand(rows, hv, generator=g)
    return x


# a few chains, more of them, whole heads: the three kernels that take prompts
@pytest.mark.parametrize("n,tokens,hk,hv,dk,dv", [(2, 75, 1, 2, 64, 64), (10, 70, 2, 4, 128, 128), (33, 40, 2, 8, 64, 128)])
@pytest.mark.parametrize("norm,softplus,sigmoid,scale", FLAGS)
@pytest.mark.parametrize("out_name", ["f32", "bf16"])
def test_prompt(n, tokens, hk, hv, dk, dv, norm, softplus, sigmoid, scale, out_name):
    g = gen(n + FLAGS.index((norm, softplus, sigmoid, scale)))
    x = flagged(g, n * tokens, hk, hv, dk, dv, norm, softplus, sigmoid)
    h0 = 0.3 * torch.randn(n, hv, dv, dk, generator=g)
    d = {k: v.to(DEV) for k, v in x.items()}
    out, h1 = torch.empty(n * tokens, hv, dv, dtype=R.TYPES[out_name], device=DEV), torch.empty(n, hv, dv, dk, device=DEV)
    ws = torch.empty(ssu.delta_prefill_workspace_size(n * tokens, n, hv), dtype=torch.uint8, device=DEV)
    cu = torch.arange(0, n * tokens + 1, tokens, dtype=torch.int32, device=DEV)
    ssu.delta_prefill(ssu.make_delta_prefill(cu, d["q"], d["k"], d["v"], d["dt"], d["beta"], d["A"], d["dt_bias"], out,
                                             initial_states=h0.to(DEV), final_states=h1, workspace=ws, scale=scale, dt_softplus=softplus,
                                             beta_sigmoid=sigmoid, qk_norm=norm))
    gates = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"], softplus, sigmoid)
    scale = dk ** -0.5 if scale is None else scale
    for s in {0, n - 1}:
        at = slice(s * tokens, (s + 1) * tokens)
        S, want = R.run(h0[s], x["q"][at], x["k"][at], x["v"][at], gates[0][at], gates[1][at], scale, norm)
        went = h0[s].double().flatten(1).norm(dim=1) + x["v"][at].double().transpose(0, 1).flatten(1).norm(dim=1)
        read = scale * (1.0 if norm else float(x["q"][at].double().norm(dim=-1).max()))  # what a query makes of it
        windows = -(-tokens // 32)
        R.check(out[at].cpu().transpose(0, 1), want.transpose(0, 1), went * read, R.tol(dk, 32, windows, out_name), "outputs %d" % s)
        R.check(h1[s].cpu(), S, went, R.tol(dk, 32, windows, "f32", out_name), "state %d" % s)


@pytest.mark.parametrize("state,L,fold,dk,dv", [("f32", 16, 11, 128, 64), ("bf16", 32, 32, 64, 128), ("f16", 16, 16, 128, 128)])
def test_flush_of_keys_as_they_are(state, L, fold, dk, dv):
    g = gen(L + fold)
    c = R.Cache(g, 4, 2, 4, dk, dv, L, state)
    c.t["k_cache"] = 0.1 * c.t["k_cache"]
    d, dc = c.upload(ssu, DEV, norm=False)
    ids = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    ssu.delta_flush(dc, ids, torch.full_like(ids, fold))
    got = c.download(d)
    for slot in (3, 1):
        k, v, gr, br = c.ring(slot, 0, fold)
        S, _ = R.run(c.states(slot), None, k, v, gr, br, 1.0, norm=False)
        have = got["state"][slot].view(c.hv, -1)[:, c.place].view(c.hv, dv, dk)
        went = c.states(slot).double().flatten(1).norm(dim=1) + v.double().transpose(0, 1).flatten(1).norm(dim=1)
        R.check(have, S, went, R.tol(dk, fold, 1, state), "slot %d" % slot)


def test_a_prompt_and_the_steps_that_continue_it_agree_on_the_flags():
    """40 tokens as one prompt, and as a prompt of 25 whose states go into a cache that takes the rest in steps."""
    g = gen(31)
    hk, hv, dk, dv = 1, 2, 64, 64
    x = flagged(g, 40, hk, hv, dk, dv, False, False, False)
    d = {k: v.to(DEV) for k, v in x.items()}
    flags = dict(scale=0.3, dt_softplus=False, beta_sigmoid=False)

    def prompt(rows, out, h1):
        ws = torch.empty(ssu.delta_prefill_workspace_size(rows, 1, hv), dtype=torch.uint8, device=DEV)
        part = {k: v[:rows] if k not in ("A", "dt_bias") else v for k, v in d.items()}
        cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        ssu.delta_prefill(ssu.make_delta_prefill(cu, part["q"], part["k"], part["v"], part["dt"], part["beta"], part["A"],
                                                 part["dt_bias"], out, final_states=h1, workspace=ws, qk_norm=False, **flags))

    whole, h1 = torch.empty(40, hv, dv, device=DEV), torch.empty(1, hv, dv, dk, device=DEV)
    prompt(40, whole, h1)
    head, h0 = torch.empty(25, hv, dv, device=DEV), torch.empty(1, hv, dv, dk, device=DEV)
    prompt(25, head, h0)
    c = R.Cache(g, 3, hk, hv, dk, dv, 16, "f32")
    t, dc = c.upload(ssu, DEV, norm=False)
    ids = torch.tensor([2], dtype=torch.int32, device=DEV)
    ssu.delta_init_state(dc, h0, ids)
    tail = torch.empty(15, hv, dv, device=DEV)
    for i in range(0, 15, 5):
        rows = slice(25 + i, 30 + i)
        part = {k: v[rows].contiguous() if k not in ("A", "dt_bias") else v for k, v in d.items()}
        ssu.delta_replay_step(dc, ssu.make_delta_step(dc, 5, ids, torch.tensor([i], dtype=torch.int32, device=DEV), None, part["q"], part["k"],
                                                      part["v"], part["dt"], part["beta"], part["A"], part["dt_bias"], tail[i:i + 5], **flags))
    ssu.delta_flush(dc, ids, torch.tensor([15], dtype=torch.int32, device=DEV))
    back = torch.empty_like(h1)
    ssu.delta_read_state(dc, back, ids)
    both = lambda t, w: [a + b for a, b in zip(R.tol(dk, 32, t, "f32"), R.tol(dk, 15, w, "f32"))]  # noqa: E731  (either side may be off)
    went = x["v"].double().transpose(0, 1).flatten(1).norm(dim=1)
    read = 0.3 * float(x["q"].double().norm(dim=-1).max())
    got = torch.cat([head, tail]).cpu().transpose(0, 1)
    R.check(got, whole.cpu().double().transpose(0, 1), went * read, both(2, 1), "outputs")
    R.check(back[0].cpu(), h1[0].cpu().double(), went, both(2, 2), "state")
