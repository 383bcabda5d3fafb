"""What the two launch forms of ssu_logits (a workgroup a row, pieces of a row)
have to do alike, and the two of ssu_history_count; prompts of more sequences
than one workgroup looks through at once."""
import numpy as np
import pytest
import torch

from tests import prompt_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu
    from tests.test_gpu_logits import Case, Pages, check, i32

DEV = "cuda:0"
FORMS = [3001, 16384, 16385, 20011]   # whole rows up to 16384 values, pieces of so few longer ones


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("vocab", FORMS)
def test_infinities_and_nan(vocab):
    inf, nan = float("inf"), float("nan")
    c = Case(4, 6, 1, vocab, history=False, mask=0.9, temperature=[1.0, 0.7, 1.3, 1.0, 0.0, 0.5])
    last = vocab - 1
    c.wide[0, 5] = c.wide[0, last] = inf
    c.mask[0, 5] = c.mask[0, last] = True
    c.wide[1, :] = -inf
    c.wide[1, 17] = nan
    c.wide[2, 3] = nan
    c.wide[3, ::2] = torch.finfo(torch.float32).min   # a mask's lowest value is a value like others
    c.wide[3, 1::2] = nan
    c.wide[4, [2500, last]] = inf                     # a greedy row takes the first
    c.wide[4, 2000] = torch.finfo(torch.float32).max  # ... and this is as large
    c.wide[4, 7] = nan
    c.mask[4, [2000, 2500, 7]] = True
    c.wide[5, :] = nan
    c.wide[5, last] = -5.0
    c.mask[5, last] = True
    out = check(c)
    assert float(out[0, 5]) == 0.5 and float(out[0, last]) == 0.5 and not out[1].any() and float(out[2, 3]) == 0.0
    assert int(out[4].argmax()) == 2000 and float(out[5, last]) == 1.0


@pytest.mark.parametrize("vocab", FORMS)
@pytest.mark.parametrize("it", ["f32", "bf16"])
def test_greedy_rows(vocab, it):
    c = Case(vocab, 6, 2, vocab, it=it, bias=4, mask=0.5, temperature=[0.0, -1.0, 0.8, float("nan"), 0.0, 0.0])
    c.mask[0] = False                  # nothing is left of one
    c.wide[8, [vocab - 1, 7]] = 60.0   # ties
    c.mask[8, [vocab - 1, 7]] = True
    c.wide[10, vocab - 1] = 80.0       # the last value
    c.mask[10, vocab - 1] = True
    check(c, it)


@pytest.mark.parametrize("temperature", [float("inf"), 0.5, 0.0])
def test_what_is_left_out_stays_out_without_softmax(temperature):
    c = Case(12, 3, 2, 3001, mask=0.5, temperature=[temperature] * 3)
    c.wide[0, ::5] = float("nan")
    c.wide[1, ::3] = -float("inf")
    out = c.call("f32", softmax=False)[0]
    x = torch.from_numpy(c.x())
    assert torch.equal(out == -float("inf"), x == -float("inf")) and not bool(torch.isnan(out).any())


@pytest.mark.parametrize("vocab", FORMS)
def test_rows_that_a_mask_leaves_nothing_of(vocab):
    c = Case(3, 3, 2, vocab, mask=0.5)
    c.mask[2] = False
    c.mask[5] = False
    c.mask[5, vocab - 2] = True
    out = check(c)
    assert not out[2].any() and float(out[5, vocab - 2]) == 1.0


# more special tokens than a workgroup lists at a time, or nearly so
@pytest.mark.parametrize("b,T,vocab,fill", [(3, 2, 9001, 0.6), (2, 3, 16001, 1.0), (70, 2, 20003, 0.3), (40, 1, 70001, 0.2), (3, 1, 4096, 1.0)])
@pytest.mark.parametrize("it", ["f32", "bf16"])
def test_full_histories(b, T, vocab, fill, it):
    c = Case(b + vocab, b, T, vocab, it=it, bias=6, mask=0.7, fill=fill, pages=Pages(b + 2, vocab, 1, fill))
    c.temperature[0] = 0.0
    out = check(c, it)
    assert torch.equal(c.call(it, in_place=True)[0], out)


@pytest.mark.parametrize("vocab", [2049, 20011])
def test_rows_at_odd_addresses(vocab):
    """Rows of 16-bit values that begin at any multiple of two bytes."""
    c = Case(vocab, 4, 2, vocab, it="bf16", bias=3, mask=0.8, stride=1)
    check(c, "bf16")
    want = c.call("f32")[0]
    flat = torch.zeros(c.rows * (vocab + 1) + 8, dtype=torch.bfloat16, device=DEV)
    for off in (1, 3, 6):
        wide = flat[off:off + c.rows * (vocab + 1)].view(c.rows, vocab + 1)
        wide.copy_(c.wide)
        args = {}
        c.call("f32", keep=args)
        made = args["args"]
        made.logits = wide.data_ptr()
        args["out"].zero_()
        ssu.logits(made)
        torch.cuda.synchronize()
        assert torch.equal(args["out"].cpu(), want), off


@pytest.mark.parametrize("vocab", [131072, 131073, 300001])
@pytest.mark.parametrize("reset", [True, False])
def test_prompts_of_large_vocabularies(vocab, reset):
    """Up to 131072 tokens a prompt's bits are collected in LDS, above not."""
    rng = np.random.default_rng(vocab)
    p = Pages(5, vocab, 3, 0.01)
    lens = [3000, 0, 1, 4097]
    cu = np.concatenate([[0], np.cumsum(lens)])
    tokens = (vocab * rng.random(cu[-1]) ** 4).astype(np.int32)
    tokens[[5, 3000]] = [vocab, vocab - 1]
    ssu.count(ssu.make_count(p.history, i32([2, 1, 4, 3]), i32(tokens), cu_seqlens=i32(cu), prompt=True, reset=reset))
    for j, s in enumerate([2, 1, 4, 3]):
        p.add(s, tokens[cu[j]:cu[j + 1]].tolist(), True, reset)
    p.check()
    assert int(p.status) == ssu.SSU_STATUS_BAD_TOKEN


@pytest.mark.parametrize("n,long", [(64, [0, 63]), (65, [3, 64]), (200, [0, 77, 199])])
@pytest.mark.parametrize("H,G,out_name", [(2, 1, "f32"), (1, 1, "bf16"), (3, 3, "bf16")])
def test_many_sequences_some_of_them_in_segments(n, long, H, G, out_name):
    g = torch.Generator()
    g.manual_seed(n + H)
    lens = torch.randint(0, 6, (n,), generator=g).tolist()
    for i, s in enumerate(long):
        lens[s] = 900 + 400 * i
    cu = [sum(lens[:i]) for i in range(n + 1)]
    rows = cu[-1]
    x = R.inputs(g, rows, H, G)
    h0 = 0.3 * torch.randn(n, H, 64, 128, generator=g)
    out = torch.empty(rows, H, 64, dtype=torch.float32 if out_name == "f32" else torch.bfloat16, device=DEV)
    h1 = torch.empty(n, H, 64, 128, device=DEV)
    d = {k: v.to(DEV) for k, v in x.items()}
    ws = torch.empty(max(16, ssu.prefill_workspace_size(rows, n, H)), dtype=torch.uint8, device=DEV)
    ssu.prefill(ssu.make_prefill(i32(cu), d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], out, initial_states=h0.to(DEV),
                                 final_states=h1, workspace=ws))
    dd, gg = R.gates(x["dt"], x["A"], x["dt_bias"])
    for s in sorted({0, 1, 2, n // 2, n - 2, n - 1, *long}):
        at = slice(cu[s], cu[s + 1])
        seq = [x[k][at] for k in ("x", "B", "C")]
        S, y = R.run(h0[s], *seq, dd[at], gg[at], x["D"])
        Sa, ya = R.run(h0[s].abs(), *(t.abs() for t in seq), dd[at], gg[at], x["D"].abs())
        R.check(out[at], y, ya, R.tol_out(lens[s], out_name), "outputs of %d" % s)
        R.check(h1[s], S, Sa, (2.0 ** -24, R.tol_state(lens[s])), "state of %d" % s)
