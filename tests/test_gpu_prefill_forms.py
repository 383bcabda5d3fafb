"""Prompts of so many sequences that a workgroup takes two heads: groups of any
number of heads, every length around a chunk's borders, segments, pieces, NaN
(the other GPU tests of prompts have few sequences, and a head a workgroup)."""
import pytest
import torch

from tests import prompt_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu
    from tests.test_gpu_prefill import call, compare, gen, want


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def lengths(n, first):
    """`first`, then short ones; more than 256 workgroups of two heads in the tests below."""
    return list(first) + [(3 * i) % 7 for i in range(n - len(first))]


@pytest.mark.parametrize("n,H,G", [(70, 8, 2), (70, 12, 4), (130, 4, 2), (100, 5, 1), (70, 14, 2)])
@pytest.mark.parametrize("out_name", ["bf16", "f32"])
def test_lengths_around_a_chunk(n, H, G, out_name):
    lens = lengths(n, [1, 16, 17, 63, 64, 65, 0, 127, 128, 129, 200])
    g = gen(n + H + G)
    a = R.inputs(g, sum(lens), H, G)
    init = 0.3 * torch.randn(n, H, 64, 128, generator=g)
    compare(a, lens, out_name, init=init, gate=H != 8)
    compare(a, lens, out_name)


@pytest.mark.parametrize("n,H,G", [(130, 4, 2), (100, 5, 1), (60, 10, 2)])
@pytest.mark.parametrize("out_name", ["bf16", "f32"])
def test_segments(n, H, G, out_name):
    lens = lengths(n, [1500, 3, 769])
    lens[-1] = 901
    g = gen(2 * n + H)
    a = R.inputs(g, sum(lens), H, G)
    init = 0.3 * torch.randn(n, H, 64, 128, generator=g)
    compare(a, lens, out_name, init=init, gate=True)
    compare(a, lens, out_name, init=init.clone(), in_place=True)


def test_both_forms_agree():
    """A few of many sequences, and the same alone."""
    lens = lengths(130, [700, 64, 0, 131])
    g = gen(9)
    a = R.inputs(g, sum(lens), 4, 2)
    many, S = call(a, lens, "f32")
    n = sum(lens[:4])
    few, T = call({k: (t[:n] if t.dim() > 1 else t) for k, t in a.items()}, lens[:4], "f32")
    cut = {k: (t[:n] if t.dim() > 1 else t) for k, t in a.items()}
    _, _, y_abs, S_abs = want(cut, lens[:4])
    R.check(few, many[:n].double(), y_abs, (2.0 ** -23, 2 * R.tol_out(700, "f32")[1]), "outputs")
    R.check(T, S[:4].double(), S_abs, (2.0 ** -23, 2 * R.tol_state(700)), "states")


def test_nan_stays_with_its_sequence_and_head():
    lens = lengths(130, [100, 150, 33])
    g = gen(10)
    a = R.inputs(g, sum(lens), 4, 2)
    clean, S = call(a, lens, "f32")
    bad = {k: t.clone() for k, t in a.items()}
    bad["x"][120, 1] = float("nan")   # sequence 1, head 1
    out, T = call(bad, lens, "f32")
    other = torch.ones(len(out), 4, dtype=torch.bool)
    other[100:250, 1] = False
    assert torch.equal(out[other], clean[other]) and bool(torch.isnan(out[120, 1]).any())
    keep = torch.ones(130, 4, dtype=torch.bool)
    keep[1, 1] = False
    assert torch.equal(T[keep], S[keep])


def test_slices_of_wider_rows_and_rows_nobody_owns():
    lens = lengths(90, [40, 0, 65])
    rows = sum(lens) + 45
    g = gen(11)
    a = R.inputs(g, rows, 6, 2, wide=24)
    for k in ("x", "B", "C", "z", "dt"):
        a[k][rows - 45:] = float("nan")
    out, _ = compare(a, lens, "bf16", gate=True)
    assert bool((out[rows - 45:] == -7).all())


@pytest.mark.parametrize("n", [3, 63, 64, 129])
def test_sequences_over_the_same_rows_write_nothing_outside(n):
    """cu_seqlens that go to the last row and back: every other sequence has all rows, and their segments are more than
    the slots."""
    g = gen(n)
    rows, H = 2000, 2
    a = R.inputs(g, rows, H, 1)
    cu = torch.tensor([rows * (i % 2) for i in range(n + 1)], dtype=torch.int32, device="cuda:0")
    d = {k: t.to("cuda:0") for k, t in a.items()}
    size = ssu.prefill_workspace_size(rows, n, H)
    ws = torch.full((size + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda:0")
    out = torch.full((rows + 64, H, 64), -7.0, device="cuda:0")
    h1 = torch.full((n + 4, H, 64, 128), -7.0, device="cuda:0")
    status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    ssu.prefill(ssu.make_prefill(cu, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], out[:rows], final_states=h1[:n],
                                 workspace=ws[:size], status=status))
    assert int(status) == ssu.SSU_STATUS_BAD_SEQLEN
    assert bool((ws[size:] == 0xA5).all()) and bool((out[rows:] == -7).all()) and bool((h1[n:] == -7).all())


def test_a_workspace_is_enough_for_fewer_rows_and_sequences():
    most = {}
    for H in (1, 4, 64, 129):
        for rows in (0, 100, 512, 513, 700, 1024, 5000, 40000, 300000):
            for n in (1, 2, 3, 17, 65, 300):
                most[H, rows, n] = ssu.prefill_workspace_size(rows, n, H)
        for (h, rows, n), size in most.items():
            assert all(size <= other for (k, r, m), other in most.items() if k == h and r >= rows and m >= n)
