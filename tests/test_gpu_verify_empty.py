"""Verification where a rejected draft leaves nothing of the residual (p <= q
everywhere) and the token comes from the row itself: entries of that kind beside
ordinary ones, in both launch forms, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_verify import as_type, draw, reference, run

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# entries, vocabulary, type: one launch (short rows; many entries of two bytes a value), two launches, a part of a piece at the
# end or none, more pieces than lanes
CASES = [(5, 1, "f32"), (5, 1000, "f32"), (4, 1024, "bf16"), (6, 40000, "f16"), (6, 40961, "f32"), (5, 65536, "bf16"),
         (3, 300001, "f32"), (200, 41003, "bf16")]


def problem(entries, vocab, dtype):
    """Two rows an entry; entry b's only draft is a token that p gives nothing, every third entry's q is p."""
    rng = np.random.default_rng(entries + vocab)
    p = draw(rng, 2 * entries, vocab)
    drafts = rng.integers(0, vocab, entries)
    q = draw(rng, 2 * entries, vocab)
    for b in range(entries):
        p[2 * b, drafts[b]] = 0.0
        if b % 3 == 0:
            q[2 * b] = p[2 * b]
        if b % 6 == 3 and vocab > 2000:  # all of its mass behind the middle
            p[2 * b, : vocab // 2] = 0.0
            q[2 * b] = p[2 * b]
    tokens = np.stack([np.zeros(entries, np.int64), drafts], 1).reshape(-1)
    u, uf = np.full(2 * entries, 0.5, np.float32), rng.random(entries).astype(np.float32)
    uf[0] = 0.0
    return tokens, p, q, u, uf


@pytest.mark.parametrize("case", CASES)
def test_empty_residuals_beside_others(case):
    entries, vocab, dtype = case
    tokens, p, q, u, uf = problem(*case)
    print("empty residuals", case, flush=True)
    out, acc, status = run(tokens, p, q, u, uf, 2, dtype=dtype)
    want, count, bits = reference(tokens, as_type(p, dtype), as_type(q, dtype), u, uf, np.arange(0, 2 * entries + 1, 2), 2, vocab)
    assert status == bits
    assert np.array_equal(acc, count) and np.array_equal(out, want)


@pytest.mark.parametrize("vocab", [3000, 70000])
def test_rows_of_nothing_at_all(vocab):
    """Neither the residual nor the row has mass, beside an entry without tokens and one that accepts: counts in place."""
    p = np.zeros((5, vocab), np.float32)
    p[3, 7], p[4, 9] = 1.0, 1.0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    live = i32([3, 5, 6])
    out, acc, status = run([0, 4, 0, 0, 7], p, p, np.zeros(5, np.float32), np.float32([0.5] * 3), 2, cu=[0, 2, 2, 4],
                           book=dict(live=live, ring_len=16, next_live=live))
    assert out.tolist() == [[-1, -1], [-1, -1], [-1, -1]] and acc.tolist() == [1, 0, 1]
    assert status == ssu.SSU_STATUS_BAD_PROBS and live.tolist() == [4, 5, 7]


def test_replayed_in_a_graph():
    """Captured once, replayed over new probabilities with eager calls between: the scratch holds the last call's sums."""
    entries, vocab = 4, 70000
    first, second = problem(entries, vocab, "f32"), problem(entries + 1, vocab, "f32")
    rows = 2 * entries
    dev = lambda x, dt: torch.as_tensor(np.asarray(x)[:rows], dtype=dt).to(DEV)  # noqa: E731
    tokens, p, q = dev(first[0], torch.int32), dev(first[1], torch.float32), dev(first[2], torch.float32)
    u, uf = dev(first[3], torch.float32), torch.as_tensor(first[4]).to(DEV)
    out, acc = torch.empty(entries, 2, dtype=torch.int32, device=DEV), torch.empty(entries, dtype=torch.int32, device=DEV)
    ws = torch.empty(ssu.verify_workspace_size(entries, vocab), dtype=torch.uint8, device=DEV)
    call = ssu.make_verify(tokens, p, q, u, uf, out, acc, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        ssu.verify(call)
    for at, (tk, pp, qq, _, _) in enumerate((first, second, first, second)):
        tokens.copy_(dev(tk, torch.int32)), p.copy_(dev(pp, torch.float32)), q.copy_(dev(qq, torch.float32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy()
        want, _, _ = reference(tk[:rows], pp[:rows].astype(np.float64), qq[:rows].astype(np.float64), first[3], first[4],
                               np.arange(0, rows + 1, 2), 2, vocab)
        assert np.array_equal(got, want), at
        ssu.verify(call)  # eager, over the same scratch
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want), at
