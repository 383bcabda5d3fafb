"""Verification of drafted tokens on the GPU against the definition of
include/ssu_verify.h in 64 bits (numpy).  Tokens, counts and bookkeeping are
whole numbers and must be equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def reference(tokens, p, q, u, uf, cu, T, vocab):
    """(out_tokens, num_accepted, status) from float64 arrays."""
    outs, counts, bits = [], [], 0
    for b in range(len(uf)):
        first, n_rows = int(cu[b]), int(cu[b + 1] - cu[b])
        out = [-1] * T
        if n_rows < 0 or n_rows > T or first < 0:
            outs.append(out), counts.append(0)
            bits |= 4
            continue
        if n_rows == 0:
            outs.append(out), counts.append(0)
            continue
        n, rejected = 0, False
        while n < n_rows - 1:
            d = int(tokens[first + n + 1])
            if not 0 <= d < vocab:
                bits |= 16
                d = -1
                rejected = True
                break
            chance = 1.0 if q is None else q[first + n, d]
            if not float(u[first + n]) * chance < p[first + n, d]:
                rejected = True
                break
            out[n] = d
            n += 1
        row = first + n
        with np.errstate(all="ignore"):
            whole = np.where(p[row] > 0, p[row], 0.0)
            r = whole
            if rejected and d >= 0:
                less = q[row] if q is not None else (np.arange(vocab) == d) * 1.0
                r = (p[row] - less).astype(np.float32).astype(np.float64)
                r = np.where(r > 0, r, 0.0)
            if not r.sum() > 0:
                r = whole
            total = r.sum()
        if not total > 0 or not np.isfinite(total):
            bits |= 32
            out[n] = -1
        else:
            want = max(float(uf[b]), 0.0) * total
            hit = np.nonzero((np.cumsum(r) > want) & (r > 0))[0]
            out[n] = int(hit[0]) if len(hit) else int(np.nonzero(r > 0)[0][-1])
        outs.append(out), counts.append(n + 1)
    return np.array(outs, np.int32).reshape(len(uf), T), np.array(counts, np.int32), bits


def run(tokens, p, q, u, uf, T, cu=None, dtype="f32", stride=None, book=None, status=None):
    """One call; p, q float arrays on the host."""
    rows, vocab = p.shape
    b = len(uf)

    def probs(x):
        if x is None:
            return None
        w = torch.full((rows, stride or vocab), float("nan"), dtype=TYPES[dtype], device=DEV)
        w[:, :vocab] = torch.as_tensor(x).to(TYPES[dtype]).to(DEV)
        return w[:, :vocab]

    i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    f32 = lambda x: torch.as_tensor(np.asarray(x, np.float32)).to(DEV)  # noqa: E731
    out = torch.full((b, T), -7, dtype=torch.int32, device=DEV)
    acc = torch.full((b,), -7, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(16, ssu.verify_workspace_size(b, vocab)), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = ssu.make_verify(i32(tokens), probs(p), probs(q), f32(u), f32(uf), out, acc, ws, None if cu is None else i32(cu),
                        status=status, **(book or {}))
    ssu.verify(d)
    torch.cuda.synchronize()
    return out.cpu().numpy(), acc.cpu().numpy(), int(status)


def as_type(x, dtype):
    return None if x is None else torch.as_tensor(x).to(TYPES[dtype]).double().numpy()


def draw(rng, rows, vocab, sharp=3.0):
    x = np.exp(sharp * rng.standard_normal((rows, vocab)))
    return (x / x.sum(1, keepdims=True)).astype(np.float32)


CASES = [  # batch, T, vocab, dtype, draft probabilities, row stride - vocab (0: as packed)
    (1, 1, 1, "f32", True, 0), (3, 4, 2, "f32", True, 0), (5, 4, 7, "bf16", False, 0), (4, 5, 1000, "f32", True, 24),
    (7, 3, 4095, "f16", True, 1), (7, 3, 4096, "f32", False, 0), (7, 3, 4097, "bf16", True, 0), (2, 64, 300, "f32", True, 0),
    (40, 8, 9001, "f32", True, 3), (3, 2, 100003, "bf16", False, 0), (33, 2, 12288, "f16", True, 8),
    # the two launches and the one at their border, entries that fill the card
    (5, 3, 40960, "f32", True, 0), (5, 3, 40961, "f32", False, 0), (195, 2, 41000, "bf16", True, 0), (195, 2, 41003, "f16", False, 1),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("varlen", [False, True])
def test_against_the_definition(case, varlen):
    b, T, vocab, dtype, drafts, extra = case
    rng = np.random.default_rng(b * 100 + T + vocab + varlen)
    lens = rng.integers(0, T + 1, b) if varlen else np.full(b, T)
    cu = np.concatenate([[0], np.cumsum(lens)]) + (2 if varlen else 0)
    rows = int(cu[-1]) + (3 if varlen else 0)
    p = draw(rng, rows, vocab)
    q = np.exp(0.7 * rng.standard_normal((rows, vocab))) * p if drafts else None
    if drafts:
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    pick = np.array([rng.choice(vocab, p=(w := (q if drafts else p)[r].astype(np.float64)) / w.sum()) for r in range(rows)])
    tokens = np.concatenate([rng.integers(0, vocab, 1), pick[:-1]]).astype(np.int32)  # row r's draft is fed in row r + 1
    u, uf = rng.random(rows).astype(np.float32), rng.random(b).astype(np.float32)
    if not drafts:
        u = (u * 2 * p[np.arange(rows), pick]).astype(np.float32)
    p64, q64 = as_type(p, dtype), as_type(q, dtype)
    print("verify", case, varlen, flush=True)
    out, acc, status = run(tokens, p, q, u, uf, T, cu if varlen else None, dtype, vocab + extra if extra else None)
    want, count, bits = reference(tokens, p64, q64, u, uf, cu, T, vocab)
    assert status == bits
    assert np.array_equal(acc, count)
    assert np.array_equal(out, want)


def test_borders():
    """u q = p exactly rejects, one step of u less accepts; u' 0 and the last number below 1; a single value with mass."""
    p = np.array([[0.25, 0.5, 0.25, 0.0]] * 2, np.float32)
    q = np.array([[0.5, 0.5, 0.0, 0.0]] * 2, np.float32)
    below = np.nextafter(np.float32(0.5), np.float32(0))
    last = np.nextafter(np.float32(1), np.float32(0))
    for u, uf, want in ((0.5, 0.0, [2, -1]), (below, 0.0, [0, 0]), (below, last, [0, 2]), (below, 0.25, [0, 1]), (below, 0.75, [0, 2])):
        out, acc, status = run([3, 0], p, q, [u, 0.0], [uf], 2)
        assert out.tolist() == [want] and status == 0, (u, uf)
    # a draft that the target gives nothing, and one that neither gives anything
    out, acc, _ = run([0, 3], p, None, [0.0, 0.0], [0.5], 2)
    assert out.tolist() == [[1, -1]] and acc.tolist() == [1]
    out, acc, _ = run([0, 3], p, q, [0.0, 0.0], [0.5], 2)
    assert out.tolist() == [[2, -1]] and acc.tolist() == [1]


def test_rows_without_mass():
    z, one = [0.0] * 5, [0.0, 1.0, 0.0, 0.0, 0.0]
    nan, inf = float("nan"), float("inf")
    # p = q where the draft is impossible: r is empty, the token comes from p
    out, _, status = run([0, 4], np.array([one, one], np.float32), np.array([one, one], np.float32), [0.5, 0], [0.3], 2)
    assert out.tolist() == [[1, -1]] and status == 0
    # nothing at all; only NaN; an infinite one; negative ones: no token
    for row in (z, [nan] * 5, [0.1, inf, 0, 0, 0], [-1.0, -0.5, 0, 0, 0]):
        out, acc, status = run([2], np.array([row], np.float32), None, [0.0], [0.5], 1)
        assert out.tolist() == [[-1]] and acc.tolist() == [1] and status == ssu.SSU_STATUS_BAD_PROBS, row
    # NaN beside numbers counts as nothing; a NaN draft probability rejects
    out, _, status = run([2], np.array([[nan, 0.2, nan, 0.8, nan]], np.float32), None, [0.0], [0.5], 1)
    assert out.tolist() == [[3]] and status == 0
    out, _, _ = run([0, 1], np.array([one, one], np.float32), np.array([[nan] * 5] * 2, np.float32), [0.0, 0], [0.5], 2)
    assert out.tolist() == [[1, -1]]
    # uniform numbers that are none: below 0 and NaN draw the first, past 1 the last
    for uf, want in ((-3.0, 1), (nan, 1), (1.0, 3), (7.0, 3)):
        out, _, _ = run([2], np.array([[0, 0.2, 0, 0.8, 0]], np.float32), None, [0.0], [uf], 1)
        assert out.tolist() == [[want]], uf


@pytest.mark.parametrize("vocab", [3000, 50000])
def test_an_empty_residual_draws_from_the_row(vocab):
    """p = q and a draft that neither gives anything: every piece is summed again, in one launch and in two."""
    rng = np.random.default_rng(6)
    p = draw(rng, 8, vocab)
    p[:, 17] = 0.0
    uf = np.float32([0.0, 0.3, 0.7, 0.9999])
    out, acc, status = run([5, 17] * 4, p, p, [0.5] * 8, uf, 2)
    want, count, bits = reference([5, 17] * 4, p.astype(np.float64), p.astype(np.float64), [0.5] * 8, uf, np.arange(0, 9, 2), 2, vocab)
    assert np.array_equal(out, want) and np.array_equal(acc, count) and status == bits == 0


def test_tokens_outside_the_vocabulary():
    p = np.array([[0.25, 0.75]] * 3, np.float32)
    for bad in (-1, 2, 2 ** 31 - 1, -2 ** 31):
        out, acc, status = run([0, 1, bad], p, None, [0.0, 0.0, 0.0], [0.5], 3)
        assert out.tolist() == [[1, 1, -1]] and acc.tolist() == [2] and status == ssu.SSU_STATUS_BAD_TOKEN


def test_lengths_outside_the_limits():
    p = np.tile(np.array([[0.25, 0.75]], np.float32), (8, 1))
    out, acc, status = run([1] * 8, p, None, [0.0] * 8, [0.5] * 3, 3, cu=[0, 4, 2, 5])
    assert status == ssu.SSU_STATUS_BAD_SEQLEN and acc.tolist() == [0, 0, 3]
    assert out.tolist() == [[-1] * 3, [-1] * 3, [1, 1, 1]]
    # a length that is 1 only where the difference wraps
    out, acc, status = run([1] * 8, p, None, [0.0] * 8, [0.5] * 2, 3, cu=[2 ** 31 - 1, -2 ** 31, 1])
    assert status == ssu.SSU_STATUS_BAD_SEQLEN and acc.tolist() == [0, 0] and out.tolist() == [[-1] * 3] * 2


def test_more_segments_than_threads():
    """A row of 300 segments: the running sum goes over them in two rounds."""
    vocab = 4096 * 300 - 5
    rng = np.random.default_rng(3)
    p = (rng.random((3, vocab)) / vocab).astype(np.float32)
    p[1, :4096 * 270] = 0.0
    p[2, 4096 * 40:] = 0.0
    for uf in (0.0, 0.2, 0.9, 0.9999, float(np.nextafter(np.float32(1), np.float32(0)))):
        out, acc, _ = run([0, 0, 0], p, None, [0.0] * 3, [uf] * 3, 1)
        want, _, _ = reference([0, 0, 0], p.astype(np.float64), None, [0.0] * 3, np.float32([uf] * 3), [0, 1, 2, 3], 1, vocab)
        assert np.array_equal(out, want), uf


@pytest.mark.parametrize("fused", [True, False])
def test_ring_bookkeeping(fused):
    """next_live = live - fold + kept; all of it is folded where max_seqlen more would not fit; in place as well."""
    rng = np.random.default_rng(4)
    b, T, L, vocab = 50, 4, 16, 33
    p = draw(rng, b * T, vocab)
    tokens = rng.integers(0, vocab, b * T)
    u = rng.random(b * T) * 0.1
    live = rng.integers(0, L - T + 1, b).astype(np.int32)
    fold = (rng.random(b) * (live + 1)).astype(np.int32)
    to = lambda x: torch.as_tensor(x).to(DEV)  # noqa: E731
    lv, fl, left = to(live), to(fold), torch.empty(b, dtype=torch.int32, device=DEV)
    book = dict(live=lv, fold=fl if fused else None, ring_len=L, next_live=lv, next_fold=fl, next_left=left)
    out, acc, _ = run(tokens, p, None, u, rng.random(b), T, book=book)
    want = live - (fold if fused else 0) + acc
    assert len(set(acc.tolist())) > 1
    nf = np.where(want + T > L, want, 0)
    assert np.array_equal(lv.cpu().numpy(), want) and np.array_equal(fl.cpu().numpy(), nf)
    assert np.array_equal(left.cpu().numpy(), want - nf) and (nf == 0).any() and (fused or (nf > 0).any())


def test_drawn_tokens_follow_the_target():
    """Many verifications of one drafted token: the first emitted token is distributed as p, whatever q drafted
    (the property the method is used for).  32768 draws: each frequency within 5 standard deviations."""
    n = 32768
    rng = np.random.default_rng(5)
    p = np.array([0.1, 0.2, 0.3, 0.05, 0.35], np.float32)
    q = np.array([0.4, 0.1, 0.1, 0.3, 0.1], np.float32)
    drafts = rng.choice(5, size=n, p=q.astype(np.float64) / q.astype(np.float64).sum())
    tokens = np.stack([np.zeros(n, np.int64), drafts], 1).reshape(-1)
    out, _, _ = run(tokens, np.tile(p, (2 * n, 1)), np.tile(q, (2 * n, 1)), rng.random(2 * n), rng.random(n), 2)
    freq = np.bincount(out[:, 0], minlength=5) / n
    assert np.all(np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / n)), freq


def test_rows_past_4_gib():
    """Probability rows past 2^32 bytes, as at the front."""
    vocab, rows = 131072, 8400
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    few = torch.softmax(torch.randn(8, vocab, generator=g, device=DEV), -1)
    far = torch.zeros(rows, vocab, device=DEV)
    far[-8:] = few
    tokens, u, uf = [5, 77] * 4, [0.0, 0.5] * 4, [0.1, 0.4, 0.6, 0.9]
    print("rows past 4 GiB", flush=True)

    def call(p, cu):
        n = p.shape[0]
        pad = lambda x, dt: torch.cat([torch.zeros(n - 8, dtype=dt), torch.tensor(x, dtype=dt)]).to(DEV)  # noqa: E731
        out, acc = torch.empty(4, 2, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int32, device=DEV)
        ws = torch.empty(ssu.verify_workspace_size(4, vocab), dtype=torch.uint8, device=DEV)
        ssu.verify(ssu.make_verify(pad(tokens, torch.int32), p, None, pad(u, torch.float32), torch.tensor(uf, device=DEV), out, acc, ws,
                                   torch.tensor(cu, dtype=torch.int32, device=DEV)))
        return out.tolist(), acc.tolist()

    want = call(few, [0, 2, 4, 6, 8])
    assert call(far, [rows - 8, rows - 6, rows - 4, rows - 2, rows]) == want and min(want[0][0]) >= 0
