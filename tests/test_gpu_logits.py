"""ssu_history_count and ssu_logits on the GPU against their definitions in 64
bits (counts must be equal)."""
import math

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Pages:
    """A history on the device, rows padded, and its mirror: per slot {token: word}."""

    def __init__(self, slots, vocab, seed, fill=0.0):
        rng = np.random.default_rng(seed)
        self.slots, self.vocab, words = slots, vocab, (vocab + 31) // 32
        self.counts = rng.integers(-5, 1 << 20, (slots, vocab + 3), dtype=np.int32)  # garbage where nothing is seen
        bits = np.zeros((slots, words * 32), bool)
        bits[:, :vocab] = rng.random((slots, vocab)) < fill
        self.seen = np.zeros((slots, words + 1), np.int32)
        self.seen[:, words] = -559038737
        self.seen[:, :words] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
        self.words = [{int(i): None for i in np.flatnonzero(bits[s])} for s in range(slots)]
        for s in range(slots):
            for i in self.words[s]:
                self.counts[s, i] = self.words[s][i] = int(rng.integers(1, 9))
        self.d_counts, self.d_seen = torch.from_numpy(self.counts).to(DEV), torch.from_numpy(self.seen).to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.history = ssu.TokenHistory(slots, vocab, self.d_counts[:, :vocab], self.d_seen[:, :words], self.status)

    def add(self, slot, tokens, prompt, reset):
        if reset:
            self.words[slot] = {}
        w = self.words[slot]
        for t in tokens:
            if 0 <= t < self.vocab:
                w[t] = (w.get(t, 0) | 1) if prompt else w.get(t, 0) + 2

    def check(self):
        counts, seen = self.d_counts.cpu().numpy(), self.d_seen.cpu().numpy()
        words = (self.vocab + 31) // 32
        bits = np.unpackbits(np.ascontiguousarray(seen[:, :words]).view(np.uint8), axis=1, bitorder="little").astype(bool)
        for s in range(self.slots):
            assert set(np.flatnonzero(bits[s]).tolist()) == set(self.words[s]), s
            at = sorted(self.words[s])
            assert counts[s, at].tolist() == [self.words[s][i] for i in at], s
            assert (counts[s, self.vocab:] == self.counts[s, self.vocab:]).all()
        assert (seen[:, words] == -559038737).all()


@pytest.mark.parametrize("vocab", [1, 31, 32, 33, 1000, 100003])
@pytest.mark.parametrize("prompt,reset", [(True, True), (True, False), (False, False), (False, True)])
def test_count_whole_rows(vocab, prompt, reset):
    rng = np.random.default_rng(vocab)
    p = Pages(9, vocab, vocab, 0.1)
    ids = [3, 0, 8, -2, 9, 1, 5, 2]
    lens = [1, 4, 0, 3, 2, 700, 1024, 5000]
    cu = np.concatenate([[0], np.cumsum(lens)])
    tokens = (vocab * rng.random(cu[-1]) ** 3).astype(np.int32)
    c = ssu.make_count(p.history, i32(ids), i32(tokens), cu_seqlens=i32(cu), prompt=prompt, reset=reset)
    for _ in range(2):
        ssu.count(c)
        for j, s in enumerate(ids):
            if 1 <= s < 9:
                p.add(s, tokens[cu[j]:cu[j + 1]].tolist(), prompt, reset)
    p.check()
    assert int(p.status) == 0


@pytest.mark.parametrize("T", [1, 5, 64, 65, 200])
@pytest.mark.parametrize("num", [True, False])
def test_count_accepted_tokens(T, num):
    rng = np.random.default_rng(T)
    p = Pages(12, 500, T, 0.2)
    ids = rng.permutation(np.arange(1, 12))[:7].tolist()
    lens = rng.integers(0, T + 1, 7).tolist() if num else [T] * 7
    tokens = rng.integers(0, 500, (7, T)).astype(np.int32)
    tokens[:, 0] = 7  # the same token in all entries
    c = ssu.make_count(p.history, i32(ids), i32(tokens), num_tokens=i32(lens) if num else None)
    ssu.count(c)
    for j, s in enumerate(ids):
        p.add(s, tokens[j, :lens[j]].tolist(), False, False)
    p.check()
    assert int(p.status) == 0


def test_count_flags():
    p = Pages(5, 100, 1, 0.3)
    ssu.count(ssu.make_count(p.history, i32([1, 2]), i32([[5, -1], [100, 7]])))
    p.add(1, [5], False, False)
    p.add(2, [7], False, False)
    p.check()
    assert int(p.status) == ssu.SSU_STATUS_BAD_TOKEN
    p.status.zero_()
    ssu.count(ssu.make_count(p.history, i32([1, 2, 3]), i32([[5, 1], [3, 7], [2, 2]]), num_tokens=i32([-1, 1, 3]), reset=True))
    p.add(2, [3], False, True)   # the others are skipped, their pages left as they are
    p.check()
    assert int(p.status) == ssu.SSU_STATUS_BAD_SEQLEN
    for cu in ([0, 2, 1, 3], [-1, 1, 2, 3], [0, 1, 3, 4], [0, 2 ** 31 - 1, -2 ** 31, 3]):
        p.status.zero_()
        q = Pages(5, 100, 1, 0.3)
        ssu.count(ssu.make_count(q.history, i32([1, 2, 3]), i32([1, 2, 3]), cu_seqlens=i32(cu)))
        assert int(q.status) & ssu.SSU_STATUS_BAD_SEQLEN, cu
    ssu.count(ssu.make_count(p.history, i32([]), i32([]).view(0, 1)))
    empty = ssu.make_count(p.history, i32([4]), i32([]), cu_seqlens=i32([0, 0]), prompt=True, reset=True)
    ssu.count(empty)
    p.add(4, [], True, True)
    p.check()


def test_large_tokens_past_4_GiB():
    """Pages so far apart that their offsets pass 32 bits."""
    slots, vocab = 3, 70000
    gap = (1 << 29) + 11  # words
    counts = torch.empty(slots * gap, dtype=torch.int32, device=DEV).as_strided((slots, vocab), (gap, 1))
    seen = torch.empty(slots * gap, dtype=torch.int32, device=DEV).as_strided((slots, (vocab + 31) // 32), (gap, 1))
    h = ssu.TokenHistory(slots, vocab, counts, seen)
    ssu.count(ssu.make_count(h, i32([2]), i32([[69999, 3, 69999]]), reset=True))
    assert counts[2, [3, 69999]].tolist() == [2, 4] and int((seen[2] != 0).sum()) == 2
    x = torch.zeros(1, vocab, device=DEV)
    out = torch.empty_like(x)
    ssu.logits(ssu.make_logits(x, out, 1, 1, history=h, slot_idx=i32([2]), frequency=torch.ones(1, device=DEV), softmax=False))
    assert out[0, [0, 3, 69999]].tolist() == [0.0, -1.0, -2.0]


# ---------------------------------------------------------------------------

class Case:
    """Random logits of a step with everything that may change them, on the host."""

    def __init__(self, seed, b, T, vocab, lens=None, it="f32", history=True, drafts=True, bias=0, mask=None, fill=0.02, temperature=None,
                 pages=None, stride=0):
        g = torch.Generator()
        g.manual_seed(seed)
        self.b, self.T, self.vocab = b, T, vocab
        self.lens = [T] * b if lens is None else lens
        self.varlen = lens is not None
        self.cu = [sum(self.lens[:i]) for i in range(b + 1)]
        self.rows = self.cu[-1] + 1 if self.varlen else b * T
        wide = 3.0 * torch.randn(self.rows, vocab + stride, generator=g)
        self.wide = wide.to(TYPES[it])
        self.logits = self.wide[:, :vocab]
        self.pages = (pages or Pages(b + 2, vocab, seed, fill)) if history else None
        self.ids = (1 + torch.randperm(b + 1, generator=g)[:b]).tolist()
        if b > 2:
            self.ids[1] = 0  # an entry without a history
        self.tokens = (vocab * torch.rand(self.rows, generator=g) ** 2).int() if drafts and history else None
        rnd = lambda lo, hi: lo + (hi - lo) * torch.rand(b, generator=g)  # noqa: E731
        self.rep, self.freq, self.pres = rnd(0.8, 1.4), rnd(-0.1, 0.6), rnd(-0.3, 0.9)
        self.temperature = rnd(0.3, 1.5) if temperature is None else torch.tensor(temperature)
        self.bias = [[(int(vocab * torch.rand(1, generator=g) ** 2), float(4 * torch.randn(1, generator=g))) for _ in range(bias)] for _ in range(b)]
        self.mask = None if mask is None else torch.rand(self.rows, vocab, generator=g) < mask

    def words(self):
        w = (self.vocab + 31) // 32
        bits = np.ones((self.rows, w * 32), bool)  # (bits behind the vocabulary are nobody's)
        bits[:, :self.vocab] = self.mask.numpy()
        return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)

    def x(self):
        """x of every row of the entries, rounded to 32 bits operation by operation."""
        out = np.full((self.rows, self.vocab), np.nan, np.float32)
        for b in range(self.b):
            slot = self.ids[b]
            held = self.pages.words[slot] if self.pages and 1 <= slot < self.pages.slots else {}
            rep, freq, pres = (np.float32(v[b]) for v in (self.rep, self.freq, self.pres))
            for t in range(self.lens[b]):
                row = self.cu[b] + t
                x = self.logits[row].float().numpy().copy()
                for i, v in dict(self.bias[b]).items():
                    x[i] = np.float32(x[i]) + np.float32(v)
                n = {i: w >> 1 for i, w in held.items()}
                if self.tokens is not None:
                    for i in self.tokens[self.cu[b] + 1:row + 1].tolist():
                        if 0 <= i < self.vocab:
                            n[i] = n.get(i, 0) + 1
                if self.pages:
                    for i, k in n.items():
                        v = x[i] / rep if x[i] > 0 else x[i] * rep
                        x[i] = v - (freq * np.float32(k) + (pres if k > 0 else np.float32(0)))
                x[np.isnan(x)] = -np.inf
                if self.mask is not None:
                    x[~self.mask[row].numpy()] = -np.inf
                out[row] = x
        return out

    def call(self, ot="f32", softmax=True, in_place=False, stream=None, keep=None):
        wide = self.wide.to(DEV)
        logits = wide[:, :self.vocab]
        if in_place:
            out_wide, out = wide, logits
        else:
            out_wide = torch.full((self.rows, self.vocab + 5), -7.0, dtype=TYPES[ot], device=DEV)
            out = out_wide[:, :self.vocab]
        kw = {}
        if self.pages:
            kw.update(history=self.pages.history, slot_idx=i32(self.ids), repetition=self.rep.to(DEV), frequency=self.freq.to(DEV),
                      presence=self.pres.to(DEV), tokens=None if self.tokens is None else self.tokens.to(DEV))
        if any(self.bias):
            flat = [p for b in self.bias for p in b]
            kw.update(bias_offsets=i32([sum(len(b) for b in self.bias[:i]) for i in range(self.b + 1)]),
                      bias_tokens=i32([p[0] for p in flat]), bias_values=torch.tensor([p[1] for p in flat], device=DEV))
        if self.mask is not None:
            kw.update(mask=self.words())
        size = ssu.logits_workspace_size(self.b, self.T, self.vocab)
        ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        args = ssu.make_logits(logits, out, self.b, self.T, cu_seqlens=i32(self.cu) if self.varlen else None,
                               temperature=self.temperature.to(DEV), softmax=softmax, workspace=ws[:size], status=status, **kw)
        ssu.logits(args, stream=stream)
        if keep is not None:
            keep.update(args=args, out=out, status=status, logits=logits)
        torch.cuda.synchronize()
        assert bool((ws[size:] == 0xA5).all())
        if not in_place:
            assert bool((out_wide[:, self.vocab:] == -7).all())
            owned = sum(self.lens)
            assert bool((out_wide[owned:] == -7).all()), "a row that nobody owns"
        return out.cpu(), int(status)


# p = exp2((x - m) k) / sum: k = log2(e) / temperature is off by two half steps, x - m by one, the product by one, all of
# the exponent, 4 x 2^-24 |x - m| / temperature of p; exp2 itself by 2 half steps, and the sum's n additions, each thread's
# and the joins, n / 1024 + 64 at most on any value's way (a thread adds n / 256 values in turn), with a few roundings again
# for each join's exponent, as large as the spread; 1 / sum and the last product 2.  |x - m| / temperature matters up to
# 104: p is 0 in fp32 below (an absolute 2^-126 is allowed, the smallest normal number).
def check_probs(got, x, temperature, ot):
    got = got.double().numpy()
    x = x.astype(np.float64)
    x = np.minimum(x, np.finfo(np.float32).max)
    for r in range(x.shape[0]):
        t = float(temperature[r])
        if not t > 0:
            want = np.zeros(x.shape[1])
            if x[r].max() > -np.inf:
                want[int(np.flatnonzero(x[r] == x[r].max())[0])] = 1.0
            assert np.array_equal(got[r], want), r
            continue
        if x[r].max() == -np.inf:
            assert not got[r].any(), r
            continue
        d = (x[r] - x[r].max()) / t
        p = np.exp(d)
        p /= p.sum()
        rel = (4 * np.abs(np.maximum(d, -110)) * 2 + 16 + 64 + x.shape[1] / 256) * 2.0 ** -24
        half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[ot]
        least = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}[ot]  # half of fp16's smallest step
        off = np.abs(got[r] - p)
        allowed = (rel + half) * p + least
        assert (off <= allowed).all(), (r, float((off / allowed).max()))
        assert abs(got[r].sum() - 1.0) <= half + 200 * 2.0 ** -24 + x.shape[1] * least


def check(c, ot="f32", **kw):
    out, status = c.call(ot, **kw)
    x = c.x()
    rows = sum(c.lens)
    temperature = np.concatenate([[float(c.temperature[b])] * c.lens[b] for b in range(c.b)] + [[]])
    empty = any(x[r].max() == -np.inf for r in range(rows))
    assert status == (ssu.SSU_STATUS_EMPTY_ROW if empty and kw.get("softmax", True) else 0)
    if kw.get("softmax", True):
        check_probs(out[:rows], x[:rows], temperature, ot)
    else:
        t = np.where(temperature > 0, temperature, 1.0).astype(np.float32)[:, None]
        want = torch.from_numpy((x[:rows] / t).astype(np.float32)).to(TYPES[ot])
        assert torch.equal(out[:rows], want)  # the same operations, the same bits
    return out


VOCABS = [1, 7, 8, 31, 33, 255, 2047, 2048, 2049, 4100, 8191, 32000, 65537, 100003]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("it,ot", [("f32", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
def test_probabilities(vocab, it, ot):
    c = Case(vocab, 3, 2, vocab, it=it, bias=5, mask=0.7, stride=vocab % 3)
    check(c, ot)


@pytest.mark.parametrize("vocab", [1, 33, 2049, 32000])
@pytest.mark.parametrize("it,ot", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_logits_out(vocab, it, ot):
    c = Case(3 * vocab, 3, 2, vocab, it=it, bias=9, mask=0.6, temperature=[0.7, 0.0, 1.3])
    check(c, ot, softmax=False)


@pytest.mark.parametrize("b,T,lens", [(1, 1, None), (2, 64, None), (5, 7, [7, 0, 3, 1, 5]), (300, 1, None), (40, 8, [8] * 20 + [5] * 20)])
@pytest.mark.parametrize("fill", [0.0, 0.05, 0.9])
def test_rows_and_histories(b, T, lens, fill):
    check(Case(b + T, b, T, 3001, lens=lens, bias=3, fill=fill))
    check(Case(b + T, b, T, 3001, lens=lens, it="bf16", fill=fill), "bf16")


# many rows, and rows whose whole vocabulary is in the history: the forms that a launch may take for them
@pytest.mark.parametrize("rows,vocab,it,fill", [(300, 20000, "bf16", 0.03), (260, 70001, "f32", 0.01), (260, 40000, "f16", 1.0),
                                                (4, 131072, "bf16", 1.0), (2, 262147, "f32", 0.3), (200, 131072, "bf16", 0.2)])
def test_large_calls(rows, vocab, it, fill):
    pages = Pages(6, vocab, rows, fill)
    c = Case(rows, rows, 1, vocab, it=it, bias=2, pages=pages)
    c.ids = [1 + i % 5 for i in range(rows)]   # histories may be read by more than one entry
    keep = [0, 1, 5, rows - 2, rows - 1] if rows > 5 else list(range(rows))
    out, status = c.call("f32")
    x = np.concatenate([_one_row(c, r) for r in keep])
    check_probs(out[keep], x, [float(c.temperature[r]) for r in keep], "f32")
    assert status == 0
    assert float((out.double().sum(1) - 1).abs().max()) < 1e-4


def _one_row(c, r):
    one = Case.__new__(Case)
    one.__dict__.update(c.__dict__)
    one.b, one.T, one.lens, one.cu, one.rows, one.varlen = 1, 1, [1], [0, 1], 1, False
    one.logits, one.ids, one.tokens, one.bias = c.logits[r:r + 1], [c.ids[r]], None, [c.bias[r]]
    one.rep, one.freq, one.pres = c.rep[r:r + 1], c.freq[r:r + 1], c.pres[r:r + 1]
    one.mask = None if c.mask is None else c.mask[r:r + 1]
    return one.x()


def test_without_anything():
    c = Case(1, 4, 2, 5000, history=False)
    check(c)
    check(c, softmax=False)


def test_in_place():
    for it in ("f32", "bf16"):
        c = Case(2, 6, 3, 5001, it=it, bias=4, mask=0.5, temperature=[1.0, 0.5, 0.0, 2.0, 0.9, 1.1])
        assert torch.equal(c.call(it)[0][:18], c.call(it, in_place=True)[0][:18])
        assert torch.equal(c.call(it, softmax=False)[0][:18], c.call(it, softmax=False, in_place=True)[0][:18])


def test_rows_that_a_mask_leaves_nothing_of():
    c = Case(3, 4, 2, 3001, mask=0.5)
    c.mask[2] = False
    c.mask[5] = False
    c.mask[5, 2999] = True   # a single token
    c.temperature[1] = 0.0   # (row 2 is a greedy entry's)
    out = check(c)
    assert not out[2].any() and float(out[5, 2999]) == 1.0


def test_infinities_and_nan():
    c = Case(4, 4, 1, 3001, history=False, mask=0.9)
    inf, nan = float("inf"), float("nan")
    c.wide[0, 5] = c.wide[0, 700] = inf
    c.mask[0, 5] = c.mask[0, 700] = True
    c.wide[1, :] = -inf
    c.wide[1, 17] = nan
    c.mask[1, 17] = True
    c.wide[2, 3] = nan
    c.wide[2, 4] = -inf
    c.wide[3, ::2] = torch.finfo(torch.float32).min   # a mask's lowest value is a value like others
    c.wide[3, 1::2] = nan
    out = check(c)
    assert out[0, 5] == 0.5 and out[0, 700] == 0.5 and not out[1].any() and out[2, 3] == 0.0
    hidden = Case(4, 4, 1, 3001, history=False, mask=0.9)
    seen = hidden.call()[0]
    hidden.wide[~hidden.mask] = nan
    assert torch.equal(hidden.call()[0], seen)
    hidden.wide[~hidden.mask] = inf
    assert torch.equal(hidden.call()[0], seen)


def test_temperatures():
    inf, nan = float("inf"), float("nan")
    c = Case(5, 8, 1, 4099, it="bf16", temperature=[0.0, -1.0, nan, 1e-30, 1e-45, 1e30, 0.01, 1.0])
    c.wide[3, 100] = c.wide[3].max() + 1   # one largest value
    c.wide[4, 100] = c.wide[4].max() + 1
    out = check(c)
    c.temperature[:] = inf
    out = c.call()[0]
    assert float((out - 1 / 4099).abs().max()) < 1e-9


def test_greedy_ties_go_to_the_lowest():
    c = Case(6, 3, 1, 9000, history=False, temperature=[0.0, 0.0, 0.0])
    c.wide[:] = -1.0
    c.wide[0, [8999, 4097, 63]] = 2.0
    c.wide[2, [8998, 4096]] = 2.0
    out = check(c)
    assert [int(out[r].argmax()) for r in range(3)] == [63, 0, 4096]


def test_biases_that_come_twice_and_lists_of_many():
    c = Case(7, 3, 2, 5000, mask=0.9)
    c.bias = [[(10, 1.0), (4999, -2.0), (10, 3.0)], [], [((i * 7) % 5000, float(i % 5)) for i in range(6000)]]
    check(c)
    check(c, softmax=False)


def test_drafts_count_up_to_their_row():
    c = Case(8, 2, 4, 1000)
    c.tokens[:] = torch.tensor([5, 9, 9, 9, 3, 3, 1000, -4], dtype=torch.int32)  # (two of them no tokens)
    check(c)
    check(c, softmax=False)


def test_flags():
    c = Case(9, 3, 2, 300, lens=[2, 1, 2], bias=2)
    for cu, kept in (([0, 2, 3, 7], (0, 3)), ([0, 3, 3, 5], (3, 5)), ([0, 2, 1, 3], (0, 2)), ([-1, 2, 3, 5], (2, 5))):
        wide = c.wide.to(DEV)
        out = torch.full((c.rows, 300), -7.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = torch.empty(ssu.logits_workspace_size(3, 2, 300), dtype=torch.uint8, device=DEV)
        ssu.logits(ssu.make_logits(wide, out, 3, 2, cu_seqlens=i32(cu), workspace=ws, status=status))
        assert int(status) == ssu.SSU_STATUS_BAD_SEQLEN, cu
        assert bool((out[kept[0]:kept[1]] != -7).all()), cu
    x = torch.zeros(2, 64, device=DEV)
    out = torch.empty_like(x)
    ws = torch.empty(64, dtype=torch.uint8, device=DEV)
    for off, toks, bit in (([0, 1, 3], [1, 2], ssu.SSU_STATUS_BAD_BIAS), ([0, 2, 1], [1, 2], ssu.SSU_STATUS_BAD_BIAS),
                           ([-1, 1, 2], [1, 2], ssu.SSU_STATUS_BAD_BIAS), ([0, 1, 2], [64, 2], ssu.SSU_STATUS_BAD_BIAS),
                           ([0, 1, 2], [3, -2], ssu.SSU_STATUS_BAD_BIAS), ([0, 1, 2], [3, 2], 0)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ssu.logits(ssu.make_logits(x, out, 2, 1, bias_offsets=i32(off), bias_tokens=i32(toks), bias_values=torch.ones(2, device=DEV),
                                   workspace=ws, status=status))
        assert int(status) == bit, (off, toks)


def test_one_mask_for_all_rows():
    c = Case(10, 3, 2, 1000, mask=0.5)
    c.mask[:] = c.mask[0].clone()
    want = c.call()[0]
    whole = c.words
    c.words = lambda: whole()[:1].expand(6, -1)
    assert torch.equal(c.call()[0], want)


def test_rows_past_4_GiB():
    vocab, rows = 1 << 20, 1100  # 4.3 GiB of f32
    x = torch.zeros(rows, vocab, device=DEV)
    x[-1, 5] = 20.0
    x[-2, vocab - 1] = 20.0
    ws = torch.empty(ssu.logits_workspace_size(rows, 1, vocab), dtype=torch.uint8, device=DEV)
    ssu.logits(ssu.make_logits(x, x, rows, 1, workspace=ws))
    e = math.exp(20.0)
    for r, i in ((-1, 5), (-2, vocab - 1)):
        assert abs(float(x[r, i]) - e / (e + vocab - 1)) < 1e-5 and abs(float(x[r, 7]) * (e + vocab - 1) - 1) < 1e-4
    assert abs(float(x[0, 0]) * vocab - 1) < 1e-5


def test_the_same_call_again_gives_the_same_bits():
    c = Case(11, 64, 4, 30000, it="bf16", bias=20, mask=0.5)
    assert torch.equal(c.call()[0], c.call()[0])


def test_front_end_refusals():
    x = torch.zeros(4, 100, device=DEV)
    ws = torch.empty(4096, dtype=torch.uint8, device=DEV)
    for kw in (dict(out=x.double()), dict(out=x[:, :99]), dict(out=x.cpu()), dict(logits=x.t().contiguous().t()), dict(batch=5),
               dict(logits=x[:1].expand(4, -1)), dict(temperature=torch.ones(3, device=DEV)), dict(temperature=torch.ones(4)),
               dict(mask=torch.zeros(4, 3, dtype=torch.int32, device=DEV)), dict(mask=torch.zeros(4, 4, device=DEV)),
               dict(tokens=i32([1, 2])), dict(history=Pages(3, 100, 0).history), dict(bias_offsets=i32([0, 1])),
               dict(cu_seqlens=i32([0, 1]))):
        base = dict(logits=x, out=torch.empty_like(x), batch=4, max_seqlen=1, workspace=ws)
        base.update(kw)
        with pytest.raises(ValueError):
            ssu.make_logits(**base)
    with pytest.raises(ssu.SsuError) as e:
        ssu.logits(ssu.make_logits(x, torch.empty_like(x), 4, 1))
    assert e.value.code == ssu.SSU_ERR_WORKSPACE
    with pytest.raises(ssu.SsuError):
        ssu.logits(ssu.make_logits(x, torch.empty_like(x), 4, 1, temperature=torch.ones(4, device=DEV), workspace=ws,
                                   history=Pages(3, 99, 0).history, slot_idx=i32([1, 1, 2, 2])))
