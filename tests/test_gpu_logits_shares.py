"""Rows of ssu_logits whose mass lies on a few values, at the borders of what a
thread, a workgroup and a launch take of a row: none of them may be lost; and
calls so large that their outputs are stored past the caches, beside the special
tokens' own stores."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests.test_gpu_logits import Case, Pages, check_probs


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def part(c, lo, hi):
    """Entries lo .. hi - 1 of a case, as a case."""
    o = Case.__new__(Case)
    o.__dict__.update(c.__dict__)
    rows = slice(c.cu[lo], c.cu[hi])
    o.b, o.lens, o.ids, o.bias = hi - lo, c.lens[lo:hi], c.ids[lo:hi], c.bias[lo:hi]
    o.cu, o.rows = [v - c.cu[lo] for v in c.cu[lo:hi + 1]], c.cu[hi] - c.cu[lo]
    o.wide, o.logits = c.wide[rows], c.logits[rows]
    o.tokens = None if c.tokens is None else c.tokens[rows]
    o.mask = None if c.mask is None else c.mask[rows]
    o.temperature, o.rep, o.freq, o.pres = (v[lo:hi] for v in (c.temperature, c.rep, c.freq, c.pres))
    return o


# An exponent is off by 4 half steps of its size (twice that with the sum's), the sum by a half step for each addition on a
# value's way (row form: a thread adds vocab / 1024 values and as many special ones, then 22 joins of 3 roundings; pieces: 8
# and 8, 10 + 6 joins and a join for every 256 pieces: fewer), exponentials, division and product by 16.
def limit(vocab, d):
    return (8 * np.abs(d) + 16 + vocab / 1024 + 16 + 22 * 3) * 2.0 ** -24


# rows up to as many as CUs, more, and rows of pieces (few of long ones, or longer than one workgroup takes)
@pytest.mark.parametrize("rows,vocab,it", [(64, 65537, "bf16"), (60, 100003, "f32"), (300, 65537, "bf16"), (300, 100003, "f32"),
                                           (70, 131071, "f16"), (1, 65537, "f32"), (2, 100003, "bf16"), (3, 200003, "f32"),
                                           (5, 16391, "f32"), (300, 16391, "f16")])
def test_no_value_is_lost(rows, vocab, it):
    whole = vocab // 8 * 8
    borders = [0, 7, 8, 511, 512, 2047, 2048, 8191, 8192, 4 * 8192, 8 * 8192 - 1, 8 * 8192, whole - 8, whole - 1, whole, vocab - 1]
    borders = sorted({i for i in borders if 0 <= i < vocab})
    c = Case(rows + vocab, rows, 1, vocab, it=it, temperature=[1.0] * rows, pages=Pages(3, vocab, 2, 0.002))
    c.ids = [1 + r % 2 for r in range(rows)]
    c.wide[:] = -60.0                    # e^-60 of all others together: less than 2^-60
    g = torch.Generator()
    g.manual_seed(vocab)
    held = sorted(c.pages.words[1])[::29][:6] + [min(c.pages.words[2])]
    for r in range(rows):
        at = [i for k, i in enumerate(borders) if (k + r) % 3] + [held[r % len(held)]]
        c.wide[r, at] = torch.rand(len(at), generator=g).to(c.wide.dtype)
    out, status = c.call("f32")
    assert status == 0
    look = list(range(rows)) if rows < 20 else list(range(12)) + [rows // 2, rows - 2, rows - 1]
    for r in look:
        x = part(c, r, r + 1).x()[0].astype(np.float64)
        p = np.exp(x - x.max())
        p /= p.sum()
        off, big = np.abs(out[r].double().numpy() - p), p > 1e-3
        assert 8 <= big.sum() < 32
        assert (off[big] <= limit(vocab, (x - x.max())[big]) * p[big]).all(), (r, np.flatnonzero(big)[(off / p)[big].argmax()])


# rows x vocab x (in + out) of 256 MiB and more against the same rows in calls of less; both of more rows than CUs
@pytest.mark.parametrize("b,T,half,vocab,it,ot", [(80, 8, 40, 131071, "bf16", "bf16"), (66, 8, 33, 100003, "f32", "f32")])
def test_outputs_stored_past_the_caches(b, T, half, vocab, it, ot):
    size = {"bf16": 2, "f32": 4}
    each = vocab * (size[it] + size[ot])
    assert half * T > 256 and half * T * each < 256 << 20 <= b * T * each
    c = Case(b, b, T, vocab, it=it, bias=8, mask=0.6, fill=0.006)
    c.temperature[5::8] = 0.0
    out, status = c.call(ot)
    halves = [part(c, 0, half), part(c, half, b)]
    for k, o in enumerate(halves):
        assert torch.equal(out[k * half * T:(k * half + o.b) * T], o.call(ot)[0])
    assert torch.equal(c.call(ot, in_place=True)[0], out)
    for e in (0, 1, 5, 30, b - 1):
        o = part(c, e, e + 1)
        check_probs(out[c.cu[e]:c.cu[e + 1]], o.x(), [float(o.temperature[0])] * T, ot)
    assert status == 0
