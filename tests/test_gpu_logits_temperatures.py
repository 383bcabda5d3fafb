"""Probabilities of ssu_logits at temperatures of 1e36 and more, where values
next to the type's ends matter: exp(x / temperature) / sum as defined."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests.test_gpu_logits import Case

TOP = float(torch.finfo(torch.float32).max)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# whole rows, pieces
@pytest.mark.parametrize("vocab", [3001, 20011])
@pytest.mark.parametrize("temperature", [1e36, 1e37, 1e38, 2e38, TOP, float("inf")])
def test_ends_of_the_type(vocab, temperature):
    c = Case(vocab, 4, 1, vocab, history=False, bias=3, temperature=[temperature] * 4)
    c.wide[0, ::3] = -TOP                     # a mask's lowest value
    c.wide[1] = torch.linspace(-TOP / 2, TOP / 2, vocab) * 1.5
    c.wide[2, ::2] = TOP
    c.wide[2, 1::4] = -TOP                    # a difference that is no finite number
    c.wide[3, [0, vocab - 1]] = float("inf")  # counts as the largest finite value
    c.wide[3, 5::7] = -float("inf")           # left out
    out, status = c.call("f32")
    x = np.minimum(c.x().astype(np.float64), TOP)
    with np.errstate(invalid="ignore"):
        y = np.where(np.isinf(x), -np.inf, x / temperature)
    d = y - y.max(axis=1, keepdims=True)
    p = np.exp(d)
    p /= p.sum(axis=1, keepdims=True)
    # As for other temperatures: 8 half steps of the exponent, 16 of roundings of the result, 64 of joins, the sum's
    # additions; and the slope is a multiple of 2^-149 at least, off by 2^-150, of differences of up to 2^129: 2^-21 of p.
    allowed = ((8 * np.abs(np.maximum(d, -110)) + 16 + 64 + vocab / 256) * 2.0 ** -24 + 2.0 ** -21) * p + 2.0 ** -126
    off = np.abs(out.double().numpy() - p)
    assert status == 0
    assert (off <= allowed).all(), float((off / allowed).max())
