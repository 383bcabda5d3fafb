"""Rows of as many pieces as put a border of the pick somewhere: a lane's run of
neighbouring pieces, the 64 lanes, the row kernel's LDS.  The piece is taken
from the source, so that the rows keep their place if it changes."""
import os
import re

import numpy as np
import pytest
import torch

from tests.test_gpu_verify import as_type, reference, run

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "speculative_replay_state_amd", "csrc", "verify_internal.h")).read()
PIECE = int(re.search(r"kVerifyPiece = (\d+);", SOURCE).group(1))
LAST = float(np.nextafter(np.float32(1), np.float32(0)))


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("less", [0, 5])  # whole pieces, the last one cut short
@pytest.mark.parametrize("pieces", [41, 63, 64, 65, 127, 128, 129, 193])
def test_two_launches(pieces, less):
    vocab = pieces * PIECE - less
    rng = np.random.default_rng(pieces + less)
    p = (rng.random((8, vocab)) / vocab).astype(np.float32)
    p[1, :(pieces - 1) * PIECE] = 0.0                  # only the last piece
    p[2, PIECE:] = 0.0                                 # only the first
    p[3] = 0.0
    p[3, PIECE - 1::PIECE] = 0.125                     # the last value of every piece
    p[4] = 0.0
    p[4, ::PIECE] = 0.125                              # the first
    p[5, PIECE:-PIECE] = 0.0                           # the two ends
    uf = np.float32([0.5, 0.7, LAST, 0.999, 0.0, 0.5, LAST, 0.001])
    out, acc, status = run([0] * 8, p, None, [0.0] * 8, uf, 1)
    want, _, bits = reference([0] * 8, p.astype(np.float64), None, [0.0] * 8, uf, np.arange(9), 1, vocab)
    assert status == bits and np.array_equal(out, want) and acc.tolist() == [1] * 8


@pytest.mark.parametrize("pieces,less", [(64, 0), (65, 3), (256, 0), (256, 1), (257, 9)])  # the row kernel holds 256
def test_many_entries_of_two_bytes(pieces, less):
    vocab, n = pieces * PIECE - less, 192
    rng = np.random.default_rng(pieces)
    one = (rng.random((4, vocab)) + 0.001).astype(np.float32)
    one[1, : vocab - PIECE] = 0.0
    one[2, PIECE:] = 0.0
    rows = np.arange(n) % 4
    uf = rng.random(n).astype(np.float32)
    uf[:8] = [0.0, 0.0, LAST, LAST, LAST, LAST, 0.0, 0.0]
    one = as_type(one / one.sum(1, keepdims=True), "bf16")
    print("many entries", pieces, less, flush=True)
    out, acc, status = run([0] * n, one[rows], None, [0.0] * n, uf, 1, dtype="bf16")
    # every entry against the sums of its row, formed once
    sums = np.cumsum(one, axis=1)
    want = [int(np.nonzero((sums[r] > float(u) * sums[r, -1]) & (one[r] > 0))[0][0]) for r, u in zip(rows, uf)]
    assert status == 0 and acc.tolist() == [1] * n and out[:, 0].tolist() == want
