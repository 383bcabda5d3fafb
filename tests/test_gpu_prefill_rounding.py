"""bf16 outputs of ssu_prefill are its fp32 ones, rounded once: nothing on the
way to them has fewer bits."""
import pytest
import torch

from tests import prompt_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests.test_gpu_prefill import call, gen, want


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# a workgroup a head, two heads a workgroup (more than 256 of them), heads of a group that are no even number, segments
@pytest.mark.parametrize("lens,H,G", [([1, 17, 64, 65], 4, 2), ([200, 129], 3, 3), ([1500, 700], 4, 1),
                                      ([5] * 70, 8, 2), ([66, 128, 0, 257] + [3] * 96, 5, 1), ([1500, 3, 901] + [2] * 127, 4, 2)])
@pytest.mark.parametrize("gate", [True, False])
def test_bf16_outputs_are_the_fp32_ones_rounded_once(lens, H, G, gate):
    g = gen(sum(lens) + H)
    a = R.inputs(g, sum(lens), H, G)
    a["z"] *= 4  # (gates far on both sides)
    init = 0.3 * torch.randn(len(lens), H, 64, 128, generator=g)
    wide, S = call(a, lens, "f32", init=init, gate=gate)
    out, T = call(a, lens, "bf16", init=init, gate=gate)
    assert torch.equal(out, wide.bfloat16()) and torch.equal(T, S)


# A value that is off by d from the exact one rounds to another neighbour with the probability |d| / step, and is then off
# by a step, at most 2^-7 of it.  The sum of the squares of what differs is then |d| step over all values, at most the norm
# of d times the norm of the steps (Cauchy and Schwarz): with d of 8 x 2^-24 of the norm (what fp32 results are held to)
# 2^-21 x 2^-7 of the norm's square, 2^-14 of the norm.  (A readout of operands of 16 bits ended at 1.0e-4, 1.6 times that.)
def test_bf16_outputs_seldom_round_the_other_way():
    g = gen(31)
    lens = [17 - i % 9 for i in range(15)]
    a = R.inputs(g, sum(lens), 64, 8)
    init = 0.3 * torch.randn(len(lens), 64, 64, 128, generator=g)
    out, _ = call(a, lens, "bf16", init=init, gate=True)
    y = want(a, lens, init, True)[0]
    exact = y.bfloat16().double()
    off = float((out.double() - exact).norm() / exact.norm())
    print("off the rounded exact ones by %.3g of the norm" % off, flush=True)
    assert off <= 2.0 ** -14
