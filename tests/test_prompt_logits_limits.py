"""What token histories and logits refuse before any launch (CPU;
the pointers are never dereferenced)."""
import pytest
import torch  # (before the library, which then shares its HIP runtime)

import speculative_replay_state_amd as ssu
from speculative_replay_state_amd import sampling
from tests.test_prompt_logits_abi import FAKE, UNSUPPORTED, _count, _history, _refused


@pytest.mark.parametrize("kw", [dict(num_tokens=None, cu_seqlens=FAKE), dict(batch=1, max_seqlen=4),
                                dict(batch=1, max_seqlen=2 ** 31 - 1, num_tokens=None)])
@pytest.mark.parametrize("rows", [2 ** 30 + 1, 2 ** 31 - 1])
def test_counts_of_more_rows_than_an_index_steps_over(kw, rows):
    """The kernels step an index of 32 bits by 4096 up to an entry's last token."""
    kw = dict(kw, rows=rows, max_seqlen=min(kw.get("max_seqlen", 4), rows))
    _refused(sampling.ssu_history_count(_history(), _count(**kw)), UNSUPPORTED, "2^30")
    _refused(sampling.ssu_history_count(_history(), _count(**{**kw, "batch": 0})), UNSUPPORTED, "2^30")


def test_counts_of_2_to_the_30_rows_are_no_refusal():
    assert sampling.ssu_history_count(_history(), _count(batch=0, rows=2 ** 30)) == ssu.SSU_OK


@pytest.mark.parametrize("kw", [{}, dict(bias_tokens=torch.zeros(2, dtype=torch.int32)), dict(bias_values=torch.zeros(2))])
def test_biases_need_tokens_and_values(kw):
    with pytest.raises(ValueError, match="bias_tokens and bias_values"):
        ssu.make_logits(torch.zeros(1, 64), torch.zeros(1, 64), 1, 1, bias_offsets=torch.zeros(2, dtype=torch.int32), **kw)
