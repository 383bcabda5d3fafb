"""The usage example of prompts, logits and verification in README.md runs as
written on the GPU."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_prompt_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    blocks = re.findall(r"```python3\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), flags=re.S)
    assert len(blocks) == 1
    print("README prompt example", flush=True)
    names = {}
    exec(compile(blocks[0], "README.md", "exec"), names)
    assert bool(torch.isfinite(names["out"].float()).all()) and bool(torch.isfinite(names["states"]).all())
    assert float((names["probs"].double().sum(1) - 1).abs().max()) < 1e-5
