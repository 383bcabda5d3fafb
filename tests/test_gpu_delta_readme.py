"""The usage example of the gated delta rule and verification in README.md runs
as written on the GPU."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_delta_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    blocks = re.findall(r"```py\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), flags=re.S)
    assert len(blocks) == 1
    print("README delta example", flush=True)
    names = {}
    exec(compile(blocks[0], "README.md", "exec"), names)
    assert bool(torch.isfinite(names["out"].float()).all()) and bool(torch.isfinite(names["y"].float()).all())
