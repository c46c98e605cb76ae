"""The README's example of a step with drafted tokens runs as printed."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_step_example():
    text = open(os.path.join(ROOT, "README.md")).read()
    block = re.findall(r"```python\n(.*?)```", text, flags=re.S)[2]
    torch.manual_seed(0)
    env = {}
    exec(compile(block, "README.md", "exec"), env)
    assert env["positions"].tolist() == [50, 51, 51, 52] and env["places"].tolist() == [50, 51, 52, 53]
    assert env["mask"].tolist() == [1, 3, 5, 11]
    assert env["out"].shape == (4, 32, 128) and torch.isfinite(env["out"].float()).all()
    kept = int(env["kept"][0])
    new = env["new"].tolist()
    assert 0 <= kept <= 2 and all(0 <= x < 32000 for x in new[:kept + 1]) and new[kept + 1:] == [-1] * (3 - kept)
