"""The README's layer example runs as printed: its last token over the 4-bit cache is the
prompt attention's last row up to what 4 bits keep."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_layer_example():
    text = open(os.path.join(ROOT, "README.md")).read()
    block = re.findall(r"```python\n(.*?)```", text, flags=re.S)[1]
    torch.manual_seed(0)
    env = {}
    exec(compile(block, "README.md", "exec"), env)
    assert env["out"].shape == (100, 32, 128) and env["one"].shape == (1, 32, 128)
    far = (env["one"][0].double() - env["out"][-1].double()).norm() / env["out"][-1].double().norm()
    # 4-bit rows: K and V each off by about 7 % of their size (0.3 sigma steps / sqrt(12), on
    # groups whose largest value is about 2.2 sigma)
    assert far < 0.25
