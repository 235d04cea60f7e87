"""The README's Python examples, run in their order in one namespace."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_examples_run():
    import __graft_entry__ as g
    g.build()
    import torch
    from paged_kv_decode_kf_gb300 import kf
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) >= 3
    space = {}
    for block in blocks:
        exec(compile(block, "README.md", "exec"), space)
        torch.cuda.synchronize()
        assert kf.kf_get_device_error() == 0, block
