"""The native binding of the experts' operators without a GPU: it is built from
these sources, and it leaves whatever is not on the GPU to the Python code."""
import os
import subprocess
import sys

import pytest
import torch

from moe_token_re_amd import _lib, build

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")


def test_binding_is_of_these_sources():
    assert _lib.binding().source_hash == build.source_hash() == _lib.library_source_hash()


def test_binding_leaves_cpu_tensors_alone():
    b = _lib.binding()
    x, p, s = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 1, 2, dtype=torch.uint8)
    assert b.quantize(x) is None and b.dequantize(p, s, torch.float32) is None
    assert b.grouped_mm(p, s, p[None], s[None], torch.tensor([2]), False, None, 1, torch.float32) is None
    assert b.few_tokens(x, x, x, x, 1, True, None, None, None, None) is None
    for call in (b.quantize, b.dequantize, b.grouped_mm, b.few_tokens):
        assert call() is None and call(None) is None and call(1, 2, 3) is None


def test_binding_loads_torch_by_itself():
    code = "from moe_token_re_amd import _lib; _lib.binding()"
    root = os.path.dirname(os.path.dirname(os.path.abspath(_lib.__file__)))
    assert subprocess.run([sys.executable, "-c", code], cwd=root, timeout=120).returncode == 0
