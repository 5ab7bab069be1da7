"""The library and the experts' operators without the torch binding: the C
library builds without torch, and where the binding is missing or of other
sources the Python code makes the calls by ctypes, with one warning."""
import os
import sys
import types
import warnings

import pytest
import torch

import moe_token_re_amd
from moe_token_re_amd import _lib, build, experts

needs_library = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")


def test_library_builds_without_torch(monkeypatch):
    """Commands are noted, not run."""
    ran = []
    monkeypatch.setattr(build, "_run", lambda cmd, verbose: ran.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: ran.append([a, b]))
    monkeypatch.setitem(sys.modules, "torch", None)  # an import of it fails
    assert build.build_library() == build.LIB_PATH
    assert [build.LIB_PATH + ".tmp", build.LIB_PATH] in ran
    assert not any("torch" in os.path.basename(word) for cmd in ran for word in cmd)
    assert len(build.build_all()) == 2


def _without(monkeypatch, binding):
    """Nothing loaded yet, and `binding` (None: an ImportError) in the module's place."""
    for name in ("_binding", "_plain_calls"):
        monkeypatch.setattr(_lib, name, None)
    monkeypatch.delattr(moe_token_re_amd, "_mrr_torch", raising=False)
    monkeypatch.setitem(sys.modules, "moe_token_re_amd._mrr_torch", binding)


@needs_library
@pytest.mark.parametrize("binding", [None, types.SimpleNamespace(source_hash="0" * 16)])
def test_calls_go_by_ctypes(monkeypatch, binding):
    _without(monkeypatch, binding)
    with pytest.warns(RuntimeWarning, match="binding|_mrr_torch"):
        with pytest.raises(ValueError, match="GPU"):  # the Python code's own check, not a failure to load
            experts.mx_quantize(torch.zeros(2, 64))
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # once is enough
        with pytest.raises(ValueError, match="GPU"):
            experts.mx_quantize(torch.zeros(2, 64))
    with pytest.raises(RuntimeError):
        _lib.binding()


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_results_are_the_same(monkeypatch):
    dev = torch.device("cuda:0")
    g = torch.Generator(dev).manual_seed(5)
    x = torch.randn(6, 96, device=dev, generator=g).to(torch.bfloat16)
    wide = torch.randn(3, 64, 96, device=dev, generator=g).to(torch.bfloat16)
    down = torch.randn(3, 96, 32, device=dev, generator=g).to(torch.bfloat16)
    logits = torch.randn(6, 3, device=dev, generator=g)
    num = torch.tensor([1, 2, 3], device=dev)

    def calls():
        rows, w = experts.mx_quantize(x), experts.mx_quantize(wide)
        return (*(t.view(torch.uint8) for t in rows), experts.mx_dequantize(*rows),
                experts.mx_grouped_mm(*rows, *w, num, gated=True),
                experts.moe_few_tokens(x, wide, down, router_logits=logits, top_k=2))

    fast = calls()
    assert _lib.plain_calls() is _lib.binding()
    _without(monkeypatch, None)
    slow = calls()
    assert _lib.plain_calls() is not None and _lib._binding is None
    assert all(torch.equal(a, b) for a, b in zip(fast, slow))
