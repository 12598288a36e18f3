"""The package without a usable native binding of the paged calls: everything else works, and the paged calls
say what is missing."""
import os
import subprocess
import sys

import pytest

from block_sparse_long_summary_b200 import build as B

REFUSED = """
import importlib.machinery, os
real = importlib.machinery.ExtensionFileLoader.create_module
def create(self, spec):
    if os.path.basename(self.path).startswith("_paged"):
        raise ImportError("undefined symbol (built for another PyTorch)")
    return real(self, spec)
importlib.machinery.ExtensionFileLoader.create_module = create
"""
MISSING = """
import os
real = os.path.exists
os.path.exists = lambda p: not os.path.basename(str(p)).startswith("_paged") and real(p)
"""
REST = """
from block_sparse_long_summary_b200 import cobs
assert cobs.version() > 0 and cobs.workspace_bytes(cobs.Params(B=1, Hq=4, Hkv=1, d=128, T=4096, topk=8, window=512), cobs.COBS_WS_DECODE) > 0
p = cobs.PagedParams(R=1, Hq=4, Hkv=1, d=128, page=64, n_pages=4, max_pages=4, n_tokens=1, max_new=1)
assert cobs.paged_workspace_bytes(p) > 0
assert not hasattr(cobs._paged, "__wrapped__")   # looking the package over does not load the binding
for _ in range(2):
    try:
        cobs.cobs_paged_append(p, None, None, None, None, None)
    except ImportError as e:
        assert "undefined symbol" in str(e) or "not built" in str(e)
    else:
        raise SystemExit("the call went on")
"""


@pytest.mark.parametrize("setup", [REFUSED, MISSING], ids=["refused", "missing"])
def test_only_the_paged_calls_need_the_binding(setup):
    B.build()
    r = subprocess.run([sys.executable, "-c", setup + REST], capture_output=True, text=True, cwd=B.ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


def test_the_binding_is_loaded_once():
    B.build()
    from block_sparse_long_summary_b200 import cobs
    with pytest.raises(TypeError, match="tensor"):
        cobs.cobs_paged_append(cobs.PagedParams(R=1, Hq=4, Hkv=1, d=128, page=64, n_pages=4, max_pages=4, n_tokens=1, max_new=1),
                               None, None, None, None, None)
    assert vars(cobs._paged)["append"] is cobs._paged.append
    with pytest.raises(AttributeError):
        cobs._paged.no_such_call


def test_another_pytorch_gets_a_binding_of_its_own(monkeypatch):
    import torch
    B.build()
    here, made = B.binding_path(), []
    monkeypatch.setattr(B, "_build_binding", lambda: made.append(B.binding_path()))
    monkeypatch.setattr(B, "_compile", lambda *a: pytest.fail("the library does not depend on PyTorch"))
    B.build()
    assert made == []
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert B.binding_path() != here
    B.build()
    assert made == [B.binding_path()]
    from block_sparse_long_summary_b200 import cobs
    with pytest.raises(ImportError, match="0.0.1"):
        cobs._load_binding()


@pytest.mark.parametrize("name", ["R", "Hq", "Hkv", "d", "page", "n_pages", "max_pages", "n_tokens", "max_new", "window", "sinks"])
def test_params_that_do_not_fit_the_struct_are_refused(name):
    import dataclasses

    from block_sparse_long_summary_b200 import cobs
    p = cobs.PagedParams(R=1, Hq=4, Hkv=1, d=128, page=64, n_pages=4, max_pages=4, n_tokens=1, max_new=1, window=8)
    for value in (2 ** 31, 2 ** 32 + 1, 2 ** 32, -2 ** 31 - 1, 2 ** 63):
        with pytest.raises(ValueError, match=name):
            dataclasses.replace(p, **{name: value})
    assert getattr(dataclasses.replace(p, **{name: 2 ** 31 - 1}).c(), name) == 2 ** 31 - 1
    with pytest.raises(TypeError):
        dataclasses.replace(p, **{name: 1.5})
