"""The extension module that marshals the calls made per token and layer saves
host time and nothing else: the library works without it."""

import os
import subprocess
import sys

import pytest

from post_pruning_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = r'''
import sys, warnings
HOW
import torch
import post_pruning_b200 as pp
from post_pruning_b200 import sgpt as S
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    assert pp.lib().sgpt_abi_version() == 2 and pp.lib() is S._lib
assert S._marshal is None and ["_marshal" in str(w.message) for w in seen] == [True], seen
assert S._lib.sgpt_workspace_bytes(64, 64, 100, S.Params("2:4").to_c()) > 0
f = dict(dtype=torch.bfloat16)
X, q = torch.zeros(4, 64, **f), torch.zeros(4, 64, dtype=torch.int8)
s, t, info = torch.zeros(4), torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
h, off = torch.zeros(4, 2, 64, **f), torch.zeros(2, dtype=torch.int32)
for call in (lambda: pp.quant_tokens(X, q, s, t, info), lambda: pp.quant_tokens_silu(X, X, q, s, t, info),
             lambda: pp.linear_i8(q, s, t, q, torch.ones(4, 2), torch.zeros(4, 4), info),
             lambda: pp.attention(h, h, h, off, h.clone(), info)):
    try:
        call()
    except TypeError:
        continue
    raise AssertionError("CPU tensors were taken")
'''


@pytest.mark.parametrize("how", [
    "sys.modules['post_pruning_b200._marshal'] = None          # as if it were not there",
    "import post_pruning_b200._marshal as m; m.torch_version = '1.0'",
    "import post_pruning_b200._marshal as m; del m.torch_version"])
def test_library_without_the_module(how):
    r = subprocess.run([sys.executable, "-c", WITHOUT.replace("HOW", how)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_module_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        assert not module.exists()                         # nothing of other sources stays if this fails
        module.touch()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    module = tmp_path / "_marshal.so"
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "MARSHAL", str(module))
    monkeypatch.setattr(B.subprocess, "run", run)
    module.touch()
    B._build_marshal()                                     # of a torch that nothing names
    assert len(ran) == 1
    B._build_marshal()
    assert len(ran) == 1                                   # up to date
    (tmp_path / "marshal.torch").write_text("1.0")
    B._build_marshal()
    assert len(ran) == 2


def test_library_is_built_where_the_module_cannot_be(monkeypatch, capsys):
    def fail():
        raise RuntimeError("no C++ compiler here")

    monkeypatch.setattr(B, "_build_marshal", fail)
    assert B.build() == B.LIB
    assert "no C++ compiler here" in capsys.readouterr().err
