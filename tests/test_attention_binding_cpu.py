"""The compiled calls (_attn.so) are a shortcut: without a compiler for Python's
API, or without the file, the library builds and every call is made in Python."""
import os
import subprocess
import sys

import pytest

import chip_fusion_amd as cf
from chip_fusion_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(cf.__file__)))

CALLS = """
import sys
sys.modules["chip_fusion_amd._attn"] = None          # as if the file were not there
import torch
import chip_fusion_amd as cf
t = lambda *shape: torch.zeros(shape, dtype=torch.float16)
cu, g = torch.tensor([0, 5], dtype=torch.int32), torch.zeros(4)
q, k = t(5, 4, 64), t(5, 2, 64)
for plan, call in [(cf.Attention, lambda p: p.run(q, k, k, cu)),
                   (cf.PrefixAttention, lambda p: p.run(q, k, k, t(5, 3, 2, 64), t(5, 3, 2, 64), torch.zeros(5, dtype=torch.int32))),
                   (cf.LinearAttention, lambda p: p.run(q, k, k, g, cu)),
                   (cf.LinearAttention, lambda p: p.step(q, k, k, g, torch.zeros(5, 4, 64, 64)))]:
    p = plan("f16", 4, 2, 64)
    try:
        call(p)
    except ValueError as e:                          # all there is to say of them
        assert "a device (cuda) tensor is expected" in str(e), e
    else:
        raise AssertionError("host tensors accepted")
    p.close()
print("made in Python")
"""


def test_calls_without_the_compiled_binding():
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "made in Python" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("error", [subprocess.CalledProcessError(1, "g++"), FileNotFoundError("g++")])
def test_build_without_pythons_headers(monkeypatch, tmp_path, capsys, error):
    """What cannot be compiled is left out, with a word about it, and a file of an
    earlier build, which may not fit the library, goes."""
    old = tmp_path / "_attn.so"
    old.write_bytes(b"old")
    monkeypatch.setattr(build, "PYATTN", str(old))

    def fail(*a, **k):
        raise error
    monkeypatch.setattr(build.subprocess, "check_call", fail)
    assert build.binding() is None
    assert not old.exists() and not list(tmp_path.iterdir())
    assert "_attn.so" in capsys.readouterr().err
