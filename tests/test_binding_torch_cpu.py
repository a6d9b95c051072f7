"""The compiled calls look into tensors of the torch they were built for, and are
not imported beside any other."""
import importlib.util

import pytest
import torch

import chip_fusion_amd as cf         # noqa: F401

_attn = pytest.importorskip("chip_fusion_amd._attn")


def _load(path):
    spec = importlib.util.spec_from_file_location("_attn", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_what_it_was_built_for():
    assert _attn.torch in (None, f"{torch.__version__} {torch.version.git_version}")


@pytest.mark.skipif(_attn.torch is None, reason="built without torch's headers")
@pytest.mark.parametrize("version", [torch.__version__, torch.version.git_version])
def test_another_torch(tmp_path, version):
    """A copy whose text names another torch, as one that was built beside it does."""
    code = open(_attn.__file__, "rb").read()
    assert version.encode() in code
    other = tmp_path / "_attn.so"
    other.write_bytes(code.replace(version.encode(), b"9" * len(version)))
    with pytest.raises(ImportError, match="built for torch"):
        _load(str(other))
    same = tmp_path / "same" / "_attn.so"
    same.parent.mkdir()
    same.write_bytes(code)
    assert _load(str(same)).torch == _attn.torch
