"""What the build says where the compiled calls do without torch's headers."""
import importlib.util

import pytest

from chip_fusion_amd import build


@pytest.mark.parametrize("flags", [["-DB2B_TORCH=\"1\""], ["-include", "no_such_header.h"]])
def test_headers_that_do_not_compile(monkeypatch, tmp_path, capfd, flags):
    out = tmp_path / "_attn.so"
    monkeypatch.setattr(build, "PYATTN", str(out))
    monkeypatch.setattr(build, "_torch_flags", lambda: (flags, []))
    assert build.binding() == str(out)
    said = capfd.readouterr().err
    assert "_attn.so is built without torch's headers" in said and "error" in said and "No such file" in said
    assert said.count("\n") == 1 and [f.name for f in tmp_path.iterdir()] == ["_attn.so"]
    spec = importlib.util.spec_from_file_location("_attn", str(out))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.torch is None
