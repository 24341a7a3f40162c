"""What the build makes, and what does without the C++ marshalling module: no
compiler runs here, a stand-in writes empty files."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import quantized_kv_decode_paged_gb300 as qk
from quantized_kv_decode_paged_gb300 import _build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The build's commands, with what they make in a folder of the test's own."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        if any(x in cmd[0] for x in getattr(run, "missing", ())):
            raise FileNotFoundError(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "libdecode_attn.so"))
    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setenv("CXX", "host-compiler")
    run.ran = ran
    return run


def _modules(tmp_path):
    return [f for f in os.listdir(tmp_path) if f.startswith("decode_attn_call")]


def test_library_without_torch(commands, tmp_path, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert _build.build() == _build.LIB_PATH and os.path.exists(_build.LIB_PATH)
    assert not _modules(tmp_path) and _build.up_to_date()


def test_library_without_a_host_compiler(commands, tmp_path):
    commands.missing = ["host-compiler"]
    with pytest.warns(RuntimeWarning, match="host-compiler"):
        _build.build()
    assert os.path.exists(_build.LIB_PATH) and not _modules(tmp_path)
    assert not _build.up_to_date()
    commands.missing = []
    made = len(commands.ran)
    _build.build()  # the module alone
    assert len(commands.ran) == made + 1 and _build.up_to_date()


def test_the_module_is_of_one_interpreter_and_torch(commands, tmp_path, monkeypatch):
    _build.build()
    (name,) = _modules(tmp_path)
    assert torch.__version__.split("+")[0] in name
    assert name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert _build.up_to_date()
    monkeypatch.setattr(_build.importlib.metadata, "version", lambda name: "0.1")
    assert not _build.up_to_date()
    _build.build()
    assert len(_modules(tmp_path)) == 2 and _build.up_to_date()


def test_calls_without_the_module_go_through_python(tmp_path, monkeypatch):
    qk.build()
    monkeypatch.setattr(qk, "_call", None)
    monkeypatch.setattr(_build, "LIB_DIR", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="through Python"):
        with pytest.raises(ValueError, match="CUDA device"):  # what the checks in Python say
            qk.decode_attn_qk_norm_rope(torch.zeros(1, 1, 64), None, None, None)
    with pytest.raises(ValueError, match="CUDA device"):
        qk.decode_attn_qk_norm_rope(torch.zeros(1, 1, 64), None, None, None)
    (tmp_path / os.path.basename(_build.call_path())).write_bytes(b"not a library")
    monkeypatch.setattr(qk, "_call", None)
    with pytest.warns(RuntimeWarning, match="through Python"):
        assert qk._load_call().prefix() is NotImplemented
