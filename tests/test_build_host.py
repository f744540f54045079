"""When the Python side's compiled binding is built again: it belongs to one
torch and one Python, so a change of either makes it stale, whatever the
files' times say."""
import pytest

import sparse_long_context_02_b200 as dsa
from sparse_long_context_02_b200 import build as dsa_build


@pytest.fixture
def calls(monkeypatch, tmp_path):
    """build_binding on files of its own, with the compiler replaced by one
    that records its calls and writes an empty file."""
    made = []

    def compile(cmd):
        made.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(dsa_build, "BINDING_PATH", str(tmp_path / "_native.so"))
    monkeypatch.setattr(dsa_build, "BINDING_STAMP", str(tmp_path / "_native.built_for"),
                        raising=False)
    monkeypatch.setattr(dsa_build.subprocess, "check_call", compile)
    return made


@pytest.mark.parametrize("what", ["torch", "python", "abi"])
def test_another_torch_or_python_builds_again(calls, monkeypatch, what):
    import torch
    dsa_build.build_binding()
    dsa_build.build_binding()
    assert len(calls) == 1
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI",
                            not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        monkeypatch.setattr(dsa_build.sysconfig, "get_config_var", lambda name: "cpython-399")
    dsa_build.build_binding()
    assert len(calls) == 2
    dsa_build.build_binding()
    assert len(calls) == 2


def test_a_build_that_fails_leaves_no_stamp_beside_another_file(calls, monkeypatch):
    dsa_build.build_binding()

    def fail(cmd):
        raise RuntimeError("no compiler")

    monkeypatch.setattr(dsa_build.subprocess, "check_call", fail)
    monkeypatch.setattr(dsa_build, "binding_key", lambda: "another")
    for _ in range(2):
        with pytest.raises(RuntimeError, match="no compiler"):
            dsa_build.build_binding()


def test_the_package_refuses_a_binding_of_another_torch(monkeypatch):
    dsa_build.build()
    monkeypatch.setattr(dsa, "_native_module", None)
    dsa._load_native()
    monkeypatch.setattr(dsa, "_native_module", None)
    monkeypatch.setattr(dsa_build, "binding_key", lambda: "another torch")
    with pytest.raises(RuntimeError, match="was built for torch"):
        dsa._load_native()
