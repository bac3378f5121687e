"""The build: the C library needs nothing of PyTorch, a binding that cannot be compiled says so,
and one that was compiled against another PyTorch is compiled again."""
import os

import pytest

from linear_attention_12_b200 import build as b

CU = 'extern "C" __attribute__((visibility("default"))) int gdn_nothing() { return 7; }\n'


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """A build of one small source into a directory of its own."""
    src = tmp_path / "nothing.cu"
    src.write_text(CU)
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libgdn.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_gdn_torch.so"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "sources", lambda: [str(src)])
    return tmp_path


def test_the_library_needs_no_pytorch(sandbox, monkeypatch, capsys):
    monkeypatch.setattr(b, "_torch_version", lambda: None)
    monkeypatch.setenv("CXX", "/nonexistent/c++")
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING)
    assert "_gdn_torch.so" in capsys.readouterr().err


def test_a_binding_that_fails_names_itself(sandbox, monkeypatch):
    monkeypatch.setenv("CXX", "/nonexistent/c++")
    with pytest.raises(RuntimeError, match="_gdn_torch.so"):
        b.build()
    assert os.path.exists(b.LIB)


def test_another_pytorch_builds_the_binding_again(sandbox, monkeypatch):
    runs = []

    def compile_(cmd):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b.subprocess, "check_call", compile_)
    b.build_binding()
    b.build_binding()
    assert len(runs) == 1
    monkeypatch.setattr(b, "_torch_version", lambda: "0.0")
    b.build_binding()
    b.build_binding()
    assert len(runs) == 2
