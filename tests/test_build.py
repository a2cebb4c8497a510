"""What the build leaves behind when the host module cannot be built (compilers replaced; nothing is compiled)."""

import os

import pytest

from expert_ffn_ragged_amd import build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The build's files go to tmp_path; a command only writes its output.  Returns the commands' list."""
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "librd.so"))
    monkeypatch.setattr(build, "MODULE", str(tmp_path / "_rd.so"))
    commands = []

    def run(cmd):
        commands.append(cmd)
        if cmd[0] == build.CXX and "fail" in commands[0:1]:
            raise RuntimeError("no host compiler")
        with open(cmd[cmd.index("-o") + 1], "w") as fh:
            fh.write("built")
        return ""

    monkeypatch.setattr(build, "_run", run)
    return commands


def test_both_are_built(made):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.MODULE)
    assert len(made) == len(build.SOURCES) + 3  # each source, the host module's, two links


def test_the_library_needs_no_torch(made, monkeypatch, capsys):
    def flags():
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(build, "_torch_flags", flags)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.MODULE)
    assert "_rd.so" in capsys.readouterr().err  # and it says what is missing


def test_a_failing_host_module_fails_the_build_after_the_library(made):
    made.append("fail")
    with pytest.raises(RuntimeError, match="no host compiler"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.MODULE)


def test_a_failing_kernel_source_builds_nothing(made, monkeypatch):
    def run(cmd):
        raise RuntimeError("does not compile")

    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError, match="does not compile"):
        build.build()
    assert not os.path.exists(build.LIB) and not os.path.exists(build.MODULE)
