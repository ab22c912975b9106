"""What build() needs: with host=False only hipcc is called, so that the C library can be built where there is no
g++ and no Python headers."""
import os
import types

import pytest

from block_diagonal_eigenbasis_amd import build as b


@pytest.fixture
def ran(monkeypatch, tmp_path):
    cmds = []

    def run(cmd, **kw):
        cmds.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stderr="")
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libdobb.so"))
    monkeypatch.setattr(b, "HOST", str(tmp_path / "_dobb_host.so"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    return cmds


def test_the_library_alone(ran):
    b.build(host=False)
    assert len(ran) == len(b.SOURCES) + 1 and {c[0] for c in ran} == {b.HIPCC}
    assert os.path.exists(b.LIB) and not os.path.exists(b.HOST)


def test_the_binding_is_built_behind_the_library(ran):
    b.build()
    assert len(ran) == len(b.SOURCES) + 2 and "-ldobb" in ran[-1] and ran[-1][0] != b.HIPCC
    assert os.path.exists(b.LIB) and os.path.exists(b.HOST)
