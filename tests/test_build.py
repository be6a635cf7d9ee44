"""The build's order, with the compilers replaced (CPU, nothing is compiled)."""

import os
import subprocess
import types

import pytest

from quantized_weight_prefill_q4_amd import build


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Compilers that write an empty output; fails: file names they refuse."""
    fails = set()

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        bad = [a for a in cmd if os.path.basename(a) in fails]
        if not bad:
            open(out, "w").close()
        return types.SimpleNamespace(returncode=len(bad), stdout="", stderr=f"no {bad}")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libmq.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_binding.so"))
    return fails


def test_builds_both(fake):
    assert build.build_lib() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.BINDING_PATH)


def test_library_does_not_need_the_binding(fake):
    fake.add("binding.cpp")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build_lib()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)


def test_no_binding_of_an_older_library_stays(fake):
    build.build_lib()
    fake.add("binding.cpp")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build_lib()
    assert not os.path.exists(build.BINDING_PATH)


def test_no_library_from_a_source_that_fails(fake):
    fake.add("gemm.hip")
    with pytest.raises(RuntimeError, match="gemm.hip"):
        build.build_lib()
    assert not os.path.exists(build.LIB_PATH)
