"""What build() compiles and when: nothing is compiled here, the compilers' command lines are caught."""
import pytest

from dynamic_sparse_attention_pw_b200 import _lib, build


@pytest.fixture
def commands(monkeypatch):
    build.build()
    ran = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd))
    return ran


def _compilers(commands):
    return ["nvcc" if "nvcc" in c[0] else c[0] for c in commands]


def test_what_is_up_to_date_stays(commands):
    build.build()
    assert commands == []


def test_force_reaches_the_binding(commands):
    build.build(force=True)
    assert _compilers(commands) == ["nvcc", "g++"]


def test_another_torch_or_python_makes_the_binding_stale(commands, monkeypatch):
    monkeypatch.setattr(build, "binding_target", lambda: "torch 0.0.1, cpython-30")
    build.build()
    assert _compilers(commands) == ["g++"] and '-DPW_BUILT_FOR="torch 0.0.1, cpython-30"' in commands[0]


def test_a_binding_for_another_torch_is_not_used(commands, monkeypatch):
    assert _lib.binding().built_for == f"[built for {build.binding_target()}]"
    monkeypatch.setattr(build, "binding_target", lambda: "torch 0.0.1, cpython-30")
    monkeypatch.setattr(_lib, "_binding", None)
    with pytest.raises(RuntimeError, match="build it"):
        _lib.binding()


def test_the_library_alone_needs_no_host_compiler(commands):
    build.build(force=True, binding=False)
    assert _compilers(commands) == ["nvcc"]
