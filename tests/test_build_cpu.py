"""The build's order: the C libraries do not depend on the Python side. The
compilers are stand-ins that write empty files."""
import os
import subprocess
import types

import pytest

import masked_gqa_attention_gb300.build as B


@pytest.fixture
def ran(tmp_path, monkeypatch):
    """The commands run, with every output under tmp_path; ran.fail: compilers that fail."""
    log = types.SimpleNamespace(commands=[], fail=set())
    out, obj = str(tmp_path / "lib"), str(tmp_path / "obj")
    for name, value in (("OUT_DIR", out), ("OBJ_DIR", obj), ("LIB", os.path.join(out, "libmgqa.so")),
                        ("LIB_DEBUG", os.path.join(out, "libmgqa_debug.so")), ("BIND", os.path.join(out, "_mgqa_bind.so"))):
        monkeypatch.setattr(B, name, value)
    monkeypatch.setattr(B, "VARIANTS", {"release": (B.LIB, obj, []), "debug": (B.LIB_DEBUG, os.path.join(obj, "debug"), [])})

    def run(cmd, **kw):
        log.commands.append(cmd)
        if cmd[0] in log.fail:
            return subprocess.CompletedProcess(cmd, 1, "", f"no {cmd[0]} today")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(B, "_bind_flags", lambda: (["-O2"], ["-l:libmgqa.so"]))
    return log


def built():
    return [os.path.exists(x) for x in (B.LIB, B.LIB_DEBUG, B.BIND)]


def test_everything_is_built_once(ran):
    assert B.build() == B.LIB and built() == [True, True, True]
    n = len(ran.commands)
    assert B.build() == B.LIB and len(ran.commands) == n
    link = next(i for i, c in enumerate(ran.commands) if c[0] == "g++" and "-shared" in c)
    assert link > max(i for i, c in enumerate(ran.commands) if c[0] == "nvcc" and "-shared" in c)


def test_libraries_are_built_without_a_host_compiler(ran):
    ran.fail = {"g++"}
    with pytest.raises(RuntimeError, match="no g\\+\\+ today"):
        B.build()
    assert built() == [True, True, False]


def test_libraries_are_built_without_the_headers_of_the_binding(ran, monkeypatch):
    def missing():
        raise ImportError("no torch")

    monkeypatch.setattr(B, "_bind_flags", missing)
    with pytest.raises(ImportError, match="no torch"):
        B.build()
    assert built() == [True, True, False]


def test_the_debug_library_alone(ran):
    B.build(variants=("debug",))
    assert built() == [False, True, False]
    assert all(c[0] == "nvcc" for c in ran.commands)
