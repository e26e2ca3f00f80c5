"""The build: what it needs, and what it names its products (compilers faked)."""
import os
import sysconfig
import types

import pytest

from block_causal_attention_wave_b200 import build


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    """A package folder of one source, and compilers that only write their outputs."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text("")
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libwave.so"))
    monkeypatch.setattr(build, "CALL", str(tmp_path / os.path.basename(build.CALL)))
    return tmp_path, ran


def test_the_library_needs_no_python_headers(tree, monkeypatch, capsys):
    path, ran = tree
    paths = dict(sysconfig.get_paths(), include=str(path / "none"))
    monkeypatch.setattr(build, "sysconfig", types.SimpleNamespace(get_paths=lambda: paths))
    assert build.build(out=build.LIB) == build.LIB
    assert (path / "libwave.so").read_text() == "built" and len(ran) == 2
    assert not os.path.exists(build.CALL) and "_call" in capsys.readouterr().err


def test_the_module_carries_pythons_abi_tag(tree):
    path, ran = tree
    (path / "_call.so").write_text("of another version")
    build.build(out=build.LIB)
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers")
    assert build.CALL.endswith("_call" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.exists(build.CALL) and not (path / "_call.so").exists()


def test_a_failing_module_is_an_error(tree, monkeypatch):
    fail = build.subprocess.run

    def run(cmd, **kw):
        r = fail(cmd, **kw)
        r.returncode = int("wave_call.cpp" in " ".join(cmd))
        return r
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    if os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        with pytest.raises(RuntimeError):
            build.build(out=build.LIB)
