"""CPU: the marshalling module is rebuilt when the torch or the Python it was made for is another, and a module
that cannot be used says why."""
import os
import subprocess
import sys

import pytest

from hstu_pointwise_attention_jagged_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "hstu_pointwise_attention_jagged_b200"


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """build_module on a module of its own, with a compiler that only counts and writes its output."""
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")

    monkeypatch.setattr(build, "MODULE", str(tmp_path / "_paged_native.so"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return runs


@pytest.mark.parametrize("what", ["torch", "python"])
def test_rebuilt_for_another_torch_or_python(compiler, monkeypatch, what):
    build.build_module()
    build.build_module()
    assert len(compiler) == 1  # up to date
    import torch
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + ".post1")
    else:
        known = build.sysconfig.get_config_var
        monkeypatch.setattr(build.sysconfig, "get_config_var",
                            lambda name: "cpython-399-other" if name == "SOABI" else known(name))
    build.build_module()
    build.build_module()
    assert len(compiler) == 2


def test_rebuilt_after_a_failed_build(compiler, monkeypatch):
    """A build that fails leaves what was there; the next one compiles again."""
    def fails(cmd, check):
        raise subprocess.CalledProcessError(1, cmd)

    works = build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run", fails)
    with pytest.raises(subprocess.CalledProcessError):
        build.build_module()
    monkeypatch.setattr(build.subprocess, "run", works)
    build.build_module()
    assert len(compiler) == 1 and os.path.exists(build.MODULE)


def _import_error(prepare):
    code = ("import sys\nfrom %s import build\n%s\ntry:\n    import %s.paged\nexcept RuntimeError as e:\n    print(e)"
            % (PACKAGE, prepare, PACKAGE))
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    return done.stdout


def test_import_errors_name_their_cause(cuda_lib, tmp_path):
    blocked = "sys.modules['%s._paged_native'] = None\n" % PACKAGE
    out = _import_error(blocked)
    assert "could not be loaded" in out and "halted" in out and "not built" not in out
    out = _import_error(blocked + "build.MODULE = %r" % str(tmp_path / "none.so"))
    assert "is not built" in out
    module = tmp_path / "_paged_native.so"
    (tmp_path / "_paged_native.so.built_for").write_text("torch 1.0, cpython-27")
    out = _import_error("build.MODULE = %r" % str(module))
    assert "was built for torch 1.0, cpython-27" in out and build.built_for() in out
    assert _import_error("") == ""
