"""What can be built and imported without the part of the Python binding that is in C++: the C library, and every
call that is marshalled in Python."""
import importlib.util
import os
import shutil
import subprocess
import sys
import types

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_dispatch_grouped_amd")


def build_module(tmp_path, monkeypatch, fails=None):
    """_build.py whose tools only leave a file where they are told to; (module, the commands)."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "_build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.OUT, b.BINDING, b.BUILD = (str(tmp_path / n) for n in ("librdg.so", "_binding.so", "_build"))
    done = []

    def run(cmd, **_):
        done.append(cmd)
        if fails and any(fails in str(c) for c in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "subprocess", types.SimpleNamespace(run=run))
    return b, done


def test_the_library_is_built_where_there_is_no_torch(tmp_path, monkeypatch):
    b, done = build_module(tmp_path, monkeypatch)
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    b.build()
    assert os.path.exists(b.OUT) and not os.path.exists(b.BINDING)
    assert len(done) == len(b.SOURCES) + 1 and not any("binding" in str(c) for cmd in done for c in cmd)


def test_the_library_is_built_where_the_binding_does_not_compile(tmp_path, monkeypatch):
    b, _ = build_module(tmp_path, monkeypatch, fails="binding.cpp")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert os.path.exists(b.OUT) and not os.path.exists(b.BINDING)


def test_both_are_built_with_torch(tmp_path, monkeypatch):
    b, done = build_module(tmp_path, monkeypatch)
    b.build()
    assert os.path.exists(b.OUT) and os.path.exists(b.BINDING) and len(done) == len(b.SOURCES) + 3


def test_calls_that_are_marshalled_in_python_need_no_binding(tmp_path):
    to = tmp_path / "routing_dispatch_grouped_amd"
    os.mkdir(to)
    for name in ("__init__.py", "librdg.so"):
        shutil.copy(os.path.join(PKG, name), to / name)
    code = """
import torch, routing_dispatch_grouped_amd as rdg
assert rdg.__file__.startswith(%r)
try:
    rdg.rdg_route(torch.empty(2, 16, dtype=torch.int32), 1, 1, 2, 1.0, None, None)
except ImportError:
    raise SystemExit("an older call wants the binding")
except Exception as e:
    print(type(e).__name__)
assert rdg.rdg_linear_workspace_bytes(64, 256, 7168, rdg.RDG_BF16) > 0
rdg._bind_torch()
for call in (lambda: rdg.rdg_add_norm(None, None, 0.0), lambda: rdg.rdg_linear(None, None, 1, None, None, None),
             lambda: rdg.rdg_route_topk(None, 0, 1, 1, 1, 1, 1, 1.0, None, None)):
    try:
        call()
    except ImportError as e:
        assert "_binding.so is not built" in str(e), e
    else:
        raise SystemExit("ran without its binding")
""" % str(to)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=dict(os.environ, PYTHONPATH=str(tmp_path)), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_without_the_library_nothing_is_imported(tmp_path):
    to = tmp_path / "routing_dispatch_grouped_amd"
    os.mkdir(to)
    shutil.copy(os.path.join(PKG, "__init__.py"), to)
    r = subprocess.run([sys.executable, "-c", "import routing_dispatch_grouped_amd"], cwd=tmp_path,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)), capture_output=True, text=True)
    assert r.returncode != 0 and "librdg.so is not built" in r.stderr
