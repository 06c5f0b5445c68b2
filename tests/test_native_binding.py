"""The binding's native module on the host: importing the package maps no kernel library, and once a call has looked for
it, the module and the ctypes calls share one copy of the library, the one that lies there then.  Each check runs in a
process of its own, on a copy of the package whose library is a stand-in that exports the names and a version."""
import os
import shutil
import subprocess
import sys

import pytest

from gated_delta_rule_76_b200 import build as gbuild
from gated_delta_rule_76_b200 import gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAPPED = """
import os
def mapped():
    '''(name, device and inode) of the package's libraries in this process.'''
    rows = [l.split() for l in open("/proc/self/maps")]
    return {(os.path.basename(r[5]), r[3] + r[4]) for r in rows if len(r) > 5 and r[5].startswith(os.getcwd()) and ".so" in r[5]}
"""


@pytest.fixture(scope="module")
def built():
    gbuild.build()


def run(code, cwd):
    env = dict(os.environ, PYTHONPATH="", PYTHONDONTWRITEBYTECODE="1")
    r = subprocess.run([sys.executable, "-c", MAPPED + code], cwd=cwd, capture_output=True, text=True, env=env)
    assert r.returncode == 0, r.stdout + r.stderr


def stand_in(path, version):
    src = path + ".c"
    with open(src, "w") as f:
        f.write("\n".join(f"int {n}(void) {{ return {version}; }}" for n in gdn.EXPORTED))
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-o", path, src])


@pytest.fixture
def package(built, tmp_path):
    """A copy of the package with the native module and a stand-in library of version 1; another of version 2 beside it."""
    to = tmp_path / "gated_delta_rule_76_b200"
    os.mkdir(to)
    for name in os.listdir(gbuild.PKG):
        if name.endswith(".py"):
            shutil.copy2(os.path.join(gbuild.PKG, name), to)
    shutil.copy2(gbuild.binding(), to)
    stand_in(str(to / "libgdn.so"), 1)
    stand_in(str(tmp_path / "new.so"), 2)
    return tmp_path


def test_importing_the_package_maps_no_library(built):
    run("""
import gated_delta_rule_76_b200
import gated_delta_rule_76_b200.build, gated_delta_rule_76_b200.inputs, gated_delta_rule_76_b200.seqpar
assert not mapped(), mapped()
""", ROOT)


def test_a_library_replaced_after_import_is_the_one_that_is_called(package):
    run("""
from gated_delta_rule_76_b200 import gdn
os.replace("new.so", gdn.LIB_PATH)
assert gdn.load().gdn_version() == 2
assert gdn._native is not None
assert len([m for m in mapped() if m[0].startswith("libgdn.so")]) == 1, mapped()
""", package)


def test_a_library_replaced_after_load_is_not_mapped_beside_the_first(package):
    run("""
from gated_delta_rule_76_b200 import gdn
assert gdn.load().gdn_version() == 1
os.replace("new.so", gdn.LIB_PATH)
assert gdn._native is not None and gdn.load().gdn_version() == 1
assert len([m for m in mapped() if m[0].startswith("libgdn.so")]) == 1, mapped()
""", package)


def test_a_module_built_after_the_first_call_is_found(package):
    run("""
from gated_delta_rule_76_b200 import build, gdn
module = build.binding()
os.rename(module, "kept.so")
assert gdn._native is None and gdn._native_calls() is None
os.rename("kept.so", module)
build._look_again()
assert gdn._native is not None and gdn._native_calls() is gdn._native
build._look_again()
assert "_native" in vars(gdn)
""", package)


def test_the_module_takes_every_entry_point_once(built):
    """A name that is missing is refused, and unbound calls leave the work to the general way."""
    run("""
import ctypes
from gated_delta_rule_76_b200 import gdn
native = gdn._native
names = native.entries()
assert len(set(names)) == len(names) and set(names) <= set(gdn.EXPORTED)
for bad in ({}, {n: 0 for n in names}, {n: 1 for n in names[1:]}):
    try:
        native.bind(bad)
    except KeyError:
        continue
    assert False, bad
try:
    native.bind(None)
except TypeError:
    pass
else:
    assert False
""", ROOT)


def test_a_module_of_another_torch_is_left_alone(package):
    run("""
import torch
torch.__version__ = "1.0"
from gated_delta_rule_76_b200 import gdn
assert gdn.load().gdn_version() == 1 and gdn._native is None
""", package)


def test_a_file_that_is_no_module_is_left_alone(package):
    run("""
from gated_delta_rule_76_b200 import build, gdn
open(build.binding(), "w").write("no library")
assert gdn.load().gdn_version() == 1 and gdn._native is None
""", package)


@pytest.mark.parametrize("compiler", ["fails", "is missing"])
def test_a_host_without_the_headers_keeps_the_library(compiler, monkeypatch, tmp_path):
    """The module is optional, also when it is built; what an older source left is taken away."""
    path = str(tmp_path / "module.so")
    open(path, "w").close()

    def run(cmd, **kw):
        assert cmd[0] == "g++"
        if compiler == "is missing":
            raise FileNotFoundError("no g++")
        return subprocess.CompletedProcess(cmd, 1, "", "no torch/csrc/Exceptions.h")

    monkeypatch.setattr(gbuild, "binding", lambda: path)
    monkeypatch.setattr(gbuild.subprocess, "run", run)
    with pytest.warns(UserWarning, match="native module is not built"):
        gbuild._build_binding(True, False)
    assert not os.path.exists(path)


def test_the_module_belongs_to_one_torch_and_one_python(monkeypatch):
    import torch
    here = gbuild.binding()
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert gbuild.binding() != here
    monkeypatch.undo()
    monkeypatch.setattr(gbuild.sysconfig, "get_config_var", lambda name: ".cpython-311.so")
    assert gbuild.binding() != here


def test_a_stream_of_another_device_is_refused():
    """The tensors' device decides where a call runs: a stream of another one would be passed over in silence."""
    import types

    import torch
    t = types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0), get_device=lambda: 0)
    other = types.SimpleNamespace(cuda_stream=77, device=torch.device("cuda", 1))
    with pytest.raises(gdn.GdnError, match="stream of cuda:1 .* cuda:0"):
        gdn._on(t, other)
