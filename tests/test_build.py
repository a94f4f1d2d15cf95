"""What build() makes of the compiled binding where torch or Python's headers are not what it needs, and when it makes it again (no GPU)."""
import os
import types

import pytest

from sparse_kv_cache_decode_gb300 import build as B


def touch(*path):
    f = os.path.join(*path)
    os.makedirs(os.path.dirname(f), exist_ok=True)
    open(f, "a").close()


@pytest.fixture
def world(tmp_path, monkeypatch):
    """A torch, a Python and an output folder of its own; `ran`: the commands that would have been run."""
    torch, include, out = (str(tmp_path / n) for n in ("torch", "include", "out"))
    for f in ("lib/libc10_cuda.so", "lib/libtorch_python.so", "include/c10/cuda/CUDAFunctions.h", "version.py"):
        touch(torch, *f.split("/"))
    touch(include, "Python.h")
    os.makedirs(out)
    w = types.SimpleNamespace(torch=torch, include=include, ran=[], spec=types.SimpleNamespace(submodule_search_locations=[torch]))

    def run(cmd, what):
        w.ran.append(cmd)
        touch(cmd[cmd.index("-o") + 1])
    monkeypatch.setattr(B, "OUT_DIR", out)
    monkeypatch.setattr(B, "BINDING", os.path.join(out, "kvs_binding.so"))
    monkeypatch.setattr(B, "_run", run)
    find, paths = B.importlib.util.find_spec, B.sysconfig.get_paths
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: w.spec if name == "torch" else find(name, *a))
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda *a, **k: paths(*a, **k) | {"include": include})
    return w


def make():
    B._link_binding(B._compile_binding())


@pytest.mark.parametrize("missing", ["torch", "lib/libc10_cuda.so", "lib/libtorch_python.so", "include/c10/cuda/CUDAFunctions.h", "Python.h"])
def test_without_what_it_needs_there_is_no_binding_and_no_error(world, missing):
    if missing == "torch":
        world.spec = None
    else:
        os.remove(os.path.join(world.include if missing == "Python.h" else world.torch, missing))
    make()
    assert world.ran == [] and not os.path.exists(B.BINDING) and not B.binding_fits()


def test_it_is_made_once(world):
    assert not B.binding_fits()
    make()
    assert len(world.ran) == 2 and os.path.exists(B.BINDING) and B.binding_fits()
    make()
    assert len(world.ran) == 2
    assert sorted(os.listdir(B.OUT_DIR)) == ["binding.o", "kvs_binding.so", "kvs_binding.so.key"]


@pytest.mark.parametrize("what", ["version", "python"])
def test_another_torch_or_python_makes_it_again(world, monkeypatch, what):
    make()
    if what == "version":
        with open(os.path.join(world.torch, "version.py"), "w") as f:
            f.write("__version__ = '3.0'")
    else:
        get = B.sysconfig.get_config_var
        monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else get(name))
    assert not B.binding_fits()
    make()
    assert len(world.ran) == 4 and B.binding_fits()


@pytest.mark.parametrize("gone", ["headers", "folder"])
def test_a_built_binding_needs_no_headers(world, gone):
    """A machine that only runs it: without Python's headers, or with the same torch in another place."""
    make()
    if gone == "headers":
        os.remove(os.path.join(world.include, "Python.h"))
    else:
        os.rename(world.torch, world.torch + "2")
        world.spec.submodule_search_locations = [world.torch + "2"]
    assert B.binding_fits()
    make()
    assert len(world.ran) == 2


def test_a_build_that_ends_half_way_is_done_again(world, monkeypatch):
    make()
    with open(os.path.join(world.torch, "version.py"), "w") as f:
        f.write("__version__ = '3.0'")
    B._compile_binding()                                  # ... and nothing linked
    assert not B.binding_fits()
    make()
    assert B.binding_fits() and world.ran[-1][1] == "-shared"


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    pytest.importorskip("torch")
    import sparse_kv_cache_decode_gb300 as K
    B.build()
    K.binding()
    monkeypatch.setattr(K, "_binding", None)
    monkeypatch.setattr(B, "binding_fits", lambda: False)
    with pytest.raises(RuntimeError, match="not built for this torch"):
        K.binding()
