"""Build libkvs.so in-tree: each CUDA source compiled for sm_103a in parallel, then linked; and kvs_binding.so, the compiled part of the
Python binding, against torch's headers."""
import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libkvs.so")
BINDING = os.path.join(OUT_DIR, "kvs_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    inc = os.path.join(os.path.dirname(HERE), "include")
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(inc, f) for f in os.listdir(inc) if f.endswith(".h")]
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_folder():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None and spec.submodule_search_locations else None


def _torch():
    """torch's folder; None where the compiled binding has nothing to be built against (no torch with CUDA, no headers of Python): libkvs.so is
    then all that is built."""
    torch = _torch_folder()
    if torch is None:
        return None
    needed = [os.path.join(torch, "lib", "libc10_cuda.so"), os.path.join(torch, "lib", "libtorch_python.so"),
              os.path.join(torch, "include", "c10", "cuda", "CUDAFunctions.h"), os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    return torch if all(os.path.exists(f) for f in needed) else None


def _binding_key():
    """What the binding's layout of tensors and of Python's objects hangs on: this torch and this Python."""
    version = os.path.join(_torch_folder() or "", "version.py")
    return "\n".join([open(version).read() if os.path.exists(version) else "", str(sysconfig.get_config_var("SOABI"))])


def _key_file():
    return BINDING + ".key"


def binding_fits():
    """Whether kvs_binding.so was built for this torch and this Python."""
    if not os.path.exists(_key_file()):
        return False
    with open(_key_file()) as f:
        return f.read() == _binding_key()


def _compile_binding():
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(OUT_DIR, "binding.o")
    torch = _torch()
    if torch is None:
        return None
    if _stale(obj, [src] + headers()) or not binding_fits():
        cuda = os.path.dirname(os.path.dirname(NVCC))
        inc = [f"-I{torch}/include", f"-I{torch}/include/torch/csrc/api/include", f"-I{cuda}/include", f"-I{sysconfig.get_paths()['include']}"]
        tmp = obj + f".tmp{os.getpid()}"
        _run(["g++", "-O2", "-std=c++17", "-fPIC"] + inc + ["-c", src, "-o", tmp], src)
        os.replace(tmp, obj)
    return obj


def _link_binding(obj):
    if obj is not None and (_stale(BINDING, [obj]) or not binding_fits()):
        torch, tmp = _torch(), BINDING + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, obj, f"-L{OUT_DIR}", "-lkvs", "-Wl,-rpath,$ORIGIN", f"-L{torch}/lib", "-ltorch_python", "-ltorch_cpu",
              "-lc10", "-lc10_cuda"], BINDING)
        os.replace(tmp, BINDING)
        with open(tmp, "w") as f:
            f.write(_binding_key())
        os.replace(tmp, _key_file())


def _compile(src):
    obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + headers()):
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [NVCC] + ARCH + FLAGS + ["-c", src, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sources()
    if force:
        for f in os.listdir(OUT_DIR):
            os.remove(os.path.join(OUT_DIR, f))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
        binding = binding.result()
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_binding(binding)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
