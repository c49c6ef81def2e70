"""Build libklein.so (the CUDA library) in-tree with nvcc for sm_100a, and
klein_torch.<ABI>.so (its binding to torch tensors, for the projection path) with
g++.  The binding's name holds the Python and torch it was compiled against, so
another of either finds none and has it built.

Usage: ``python -m diffusion_transformer_image_nvfp4_b200.build [--force] [--lib-only]``
(``--lib-only``: no binding, for users of the C ABI; needs nvcc alone).
"""

import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libklein.so")
BIND_SOURCE = os.path.join(CSRC, "kl_python.cpp")
HEADER = os.path.join(ROOT, "include", "klein.h")


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if not f.endswith(".cpp")] + [HEADER]


def bind_path():
    """The binding compiled against the running Python and torch."""
    import sysconfig

    import torch

    abi = "-".join([sysconfig.get_config_var("SOABI"), "torch", torch.__version__, str(torch.version.git_version)[:8],
                    f"cxx11abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"])
    return os.path.join(PKG_DIR, f"klein_torch.{abi}.so")


def _stale(path, sources):
    return not os.path.exists(path) or any(os.path.getmtime(s) > os.path.getmtime(path) for s in sources)


def needs_build():
    return _stale(LIB_PATH, _sources())


def build(force=False, verbose=False, binding=True):
    """Compile csrc/klein.cu into libklein.so and, unless ``binding`` is false,
    csrc/kl_python.cpp into the binding next to this file; returns libklein.so's
    path."""
    if force or needs_build():
        _build_lib(verbose)
    if binding and (force or _stale(bind_path(), [BIND_SOURCE, HEADER])):
        _build_binding()
    return LIB_PATH


def _run(cmd, path):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + r.stdout + r.stderr)
    os.replace(path + ".tmp", path)
    return r


def _build_binding():
    import sysconfig

    import torch

    root, path = os.path.dirname(torch.__file__), bind_path()
    inc, cuda = os.path.join(root, "include"), os.path.dirname(os.path.dirname(_nvcc()))
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
            sysconfig.get_paths()["include"]]
    # the system's g++ and its shared libstdc++: torch's exceptions are caught
    # in the binding, which a C++ runtime of its own (linked statically) cannot do
    _run([shutil.which("g++", path="/usr/bin:/usr/local/bin") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in dirs), BIND_SOURCE,
          "-o", path + ".tmp", f"-L{PKG_DIR}", f"-L{os.path.join(root, 'lib')}", "-l:libklein.so", "-ltorch_python",
          "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"], path)


def _build_lib(verbose):
    cmd = [
        _nvcc(),
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-O3", "-lineinfo", "-std=c++17",
        "-Xcompiler", "-fPIC", "-shared",
        "-I", os.path.join(ROOT, "include"),
        os.path.join(CSRC, "klein.cu"),
        "-o", LIB_PATH + ".tmp",
    ]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = _run(cmd, LIB_PATH)
    if verbose:
        sys.stderr.write(r.stderr)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, binding="--lib-only" not in sys.argv))
