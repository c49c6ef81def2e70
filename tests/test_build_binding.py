"""The binding is compiled against one Python and one torch: neither the build
nor the loader takes it for another."""

import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from diffusion_transformer_image_nvfp4_b200 import build


def _other_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")


def _other_torch_commit(monkeypatch):
    monkeypatch.setattr(torch.version, "git_version", "0" * 40)


def _other_cxx_abi(monkeypatch):
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)


def _other_python(monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-other" if n == "SOABI" else real(n))


@pytest.mark.parametrize("other", [_other_torch, _other_torch_commit, _other_cxx_abi, _other_python])
def test_a_binding_of_another_abi_is_neither_kept_nor_loaded(other, monkeypatch):
    build.build()
    built = []
    monkeypatch.setattr(build, "_build_binding", lambda: built.append(1))
    build.build()
    assert not built  # ours is current
    other(monkeypatch)
    build.build()
    assert built == [1]
    monkeypatch.setattr(kl, "_EXT", None)
    with pytest.raises(RuntimeError, match="missing"):
        kl._ext()


def test_the_loaded_binding_is_this_abis():
    build.build()
    path = kl._ext().__file__
    assert path == build.bind_path() and torch.__version__ in os.path.basename(path)


def test_the_library_is_built_without_the_binding(monkeypatch):
    # what the C ABI needs does not depend on g++, or on torch's and Python's headers
    ran = []
    monkeypatch.setattr(build, "_build_lib", lambda verbose: ran.append("lib"))
    monkeypatch.setattr(build, "_build_binding", lambda: ran.append("binding"))
    assert build.build(force=True, binding=False) == build.LIB_PATH and ran == ["lib"]
    ran.clear()
    build.build(force=True)
    assert ran == ["lib", "binding"]


def test_lib_only_from_the_command_line():
    build.build()
    before = os.stat(build.bind_path()).st_mtime_ns
    os.utime(build.bind_path(), (1, 1))  # out of date
    try:
        r = subprocess.run([sys.executable, "-m", "diffusion_transformer_image_nvfp4_b200.build", "--lib-only"],
                           capture_output=True, text=True, cwd=build.ROOT)
        assert r.returncode == 0 and r.stdout.strip() == build.LIB_PATH, r.stderr
        assert os.stat(build.bind_path()).st_mtime == 1
    finally:
        os.utime(build.bind_path(), ns=(before, before))
