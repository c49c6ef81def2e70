"""What the library keeps per device may be asked for by several host threads at
once: no data race (ThreadSanitizer, on the header alone), and the same results
(on a GPU, the first calls of a process made by many threads)."""

import os
import re
import subprocess
import sys

import pytest

from diffusion_transformer_image_nvfp4_b200 import build

PROGRAM = r"""
#include <thread>
#include <vector>
#include "kl_host.h"
static kl::DeviceValue value;
int main() {
  std::vector<std::thread> ts;
  std::atomic<int> bad{0};
  for (int t = 0; t < 8; ++t)
    ts.emplace_back([&] {
      for (int round = 0; round < 100; ++round)
        for (int dev = -1; dev <= kl::kMaxDevices; ++dev)
          if (value.get(dev, [dev] { return 100 + dev; }) != 100 + dev) bad = 1;
    });
  for (auto& t : ts) t.join();
  int asked = 0;
  for (int k = 0; k < 2; ++k) {
    value.get(3, [&] { return ++asked; });                 // kept
    value.get(kl::kMaxDevices, [&] { return ++asked; });   // not kept
  }
  return bad || asked != 2;
}
"""


def test_no_data_race(tmp_path):
    src, exe = tmp_path / "t.cpp", str(tmp_path / "t")
    src.write_text(PROGRAM)
    probe = tmp_path / "p.cpp"
    probe.write_text("int main() { return 0; }")
    tsan = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-pthread"]
    if subprocess.run([*tsan, str(probe), "-o", exe], capture_output=True).returncode or subprocess.run([exe]).returncode:
        pytest.skip("no ThreadSanitizer on this machine")
    r = subprocess.run([*tsan, "-I", build.CSRC, str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr


def test_no_other_table_of_devices_without_a_lock():
    # plain arrays over the devices are in kl_noalloc.cu alone, under its mutex
    for f in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, f)) as s:
            if f not in ("kl_host.h", "kl_noalloc.cu"):
                assert not re.search(r"\w+\[kMaxDevices\]", s.read()), f


@pytest.mark.gpu
def test_first_calls_by_many_threads():
    # ctypes releases the interpreter's lock, so the C entry points do run at once
    code = """
import ctypes, threading, torch
import diffusion_transformer_image_nvfp4_b200 as kl
L = kl.lib()
torch.manual_seed(0)
sizes = [(1, 1000, 1328), (10, 256, 4096), (40, 512, 2048), (64, 1024, 1024), (100, 384, 8192), (333, 1000, 1328)] * 2
ops = []
for m, n, k in sizes:
    a, w = (torch.randn(r, k, device="cuda").bfloat16() for r in (m, n))
    ops.append((kl.quantize_fp8_block(a), kl.quantize_fp8_block(w, "tile"), torch.zeros(m, n, device="cuda")))
torch.cuda.synchronize()
go, bad = threading.Barrier(len(ops)), []
def call(A, W, out):
    fa, fw = (kl._FP8Tensor(t.codes.data_ptr(), t.scales.data_ptr(), t.codes.stride(0)) for t in (A, W))
    torch.cuda.set_device(0)
    go.wait()
    st = L.kl_gemm_fp8_block(ctypes.byref(fa), ctypes.byref(fw), A.rows, W.rows, A.cols, out.data_ptr(), 1, W.rows, 0, None)
    if st:
        bad.append(st)
ts = [threading.Thread(target=call, args=o) for o in ops]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
assert not bad, bad
for A, W, out in ops:
    assert torch.equal(out, kl.gemm_fp8_block(A, W, out_dtype=torch.float32))
assert kl.device_status() == "KL_OK"
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240, cwd=build.ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
