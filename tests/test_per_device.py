"""csrc/per_device.h, compiled for the host: one value per device, looked up
from several threads without a data race (the thread sanitizer's word)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_gate_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include "per_device.h"
int main() {
  dsmoe::PerDevice p;
  int got[4];
  std::thread t[4];
  for (int i = 0; i < 4; ++i)
    t[i] = std::thread([&, i] { got[i] = p.get(i & 1, [&] { return 10 + (i & 1); }); });
  for (auto& x : t) x.join();
  for (int i = 0; i < 4; ++i)
    if (got[i] != 10 + (i & 1)) return 1;
  auto never = [] { return -1; };
  if (p.get(0, never) != 10 || p.get(1, never) != 11) return 2;
  // devices that have no place are looked up every time
  if (p.get(64, [] { return 5; }) != 5 || p.get(64, [] { return 6; }) != 6) return 3;
  if (p.get(-1, [] { return 7; }) != 7) return 4;
  puts("ok");
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
@pytest.mark.parametrize("sanitize", [[], ["-fsanitize=thread"]])
def test_values_per_device_from_several_threads(tmp_path, sanitize):
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    build = ["g++", "-std=c++17", "-O1", "-pthread", *sanitize, "-I", CSRC, str(src), "-o", str(exe)]
    if subprocess.run(build, capture_output=True).returncode and sanitize:
        pytest.skip("no thread sanitizer here")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    if sanitize and "unexpected memory mapping" in r.stderr:
        pytest.skip("the thread sanitizer does not start here")
    assert r.returncode == 0 and r.stdout == "ok\n", r.stderr
