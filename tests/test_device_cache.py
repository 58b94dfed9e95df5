"""The per-device numbers that launches look up are safe to ask for from
several host threads at once (the header has no CUDA in it: built with the
thread sanitizer here)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_swiglu_experts_b200", "csrc")

MAIN = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_cache.h"
moe::DeviceCache& cache() {
  static moe::DeviceCache c;
  return c;
}
int main() {
  std::atomic<int> wrong{0}, found{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&, i] {
      for (int n = 0; n < 2000; ++n) {
        const int dev = (n + i) % 3;
        if (cache().get(dev, [&] { ++found; return 70 + dev; }) != 70 + dev) ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  if (cache().get(5, [] { return -1; }) != 0) ++wrong;       // a failure is not kept
  if (cache().get(5, [] { return 0; }) != 0) ++wrong;
  if (cache().get(5, [] { return 9; }) != 0) ++wrong;        // 0 is an answer
  if (cache().get(-1, [] { return 9; }) != 0 || cache().get(64, [] { return 9; }) != 0) ++wrong;
  printf("%d %d\n", wrong.load(), found.load());
  return 0;
}
"""


def test_threads_agree(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "c.cc", tmp_path / "c"
    src.write_text(MAIN)
    build = [cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)]
    checked = subprocess.run(build + ["-fsanitize=thread"], capture_output=True).returncode == 0
    if not checked:
        subprocess.run(build, check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-1000:]
    wrong, found = map(int, r.stdout.split())
    assert wrong == 0 and 3 <= found <= 24


def test_launches_keep_their_numbers_in_it():
    """No launch keeps a per-device number in plain statics of its own."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = open(os.path.join(CSRC, name)).read()
            assert "static bool known" not in text, name
