"""The record of a kernel attribute that was already set never runs ahead of the attribute, whatever
threads make their first calls at once (host code, compiled and run on the CPU)."""
import os
import subprocess

from bit_mixed_precision_channel_b200 import build as kbuild

MAIN = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "kvq_limit.cuh"

using namespace std::chrono_literals;
int seen = 0;
std::atomic<int> limit{0}, started{0}, calls{0};

int set(int n) {
  ++calls;
  if (n == 16) {  // the smaller call is slow: the larger one has all the time to overtake it
    started = 1;
    std::this_thread::sleep_for(300ms);
  }
  limit = n;
  return 0;
}

int main() {
  std::thread small([] { kvq::raise_limit(seen, 16, set); });
  std::thread large([] {
    while (!started) std::this_thread::yield();
    kvq::raise_limit(seen, 64, set);
  });
  small.join();
  large.join();
  if (limit.load() != 64 || seen != 64 || calls.load() != 2) return std::printf("limit %d, recorded %d\n", limit.load(), seen), 1;
  kvq::raise_limit(seen, 32, set);  // below what was set: no call
  if (limit.load() != 64 || calls.load() != 2) return std::printf("lowered to %d\n", limit.load()), 1;
  const int e = kvq::raise_limit(seen, 128, [](int) { return 7; });  // refused: reported, not recorded
  if (e != 7 || seen != 64) return std::printf("status %d, recorded %d\n", e, seen), 1;
  return 0;
}
"""


def test_a_smaller_size_set_late_does_not_lower_a_larger_one(tmp_path):
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(MAIN)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-pthread", "-I", os.path.join(kbuild.HERE, "csrc"), str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
