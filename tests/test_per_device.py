"""What a kernel's first launch sets up holds for the current device only: it is kept for each device."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_gb300", "csrc")

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
#include <thread>
#include <vector>
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
enum Err { kOk = 0, kBad = 700 };
int main() {
  static mla::PerDevice<int> known;
  int made[70] = {}, v = 0;
  bool fail = true;
  auto on = [&](int dev) { return known.get(dev, v, [&](int& x) { ++made[dev]; x = 10 * dev + 1; return fail ? kBad : kOk; }); };
  CHECK(on(0) == kBad && on(0) == kBad && made[0] == 2);   // a failure is not kept
  fail = false;
  for (int i = 0; i < 3; ++i)
    for (int dev : {0, 1, 63, 5}) { v = -1; CHECK(on(dev) == kOk && v == 10 * dev + 1); }
  CHECK(made[0] == 3 && made[1] == 1 && made[63] == 1 && made[5] == 1 && made[2] == 0);
  CHECK(on(69) == kOk && v == 691 && on(69) == kOk && made[69] == 2);  // beyond the table: each time
  static mla::PerDevice<int> shared;
  std::atomic<int> n{0}, wrong{0};
  std::vector<std::thread> t;
  for (int i = 0; i < 16; ++i)
    t.emplace_back([&, i] {
      int x = 0;
      if (shared.get(i % 4, x, [&](int& y) { ++n; y = i % 4 + 7; return kOk; }) != kOk || x != i % 4 + 7) ++wrong;
    });
  for (auto& x : t) x.join();
  CHECK(n == 4 && wrong == 0);
  return 0;
}
"""


def test_values_are_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "per_device.cpp", tmp_path / "per_device"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_every_attribute_goes_through_it():
    """No launcher keeps an attribute or an occupancy of its own."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")) and name != "internal.h":
            text = open(os.path.join(CSRC, name)).read()
            assert not re.search(r"cudaFuncSetAttribute|cudaOccupancyMaxActiveClusters", text), name
