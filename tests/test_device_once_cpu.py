"""Kernel attributes are set on every device that a process uses: the mask that remembers where, and that the
launchers have no other memory."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_split_kv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_once.h"
enum Status { kOk = 0, kFailed = 1 };
int fail(int line) { std::printf("line %d\n", line); return 1; }
#define CHECK(x) if (!(x)) return fail(__LINE__)
int main() {
  mla::DeviceOnce once;
  int calls[80] = {};
  auto set = [&](int dev) { return once(dev, [&] { ++calls[dev]; return kOk; }); };
  for (int k = 0; k < 3; ++k)
    for (int dev : {0, 1, 5, 63}) CHECK(set(dev) == kOk);
  CHECK(calls[0] == 1 && calls[1] == 1 && calls[5] == 1 && calls[63] == 1 && calls[2] == 0);
  CHECK(set(64) == kOk && set(64) == kOk && calls[64] == 2);  // past the mask
  CHECK(calls[0] == 1);
  int tries = 0;
  auto flaky = [&] { return once(7, [&] { return ++tries < 3 ? kFailed : kOk; }); };
  CHECK(flaky() == kFailed && flaky() == kFailed && flaky() == kOk && flaky() == kOk && tries == 3);
  mla::DeviceOnce shared;
  std::atomic<int> many{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&] { for (int dev = 0; dev < 64; ++dev) shared(dev, [&] { ++many; return kOk; }); });
  for (auto& t : threads) t.join();
  CHECK(many >= 64 && many <= 8 * 64);
  const int before = many;
  for (int dev = 0; dev < 64; ++dev) shared(dev, [&] { ++many; return kOk; });
  CHECK(many == before);
  std::printf("ok\n");
  return 0;
}
"""


def test_a_device_is_set_once_and_every_device_is(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "once.cpp"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "once")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_launchers_set_attributes_by_device(name):
    """No flag for the whole process beside an attribute of the current device: a second GPU's first launch would
    go without it."""
    with open(os.path.join(CSRC, name)) as f:
        source = f.read()
    assert not re.search(r"\bstatic\s+bool\b", source)
    if name != "device_common.cuh":
        assert "cudaFuncSetAttribute" not in source
