"""The arithmetic of windows and tiles at the ends of its range, compiled for the host with overflow checks."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_split_kv_gb300", "csrc")
CUDA = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda") if d and os.path.isdir(os.path.join(d, "include"))), None)

PROGRAM = r"""
#include <cstdio>
#include "kernels.h"
int fail(int line) { std::printf("line %d\n", line); return 1; }
#define CHECK(x) if (!(x)) return fail(__LINE__)
int main() {
  const int64_t top = 2147483647;
  const int64_t values[] = {1, 2, 31, 4096, 1 << 30, top - 32, top - 1, top};
  const int64_t positions[] = {-32, -31, -2, -1, 0, 1, 31, 4095, 4096, 1 << 30, top - 1};
  for (int64_t w : values)
    for (int64_t pos : positions) {
      const int64_t low = pos - w;  // the rule in 64 bits: a row at pos >= 0 sees t > low
      const int64_t want = low > -1 ? low : -1;
      CHECK(mla::window_floor(static_cast<int32_t>(pos), static_cast<int32_t>(w)) == want);
    }
  for (int64_t L : {int64_t{0}, int64_t{1}, int64_t{100}, top - 64, top})
    for (int64_t w : values)
      for (int64_t s : {int64_t{0}, int64_t{1}, int64_t{64}, top})
        for (int bs : {16, 32, 64})
          for (int q : {1, 32})
            for (int causal : {0, 1}) {
              const mla::WindowView v = mla::window_view(static_cast<int32_t>(L), q, bs, causal, static_cast<int32_t>(w), static_cast<int32_t>(s));
              CHECK(v.n >= 0 && v.sa >= 0 && v.skip >= 0 && int64_t{v.n} + v.skip == L && v.sa % bs == 0 && v.skip % bs == 0);
            }
  const int32_t last = static_cast<int32_t>(top / 96);  // a tile of 96 that 2^31 - 1 tokens end in
  for (int t = 0; t < 128; ++t) CHECK(mla::run_position(last, 96, t) == static_cast<uint32_t>(int64_t{last} * 96 + t));
  CHECK(mla::run_position(last, 96, 127) > 2147483647u);
  std::printf("ok\n");
  return 0;
}
"""


def test_windows_and_tiles_at_the_ends_of_their_range(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or CUDA is None:
        pytest.skip("no g++ or no CUDA headers")
    src, exe = tmp_path / "bounds.cpp", str(tmp_path / "bounds")
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all", "-I", CSRC,
                    "-I", os.path.join(CUDA, "include"), "-I", os.path.join(os.path.dirname(os.path.dirname(CSRC)), "include"),
                    str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
