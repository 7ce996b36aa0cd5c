"""Host threads that allow one kernel different amounts of shared memory at the same time: the larger
amount stays. The attribute is a variable here, and a thread is held inside its call."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <initializer_list>
#include <thread>
#include "smem_limit.h"

// The second thread asks while the first is inside its call, before or after the first's write.
static bool larger_stays(int first, int second, bool write_before) {
  std::atomic<int> allowed{0}, attribute{0};
  std::atomic<bool> inside{false}, done{false};
  std::mutex mu;
  std::thread a([&] {
    bskv::raise_smem_limit(allowed, mu, first, [&](int bytes) {
      if (write_before) attribute = bytes;
      inside = true;
      for (int i = 0; i < 200 && !done; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
      if (!write_before) attribute = bytes;
      return BSKV_OK;
    });
  });
  while (!inside) std::this_thread::yield();
  std::thread b([&] {
    bskv::raise_smem_limit(allowed, mu, second, [&](int bytes) {
      attribute = bytes;
      return BSKV_OK;
    });
    done = true;
  });
  a.join();
  b.join();
  return attribute == 131072 && allowed == 131072;
}

int main() {
  int bad = 0;
  for (bool before : {true, false}) {
    bad += !larger_stays(131072, 40960, before);
    bad += !larger_stays(40960, 131072, before);
  }
  // an error is passed on and leaves nothing allowed
  std::atomic<int> allowed{0};
  std::mutex mu;
  bad += bskv::raise_smem_limit(allowed, mu, 8, [](int) { return BSKV_ERR_CUDA; }) != BSKV_ERR_CUDA || allowed != 0;
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_the_larger_amount_stays(tmp_path):
    src = tmp_path / "limit.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I" + os.path.join(ROOT, "include"),
                    "-I" + os.path.join(ROOT, "block_sparse_kv_gb300", "csrc"), str(src), "-o", str(tmp_path / "limit")],
                   check=True)
    r = subprocess.run([str(tmp_path / "limit")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
