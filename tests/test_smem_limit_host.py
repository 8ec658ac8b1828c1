"""The shared-memory limit of a kernel instance (pd_smem_limit.h) under many
host threads, against a stand-in for the attribute that a call sets: what a
thread asked for stays allowed."""

import ctypes
import os
import shutil
import subprocess

import pytest

from paged_split_kv_02_gb300 import _build

BODY = r"""
#include "pd_smem_limit.h"
#include <chrono>
#include <random>
#include <thread>
#include <vector>

struct Instance {
  pd::SmemLimit limit;
  std::atomic<int> attribute[2] = {};   // of the device
  std::atomic<int> calls{0};
  int raise(int dev, int bytes, int pause_us, int error = 0) {
    return limit.raise(dev, bytes, [&](int b) {
      ++calls;
      std::this_thread::sleep_for(std::chrono::microseconds(pause_us));
      if (error) return error;
      attribute[dev] = b;
      return 0;
    });
  }
};

extern "C" int launches_refused(int threads, int rounds) {
  std::atomic<int> refused{0};
  for (int r = 0; r < rounds; ++r) {
    Instance it;
    std::vector<std::thread> t;
    for (int k = 0; k < threads; ++k)
      t.emplace_back([&, k] {
        std::mt19937 g(r * 1000 + k);
        for (int i = 0; i < 6; ++i) {
          const int dev = (int)(g() % 2), bytes = 1000 * (1 + (int)(g() % 200));
          if (it.raise(dev, bytes, (int)(g() % 60)) != 0) ++refused;
          std::this_thread::sleep_for(std::chrono::microseconds(g() % 60));
          if (it.attribute[dev] < bytes) ++refused;   // the launch
        }
      });
    for (auto &x : t) x.join();
  }
  return refused;
}

extern "C" int one_thread() {
  Instance it;
  if (it.raise(0, 100, 0) || it.attribute[0] != 100 || it.calls != 1) return 1;
  if (it.raise(0, 100, 0) || it.raise(0, 7, 0) || it.calls != 1) return 2;      // allowed already
  if (it.raise(1, 50, 0) || it.attribute[1] != 50 || it.calls != 2) return 3;   // another device
  if (it.raise(0, 300, 0, 9) != 9 || it.attribute[0] != 100) return 4;          // the call's error
  if (it.raise(0, 300, 0) || it.attribute[0] != 300) return 5;                  // asked again after it
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("smem")
    src, path = str(d / "limit.cpp"), str(d / "limit.so")
    with open(src, "w") as f:
        f.write(BODY)
    subprocess.run([shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread",
                    "-I" + _build.CSRC, src, "-o", path], check=True)
    return ctypes.CDLL(path)


def test_limits_of_one_thread(lib):
    assert lib.one_thread() == 0


def test_limits_of_many_threads(lib):
    assert lib.launches_refused(8, 60) == 0


def test_every_launcher_takes_it():
    for name in sorted(os.listdir(_build.CSRC)):
        text = open(os.path.join(_build.CSRC, name)).read()
        if "cudaFuncAttributeMaxDynamicSharedMemorySize" in text:
            assert name == "pd_internal.h"
