"""The library's launcher against a stand-in of the CUDA runtime (compiled here, no GPU): a launch
is judged by its own result, and leaves no error behind for the next call."""

import os
import subprocess

import pytest

from matrix_aware_optimizers_gb300 import _abi, build

# The runtime's part: what the next launch returns, and the last error.
RUNTIME = r"""
#include <cuda_runtime_api.h>

cudaError_t g_next = cudaSuccess, g_last = cudaSuccess;
int g_launches = 0, g_device = 0;

extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) {
  if (g_next != cudaSuccess) g_last = g_next;
  else ++g_launches;
  return g_next;
}
extern "C" cudaError_t cudaGetDevice(int* device) {
  *device = g_device;
  return cudaSuccess;
}
extern "C" cudaError_t cudaGetLastError(void) {
  const cudaError_t e = g_last;
  g_last = cudaSuccess;
  return e;
}
"""

PROGRAM = r"""
#include <cstdio>
#include "internal.h"

extern cudaError_t g_next, g_last;
extern int g_launches, g_device;
namespace mao {
void count_launch() {}
}

struct P { int x; };
static void kernel(const P) {}

static int launch(cudaError_t result) {
  g_next = result;
  return mao::launch_dependent(kernel, 1, 1, 0, nullptr, P{1});
}

int main() {
  std::printf("good %d\n", launch(cudaSuccess));
  g_last = cudaErrorInvalidValue;  // left by other code
  std::printf("after another's error %d\n", launch(cudaSuccess));
  std::printf("its own error %d\n", launch(cudaErrorInvalidConfiguration));
  std::printf("after its own error %d\n", launch(cudaSuccess));
  g_last = cudaSuccess;
  std::printf("its own error %d\n", launch(cudaErrorInvalidConfiguration));
  std::printf("left behind %d\n", int(g_last));
  std::printf("launches %d\n", g_launches);
  // what a device is set up with: tried again after a failure, and once for each device
  static std::atomic<bool> ready[64];
  int calls = 0;
  auto once = [&](cudaError_t result) {
    g_last = result;
    return mao::once_per_device(ready, [&] { return ++calls, result; });
  };
  const int first = once(cudaErrorInvalidValue), pending = int(g_last);
  const int second = once(cudaSuccess), third = once(cudaSuccess);
  g_device = 1;
  const int other = once(cudaSuccess);
  std::printf("set up %d %d %d %d %d calls %d\n", first, pending, second, third, other, calls);
}
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    for name, text in (("runtime.cpp", RUNTIME), ("launch.cu", PROGRAM)):
        with open(str(d / name), "w") as f:
            f.write(text)
    exe = str(d / "launch")
    cmd = [build.nvcc()] + build.ARCH + ["-std=c++17", "-cudart", "shared", "-I", build.INCLUDE, "-I", build.CSRC,
                                         "-o", exe, str(d / "launch.cu"), str(d / "runtime.cpp")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    libs = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "lib64")
    env = dict(os.environ, LD_LIBRARY_PATH=libs)
    return subprocess.run([exe], capture_output=True, text=True, check=True, env=env).stdout.splitlines()


def test_a_launch_is_judged_by_its_own_result(answers):
    ok, failed = str(_abi.MAO_OK), str(_abi.MAO_ERR_CUDA)
    assert answers[0] == "good " + ok
    assert answers[1] == "after another's error " + ok
    assert answers[2] == "its own error " + failed
    assert answers[3] == "after its own error " + ok
    assert answers[6] == "launches 3"


def test_a_failed_launch_leaves_no_error(answers):
    assert answers[4] == "its own error %d" % _abi.MAO_ERR_CUDA and answers[5] == "left behind 0"


def test_setting_up_a_device_is_tried_again_after_a_failure(answers):
    assert answers[7] == "set up %d 0 0 0 0 calls 3" % _abi.MAO_ERR_CUDA
