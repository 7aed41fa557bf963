"""Host helpers of the launches, compiled with g++ against the stand-in CUDA
runtime of the executor's dry run: what is kept per device, and what is not."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "micro_pipeline_re_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "launch_util.cuh"

static int device = 0, asked = 0;
static cudaError_t device_rc = cudaSuccess;
cudaError_t cudaGetDevice(int* dev) {
  *dev = device;
  return device_rc;
}
#define EXPECT(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

int main() {
  static gp::PerDevice<4> counts;
  const cudaError_t bad = static_cast<cudaError_t>(1);
  int n = 0;
  auto answer = [&](int value, cudaError_t rc = cudaSuccess) {
    return [=](int* out) { ++asked; *out = value; return rc; };
  };
  // a query that fails is reported, not remembered
  EXPECT(counts.get(2, answer(5, bad), &n) == bad && asked == 1);
  EXPECT(counts.get(2, answer(7), &n) == cudaSuccess && n == 7 && asked == 2);
  EXPECT(counts.get(2, answer(9), &n) == cudaSuccess && n == 7 && asked == 2);
  // an answer of nothing is a failure as well
  EXPECT(counts.get(3, answer(0), &n) != cudaSuccess && asked == 3);
  EXPECT(counts.get(3, answer(4), &n) == cudaSuccess && n == 4 && asked == 4);
  // another key, another device
  EXPECT(counts.get(1, answer(6), &n) == cudaSuccess && n == 6 && asked == 5);
  device = 1;
  EXPECT(counts.get(2, answer(11), &n) == cudaSuccess && n == 11 && asked == 6);
  device = 0;
  EXPECT(counts.get(2, answer(12), &n) == cudaSuccess && n == 7 && asked == 6);
  // a device beyond those that are kept, and one that cannot be told
  device = 64;
  EXPECT(counts.get(2, answer(13), &n) == cudaSuccess && n == 13 && asked == 7);
  EXPECT(counts.get(2, answer(14), &n) == cudaSuccess && n == 14 && asked == 8);
  device = 0;
  device_rc = bad;
  EXPECT(counts.get(2, answer(15), &n) == cudaSuccess && n == 15 && asked == 9);
  return 0;
}
"""


def test_answers_are_kept_by_device_and_only_when_they_succeed(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(HERE, "dryrun"), "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_streamed_distillation_keeps_its_clusters_that_way():
    """No answer in a variable without the device."""
    with open(os.path.join(CSRC, "distill.cu")) as f:
        src = f.read()
    assert "PerDevice<kMaxCluster + 1>" in src and "static std::atomic<int>" not in src
