"""Bounded waits of the 8-bit kernels that run out (GPU).

A one-CTA kernel is compiled here from the kernels' own headers.  Its warp waits
on a barrier that nothing ever arrives on, with nothing else in flight: the wait
ends by its bound, records the timeout in the error word that sharq_check_status
reads, and the kernel ends as a warp.  No fault, trap or endless loop is involved.
"""
import ctypes
import os
import subprocess

import pytest
import torch

import sparse_activation_quantization_b200 as sq
from sparse_activation_quantization_b200 import build
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu
SHARQ_ERR_TIMEOUT = -5
NOBODY, GAVE_UP, LATE = 0, 1, 2

SOURCE = r"""
#include "fp8_skinny.cuh"
using namespace sharq;
using namespace sharq::fp8;
constexpr int kGaveUp = 1, kLate = 2;

// out: lanes whose wait ended well, lanes that saw the warp stop, the nanoseconds it took
__global__ void wait_kernel(int what, int* err, unsigned long long* out) {
  __shared__ SkinnyBars<2> bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bars.init(1, 1);
    if (what == kGaveUp) bars.give_up(err);
  }
  __syncthreads();
  if (warp == 0) {
    const uint64_t start = globaltimer_ns();
    const bool ok = mbar_wait_short(&bars.full[0], 0, &bars.abort);
    if (!ok) bars.give_up(err);
    __syncwarp();
    const uint64_t took = globaltimer_ns() - start;
    const int well = __popc(__ballot_sync(0xffffffffu, ok));
    const int stopped = __popc(__ballot_sync(0xffffffffu, warp_stopped(&bars.abort)));
    if (lane == 0) {
      out[0] = well;
      out[1] = stopped;
      out[2] = took;
    }
  } else if (what == kLate && lane == 0) {  // arrives after 20 ms
    const uint64_t start = globaltimer_ns();
    while (globaltimer_ns() - start < 20000000ull) {
    }
    mbar_arrive_cta(&bars.full[0]);
  }
}
extern "C" int launch(int what, int* err, unsigned long long* out, void* stream) {
  wait_kernel<<<1, 64, 0, (cudaStream_t)stream>>>(what, err, out);
  return cudaGetLastError();
}
extern "C" double bound_ns() { return (double)kWaitNs; }
"""


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    H.ensure_built()
    d = tmp_path_factory.mktemp("waits")
    src, lib = d / "waits.cu", d / "waits.so"
    src.write_text(SOURCE)
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-shared", str(src), "-o", str(lib)],
                   check=True)
    L = ctypes.CDLL(os.fspath(lib))
    L.bound_ns.restype = ctypes.c_double
    L.launch.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]

    def run(what):
        ws, out = sq.Fp8Workspace(256), torch.zeros(3, dtype=torch.int64, device="cuda")
        assert L.launch(what, ws.ptr, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        status = ws.check()
        assert ws.check() == 0  # reading the error word clears it
        return (*out.tolist(), status, L.bound_ns())

    return run


def test_wait_that_runs_out_ends_and_is_reported(probe):
    well, stopped, took, status, bound = probe(NOBODY)
    assert well == 0 and stopped == 32 and status == SHARQ_ERR_TIMEOUT
    assert bound <= took < bound + 2e9  # lanes give up within one try of the first


def test_wait_ends_at_once_after_another_warp_gave_up(probe):
    well, stopped, took, status, bound = probe(GAVE_UP)
    assert well == 0 and stopped == 32 and status == SHARQ_ERR_TIMEOUT and took < 0.1 * bound


def test_wait_outlasts_a_late_arrival(probe):
    well, stopped, took, status, bound = probe(LATE)
    assert well == 32 and stopped == 0 and status == 0 and took >= 19e6
