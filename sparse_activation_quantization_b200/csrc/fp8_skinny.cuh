// fp8_skinny.cuh - an E4M3 weight times a few columns on tcgen05, bound by
// reading the weight from HBM once.
//
// The weight is the MMA's A operand: a unit is 128 weight rows x 128 k (16 KB,
// one weight-scale block along k) and the few activation columns are B (N =
// 16 .. 96).  A ring of stages holds units in flight; stage s has its own N
// columns of TMEM, so one set of barriers guards both:
//   full[s]   the unit has landed: the copy thread's bytes and, where the
//             columns are formed on the fly, one arrival per forming warp
//   done[s]   its four MMAs (K = 32 each) have completed
//   empty[s]  the four sum warps have read the stage's TMEM and scales
// Per unit every sum thread (one weight row) reads N values, scales them in
// float32 and adds them to its registers.  A unit's four MMAs take 214 to 260
// cycles whatever N is, its sums 500 to 600 (waits and latencies, not arithmetic),
// and its bytes 370 ns (700 cycles) of the HBM rate's share of an SM.  One CTA
// on an SM reaches three quarters of that rate, two reach it: 152000 x 4096
// against one row in 93.7 us, 6650 GB/s.  (Warp-level MMAs fed by per-lane
// copies reached 2.4 TB/s.)
#pragma once
#include "fp8.cuh"

namespace sharq {
namespace fp8 {

constexpr int kUnitRows = 128;
constexpr int kUnitBytes = kUnitRows * kBlock;
constexpr int kSumWarps = 4;  // warps 0-3: TMEM lanes 32 w .. 32 w + 31 belong to warp w

constexpr int tmem_cols(int n) {  // allocations are powers of two, 32 at least
  int c = 32;
  while (c < n) c *= 2;
  return c;
}

template <int kStages>
struct SkinnyBars {
  uint64_t full[kStages], done[kStages], empty[kStages];
  uint32_t tmem;
  volatile int abort;
  __device__ __forceinline__ void init(int full_arrivals, int done_arrivals) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], full_arrivals);
      mbar_init(&done[s], done_arrivals);
      mbar_init(&empty[s], kSumWarps);
    }
    fence_mbar_init();
    abort = 0;
  }
  __device__ __forceinline__ void give_up(int* err) {
    record_error_word(err, kErrTimeoutWord);
    abort = 1;
  }
};

// position of a unit in the ring
template <int kStages>
struct RingPos {
  int s = 0;
  uint32_t phase = 0;
  bool wrapped = false;  // the stage has been used before
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      phase ^= 1u;
      wrapped = true;
    }
  }
};

// The copy thread's wait for a free stage
template <int kStages>
__device__ __forceinline__ bool wait_empty(SkinnyBars<kStages>& b, const RingPos<kStages>& p, uint64_t deadline) {
  return !p.wrapped || mbar_wait(&b.empty[p.s], p.phase ^ 1u, deadline, &b.abort);
}

// A sum warp's wait for a unit: its scales are visible and its MMAs complete.
// The answer is the same for the whole warp.
template <int kStages>
__device__ __forceinline__ bool wait_done(SkinnyBars<kStages>& b, const RingPos<kStages>& p, uint64_t deadline) {
  const bool ok = mbar_wait(&b.full[p.s], p.phase, deadline, &b.abort) &&
                  mbar_wait(&b.done[p.s], p.phase, deadline, &b.abort);
  if (!__all_sync(0xffffffffu, ok)) return false;
  tc_fence_after();
  return true;
}
template <int kStages>
__device__ __forceinline__ void release_unit(SkinnyBars<kStages>& b, const RingPos<kStages>& p, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive_cta(&b.empty[p.s]);
}

// After a wait has run out: copies in flight land before the CTA leaves.  n: units
// issued so far.
template <int kStages>
__device__ __forceinline__ void drain_copies(SkinnyBars<kStages>& b, int n) {
  const uint64_t lim = globaltimer_ns() + kWaitNs;
  for (int j = n > kStages ? n - kStages : 0; j < n; ++j)
    while (!mbar_try_wait(&b.full[j % kStages], (j / kStages) & 1) && globaltimer_ns() < lim) {
    }
}

// One unit's MMAs: A at `a_smem`, B right behind it
__device__ __forceinline__ void unit_mma(uint32_t d, uint32_t a_smem, uint32_t idesc) {
#pragma unroll
  for (int j = 0; j < kBlock / 32; ++j)
    mma_f8(d, smem_desc(a_smem + 32 * j, 16, 1024, kSw128), smem_desc(a_smem + kUnitBytes + 32 * j, 16, 1024, kSw128),
           idesc, j > 0);
}

// N consecutive TMEM columns of this thread's lane
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t addr, uint32_t (&v)[N]) {
  static_assert(N % 8 == 0, "columns");
  constexpr int n32 = N / 32;
#pragma unroll
  for (int i = 0; i < n32; ++i) tmem_ld32(addr + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * i]));
  if (N % 32 >= 16) tmem_ld16(addr + 32 * n32, &v[32 * n32]);
  if (N % 16 >= 8) tmem_ld8(addr + (N / 16) * 16, &v[(N / 16) * 16]);
}

// A weight row's scales along k, 32 blocks at a time: lane l holds block base + l
struct ScaleRow {
  const float* p;  // the row of scales
  int n, base;
  float cur, ahead;
  __device__ __forceinline__ float load(int b) const { return b < n ? p[b] : 0.0f; }
  __device__ __forceinline__ void start(const float* row, int blocks, int b0, int lane) {
    p = row;
    n = blocks;
    base = b0;
    cur = load(b0 + lane);
    ahead = load(b0 + 32 + lane);
  }
  __device__ __forceinline__ float at(int b, int lane) {  // b ascends
    if (b - base >= 32) {
      base += 32;
      cur = ahead;
      ahead = load(base + 32 + lane);
    }
    return __shfl_sync(0xffffffffu, cur, b - base);
  }
};

}  // namespace fp8
}  // namespace sharq
