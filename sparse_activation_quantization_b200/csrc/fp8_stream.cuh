// fp8_stream.cuh - streaming E4M3 weights from HBM through warp-level MMAs, for
// the kernels that multiply a weight by a few columns only and are bound by
// reading it once.
//
// The unit is 16 weight rows x 128 k (2 KB, one weight-scale block).  A warp
// keeps a few units in flight in a ring of its own in shared memory: each lane
// copies the pieces that it will multiply itself (rows g and g + 8 of the MMA's
// A operand, 16 bytes of k per 64), so no barrier guards the ring and it keeps
// filling across work items.  The same k order serves A and B: within 64 k a
// lane of quad position q holds k = 16 q .. 16 q + 15, which m16n8k32 sums like
// any other order.
#pragma once
#include "fp8.cuh"

namespace sharq {
namespace fp8 {

constexpr int kWeightUnit = 2048;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  // fewer than 16 bytes: the rest is zeros and is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// Copy 16 rows (p0: this lane's row g, p1: row g + 8, both already at k = 16 q
// of the unit) into `slot`.  left: k from the lane's first byte to the row's
// end (multiples of 16; 0 or less: none).
__device__ __forceinline__ void rows16_load(uint32_t slot, const uint8_t* p0, const uint8_t* p1, int left, int lane) {
  const uint32_t n0 = left > 0 ? 16u : 0u, n1 = left > 64 ? 16u : 0u;
  const uint32_t d = slot + lane * 16;
  // nothing is read through a pointer past the row's end, but it stays inside it
  const int o0 = left > 0 ? 0 : left - 16, o1 = left > 64 ? 64 : o0;
  copy16(d, p0 + o0, n0);
  copy16(d + 512, p1 + o0, n0);
  copy16(d + 1024, p0 + o1, n1);
  copy16(d + 1536, p1 + o1, n1);
}

// this lane's A operand of a unit
struct WeightUnit {
  uint4 v[2][2];  // [64-k half][row half]
  __device__ __forceinline__ void read(uint32_t slot, int lane) {
    const uint32_t s = slot + lane * 16;
    v[0][0] = lds128(s);
    v[0][1] = lds128(s + 512);
    v[1][0] = lds128(s + 1024);
    v[1][1] = lds128(s + 1536);
  }
  // c (rows g, g + 8 x columns 2 q, 2 q + 1) = unit x eight columns, whose
  // bytes of the two 64-k halves are b0 and b1; two chains of dependent MMAs
  __device__ __forceinline__ void times(const uint4& b0, const uint4& b1, float (&c)[4]) const {
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    c[0] = c[1] = c[2] = c[3] = 0.0f;
    mma_e4m3(c, v[0][0].x, v[0][1].x, v[0][0].y, v[0][1].y, b0.x, b0.y);
    mma_e4m3(d, v[1][0].x, v[1][1].x, v[1][0].y, v[1][1].y, b1.x, b1.y);
    mma_e4m3(c, v[0][0].z, v[0][1].z, v[0][0].w, v[0][1].w, b0.z, b0.w);
    mma_e4m3(d, v[1][0].z, v[1][1].z, v[1][0].w, v[1][1].w, b1.z, b1.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += d[i];
  }
};

}  // namespace fp8
}  // namespace sharq
