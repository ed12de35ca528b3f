// fp8.cuh - device helpers of the 8-bit (E4M3, block-scaled) path: format
// conversion, bounded waits, tensor-map copies and the 8-bit tcgen05 MMA; and
// what its launchers share.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sharq_device.cuh"

namespace sharq {
namespace fp8 {

constexpr int kBlock = 128;                 // elements (and weight columns) per scale
constexpr float kE4m3Max = 448.0f;
// Bound of a device-side wait, far beyond any tile's work.  Copy, MMA and forming warps count it from the start of the
// kernel (of the tile in the pair kernel; twice it in the expert layer's down, beside gate-up), sum warps from the start
// of each wait.  A kernel whose wait has run out leaves within a few of them.
constexpr uint64_t kWaitNs = 4000000000ull;
constexpr int kErrTimeoutWord = -5;          // SHARQ_ERR_TIMEOUT

__host__ __device__ __forceinline__ int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// s = max / 448 to nearest, at least the smallest normal float (so 1/s is
// finite), 1 for a block of zeros.  The quotient by Markstein's correction: q =
// max y with y = 1/448 to nearest, then q + (max - 448 q) y, whose remainder an
// FMA gives exactly.  (Where q is below the normal numbers the maximum takes
// over.)  A NaN in the block is skipped by the maximum and keeps its own code; an
// infinity makes s infinite and the block NaN.
__device__ __forceinline__ float block_scale_e4m3(float amax) {
  constexpr float y = 1.0f / kE4m3Max;
  const float q = amax * y;
  const float s = fmaxf(fmaf(fmaf(-kE4m3Max, q, amax), y, q), 0x1p-126f);
  return amax > 0.0f ? (amax < INFINITY ? s : amax) : 1.0f;
}

// four floats -> four E4M3 bytes, a in the lowest (round to nearest even,
// saturating; NaN -> 0x7F)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return out;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// silu(g) * u in float32: silu(g) = (g >= 0 ? g : g e^-|g|) / (1 + e^-|g|), so
// the divisor stays in [1, 2] and nothing overflows; silu(-inf) = -0
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = __expf(-fabsf(g));
  return __fdividef(g >= 0.0f ? g : fmaxf(g, -200.0f) * e, 1.0f + e) * u;
}

// Programmatic dependent launch.  wait: the preceding grid has completed and
// its memory is visible; trigger: the next grid may start its set-up.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// One thread of a whole warp, chosen by the hardware.  The compiler then knows
// that a single thread runs the branch and keeps MMA descriptors and copy
// coordinates in uniform registers: four MMAs and a commit issue in 214 cycles
// instead of the 455 of a branch on the lane number.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void record_error_word(int* err, int code) {
  if (err) atomicCAS(err, 0, code);
}

// two E4M3 bytes (low half of w) as floats (exact, through f16)
__device__ __forceinline__ float2 e4m3x2_to_float(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\t"
      "mov.b32 {l, u}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h)
      : "r"(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ void mbar_arrive_cta(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The same wait for loops that are short of registers: no 64-bit deadline is
// carried through them (70 cycles a wait).  The low half of the timer is read
// when the first try has run out, and kWaitNs lies below its period of 2^32 ns.
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool mbar_wait_short(uint64_t* bar, uint32_t parity, volatile int* abort) {
  static_assert(kWaitNs < 1ull << 32, "the bound in 32 bits");
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t start = globaltimer_lo();
  while (!mbar_try_wait(bar, parity))
    if (*abort || globaltimer_lo() - start > (uint32_t)kWaitNs) return false;
  return true;
}
// Whether the CTA has given up, the same answer for every lane: for loops of
// whole warps, whose shuffles and TMEM reads no lane may leave alone.
__device__ __forceinline__ bool warp_stopped(volatile int* abort) { return __any_sync(0xffffffffu, *abort); }
// whether the phase of parity `parity` is complete, without waiting for it
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// from shared memory of a CTA of the cluster
__device__ __forceinline__ float ld_shared_cluster_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_shared_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------- tensor-map copies ----

// 2-D tile (c0: element along the contiguous axis, c1: row) -> shared memory,
// bytes counted on `bar`
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// the same from a CTA of a pair: `bar_cluster` may be the other CTA's barrier
__device__ __forceinline__ void tma_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}
// 5-D tile -> shared memory
__device__ __forceinline__ void tma_5d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// shared memory -> 2-D tile, of which only what lies inside the map is written;
// part of this thread's bulk group
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
// every bulk store of this thread has been written
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// hint: bring a tile into L2.  Nothing is read into the program, so it may run
// before the preceding grid has completed.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(c0), "r"(c1)
               : "memory");
}

// ------------------------------------------------------- tcgen05, 8-bit ----

// Instruction descriptor of kind::f8f6f4: D float32 (1 in bits 4-5), A and B
// E4M3 (0 in bits 7-9 and 10-12), both K-major, N >> 3 in bits 17-22, M >> 4
// in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D(tmem) (+)= A(smem) x B(smem), K = 32
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// TMEM -> registers: this thread's lane, 16 or 8 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// two independent float32 multiply-adds in one instruction: d = a * b + d
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b) {
  asm("{\n\t.reg .b64 d, a, b;\n\t"
      "mov.b64 d, {%0, %1};\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %4};\n\t"
      "fma.rn.f32x2 d, a, b, d;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1), "f"(b));
}

// ----------------------------------------------------------- host side ----

// device properties that the launchers need, looked up once per device
struct Device {
  int sms = 0;
};
// nullptr if the current device cannot be used
const Device* device();
// a kernel's attribute that is set once per device: `done` is the kernel's own table
cudaError_t opt_in_smem(const void* kernel, int bytes, bool (&done)[64]);
// How many clusters of a kernel reside on the device at once, one CTA to an SM, asked once per device and cluster
// size: `known` is the kernel's own table.  SMs lie in groups of unequal size, and a cluster needs one group, so fewer
// may fit than the number of SMs says (15 of 8 on 148 SMs, 33 of 4); one that has to wait for a second wave doubles a
// short kernel's time.  (The query counts one CTA per SM for a kernel that allocates TMEM; where two reside, twice as
// many clusters do.)  0: could not be asked.
struct Resident {
  int n[64][9] = {};
};
int resident_clusters(const void* kernel, int threads, int smem, int cluster, Resident& known);
// launch with programmatic dependence on the preceding kernel, and a cluster along x
cudaError_t launch_pdl(const void* kernel, dim3 grid, dim3 block, int smem, int cluster, cudaStream_t stream,
                       void** args);
// tensor map of a row-major byte matrix [rows][cols] with 128-byte swizzle and
// a box of 128 columns x `box_rows` rows
bool byte_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);
// tensor map of rows of `cols` elements of 2 (bf16) or 4 (float32) bytes, `ld` elements apart, with 128-byte swizzle and
// a box of 128 bytes x `box_rows` rows; the base and the rows start on 16-byte boundaries
bool rows_map(CUtensorMap* map, void* base, uint64_t rows, uint64_t cols, uint64_t ld, int bytes, uint32_t box_rows);
// byte map of [E][2][rows][cols], rows a multiple of 16, as {cols, 16, 2, rows / 16, E}: a box of 128 columns and
// `box_rows` rows of both halves, 16 of one and 16 of the other in turn
bool halves_map(CUtensorMap* map, const void* base, uint64_t E, uint64_t rows, uint64_t cols, uint32_t box_rows);

}  // namespace fp8
}  // namespace sharq
