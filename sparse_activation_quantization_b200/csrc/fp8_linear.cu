// fp8_linear.cu - Y = X W of E4M3 operands with float32 scales per row and 128
// k of X and per 128 x 128 block of W:
//
//   Y[t][d] = sum_b xs[t][b] ws[d / 128][b] sum_{k in block b} x[t][k] w[d][k]
//
// The tensor cores sum the products of one 128-k block exactly as they are;
// each block's sum is then scaled and added in float32 registers.  Three
// kernels, chosen by shape (fp8_linear_plan):
//   stream  few rows: every weight byte goes from HBM to a register once and
//           into warp-level MMAs (m16n8k32), 16 weight rows per CTA, K split
//           over its warps.
//   tile    128 x 128 output tiles on tcgen05, K split over a cluster when the
//           tiles alone cannot fill the SMs.
//   pair    256 x 256 output tiles on CTA pairs (tcgen05 cta_group::2), a
//           persistent grid.
#include "fp8_stream.cuh"

namespace sharq {
namespace fp8 {

namespace {

struct LinearArgs {
  const uint8_t* x;   // [T][K]
  const float* xs;    // [blocks][lds]
  const uint8_t* w;   // [D][K]
  const float* ws;    // [D blocks][K blocks]
  void* y;
  long long ldy;
  int* err;
  int T, K, D, lds;
  int out_f32;
  int vec_y;          // rows of Y start on 16-byte boundaries
  int splits;
};

__device__ __forceinline__ void mbar_arrive_cta(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ------------------------------------------------------------ stream form ---
// Item = 16 weight rows; the CTA's eight warps share its K block by block and
// join their sums through shared memory.  A ring slot holds a unit of the
// weight, the same 128 k of the NT x 8 rows of X, and both scales.

constexpr int kStreamWarps = 8;
template <int NT>
struct Stream {
  static constexpr int kRing = NT == 1 ? 4 : 3;
  static constexpr int kX = kWeightUnit, kXs = kX + 1024 * NT, kWs = kXs + 32 * NT;
  static constexpr int kSlot = kWs + 16;
  static constexpr int kSmemBytes = kStreamWarps * kRing * kSlot;
};

template <int NT>
__global__ void __launch_bounds__(32 * kStreamWarps, 2) fp8_stream_kernel(const LinearArgs a) {
  using C = Stream<NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][kStreamWarps][16][8 * NT + 1];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int nkb = blocks_of(a.K), items = (a.D + 15) / 16;
  const uint32_t ring = smem_u32(smem) + warp * C::kRing * C::kSlot;
  // the next unit to load
  int li = blockIdx.x, lb = warp;
  const uint8_t *w0 = nullptr, *w1 = nullptr;
  const float* ws = nullptr;
  auto item = [&]() {
    const int d = li * 16 + g;  // rows past the last one read the last one and are not stored
    w0 = a.w + (size_t)min(d, a.D - 1) * a.K + 16 * q;
    w1 = a.w + (size_t)min(d + 8, a.D - 1) * a.K + 16 * q;
    ws = a.ws + (size_t)(li / 8) * nkb;
  };
  auto load = [&](uint32_t slot) {
    if (li < items && lb < nkb) {
      const int k = lb * kBlock, left = a.K - k - 16 * q;
      rows16_load(slot, w0 + k, w1 + k, left, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = 8 * n + g;
        const bool in = t < a.T;
        const uint8_t* x = a.x + (size_t)(in ? t : 0) * a.K + k + 16 * q;
        const uint32_t d = slot + C::kX + n * 1024 + lane * 16;
        copy16(d, left > 0 ? x : a.x, in && left > 0 ? 16u : 0u);
        copy16(d + 512, left > 64 ? x + 64 : a.x, in && left > 64 ? 16u : 0u);
      }
      if (lane < 2 * NT) {
        const int n = min(4, a.T - 4 * lane);
        copy16(slot + C::kXs + lane * 16, a.xs + (size_t)lb * a.lds + (n > 0 ? 4 * lane : 0), n > 0 ? 4u * n : 0u);
      } else if (lane == 2 * NT) {
        copy4(slot + C::kWs, ws + lb);
      }
      lb += kStreamWarps;
      if (lb >= nkb) {
        lb = warp;
        li += gridDim.x;
        if (li < items) item();
      }
    }
    copies_commit();
  };
  pdl_wait();
  item();
#pragma unroll
  for (int i = 0; i < C::kRing; ++i) load(ring + i * C::kSlot);
  uint32_t slot = ring;
  int buf = 0;
  for (int it = blockIdx.x; it < items; it += gridDim.x, buf ^= 1) {
    float acc[NT][4] = {};
    for (int b = warp; b < nkb; b += kStreamWarps) {
      copies_wait<C::kRing - 1>();
      __syncwarp();  // the scales come from other lanes' copies
      WeightUnit w;
      w.read(slot, lane);
      float s_w;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s_w) : "r"(slot + C::kWs) : "memory");
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t x = slot + C::kX + n * 1024 + lane * 16;
        float c[4];
        w.times(lds128(x), lds128(x + 512), c);
        const float2 s = lds_f2(slot + C::kXs + (8 * n + 2 * q) * 4);
        acc[n][0] = fmaf(c[0], s.x * s_w, acc[n][0]);
        acc[n][1] = fmaf(c[1], s.y * s_w, acc[n][1]);
        acc[n][2] = fmaf(c[2], s.x * s_w, acc[n][2]);
        acc[n][3] = fmaf(c[3], s.y * s_w, acc[n][3]);
      }
      __syncwarp();
      load(slot);
      slot = slot == ring + (C::kRing - 1) * C::kSlot ? ring : slot + C::kSlot;
    }
    auto& r = red[buf];  // two in turn: an item's readers are past it before the next but one writes it
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      r[warp][g][8 * n + 2 * q] = acc[n][0];
      r[warp][g][8 * n + 2 * q + 1] = acc[n][1];
      r[warp][g + 8][8 * n + 2 * q] = acc[n][2];
      r[warp][g + 8][8 * n + 2 * q + 1] = acc[n][3];
    }
    __syncthreads();
    if (threadIdx.x < 128 * NT) {
      const int t = threadIdx.x >> 4, d = threadIdx.x & 15;
      float s = r[0][d][t];
#pragma unroll
      for (int v = 1; v < kStreamWarps; ++v) s += r[v][d][t];
      if (t < a.T && it * 16 + d < a.D) {
        const size_t o = (size_t)t * a.ldy + it * 16 + d;
        if (a.out_f32)
          static_cast<float*>(a.y)[o] = s;
        else
          static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(s);
      }
    }
  }
  copies_wait<0>();
}

// -------------------------------------------------------------- tile form ---
// 128 x 128 output tile per CTA (or per cluster of S CTAs that share its K).
//   warp 0      producer: per 128-k block one box of X and one of W (16 KB
//               each, 128-byte swizzle) into a six-slot ring; rows and columns
//               past the operands' ends arrive as zeros
//   warp 1      TMEM allocation; one thread issues the block's four MMAs into
//               one of four 128-column TMEM buffers (the first overwrites it)
//   warps 4-11  each 128-k block: TMEM -> registers, acc += tmem * (xs * ws).
//               A thread holds one row and 64 columns.
// At the end the sums go through shared memory (the ring, free by then): with
// a cluster every CTA adds its share of the rows over all S partial tiles in
// rank order, so the result does not depend on timing.

struct Tile {
  static constexpr int BM = 128, BN = 128;
  static constexpr int kStages = 6;
  static constexpr int kStageBytes = 2 * 16384;
  static constexpr int kBufs = 4;
  static constexpr int kThreads = 384;
  static constexpr int kRowFloats = BN + 4;  // padded: conflict-free 16-byte access by row
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
  static_assert(BM * kRowFloats * 4 <= kStages * kStageBytes, "the sums must fit the ring");
};

__device__ __forceinline__ void consumer_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// one output value pair of four consecutive columns of a row
__device__ __forceinline__ void store_cols4(const LinearArgs& a, int row, int col, float4 v) {
  const size_t o = (size_t)row * a.ldy + col;
  if (a.out_f32) {
    float* y = static_cast<float*>(a.y) + o;
    if (a.vec_y && col + 4 <= a.D) {
      *reinterpret_cast<float4*>(y) = v;
    } else {
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < a.D) y[i] = e[i];
    }
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + o;
    if (a.vec_y && col + 4 <= a.D) {
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < a.D) y[i] = __float2bfloat16_rn(e[i]);
    }
  }
}

__global__ void __launch_bounds__(Tile::kThreads, 1)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap mapx, const __grid_constant__ CUtensorMap mapw,
                    const LinearArgs a) {
  using C = Tile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::kStages];
  __shared__ __align__(8) uint64_t empty_bar[C::kStages];
  __shared__ __align__(8) uint64_t acc_full[C::kBufs];
  __shared__ __align__(8) uint64_t acc_empty[C::kBufs];
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.splits;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int nt = blockIdx.y, mt = blockIdx.z;
  const int nkb = blocks_of(a.K);
  const int b0 = (int)((long long)rank * nkb / S), b1 = (int)((long long)(rank + 1) * nkb / S);
  const uint64_t deadline = globaltimer_ns() + kWaitNs;

  pdl_trigger();
  if (threadIdx.x == 0) {
    tma_prefetch_map(&mapx);
    tma_prefetch_map(&mapw);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);  // one arrival per consumer warp
    }
    fence_mbar_init();
    abort_sh = 0;
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (int b = b0; b < b1; ++b, ++i) {
        const int s = i % C::kStages;
        if (i >= C::kStages && !mbar_wait(&empty_bar[s], ((i / C::kStages) & 1) ^ 1, deadline, &abort_sh)) {
          record_error_word(a.err, kErrTimeoutWord);
          abort_sh = 1;
          break;
        }
        uint8_t* st = smem + s * C::kStageBytes;
        mbar_arrive_expect_tx(&full_bar[s], C::kStageBytes);
        tma_2d(st, &mapx, b * kBlock, mt * C::BM, &full_bar[s]);
        tma_2d(st + 16384, &mapw, b * kBlock, nt * C::BN, &full_bar[s]);
      }
      if (abort_sh) {  // copies in flight land before the CTA leaves
        const uint64_t lim = globaltimer_ns() + kWaitNs;
        for (int j = i > C::kStages ? i - C::kStages : 0; j < i; ++j)
          while (!mbar_try_wait(&full_bar[j % C::kStages], (j / C::kStages) & 1) && globaltimer_ns() < lim) {
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(C::BM, C::BN);
      for (int b = b0, i = 0; b < b1; ++b, ++i) {
        const int s = i % C::kStages, u = i % C::kBufs;
        if (!mbar_wait(&full_bar[s], (i / C::kStages) & 1, deadline, &abort_sh) ||
            (i >= C::kBufs && !mbar_wait(&acc_empty[u], ((i / C::kBufs) & 1) ^ 1, deadline, &abort_sh))) {
          record_error_word(a.err, kErrTimeoutWord);
          abort_sh = 1;
          break;
        }
        tc_fence_after();
        const uint32_t st = smem_u32(smem + s * C::kStageBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f8(tmem + u * C::BN, smem_desc(st + 32 * j, 16, 1024, kSw128),
                 smem_desc(st + 16384 + 32 * j, 16, 1024, kSw128), idesc, j > 0);
        tc_commit(&empty_bar[s]);
        tc_commit(&acc_full[u]);
      }
    }
  } else if (warp >= 4) {
    const int sp = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quarter; column half
    const int rl = sp * 32 + lane, row = mt * C::BM + rl;
    const uint32_t col0 = (uint32_t)half * 64;
    const float* xs = a.xs + min(row, a.T - 1);
    const float* ws = a.ws + (size_t)nt * nkb;
    float acc[64] = {};
    float s_next = b0 < b1 ? xs[(size_t)b0 * a.lds] * ws[b0] : 0.0f;
    for (int b = b0, i = 0; b < b1; ++b, ++i) {
      const int u = i % C::kBufs;
      const float s = s_next;
      if (b + 1 < b1) s_next = xs[(size_t)(b + 1) * a.lds] * ws[b + 1];
      if (!mbar_wait(&acc_full[u], (i / C::kBufs) & 1, deadline, &abort_sh)) {
        record_error_word(a.err, kErrTimeoutWord);
        abort_sh = 1;
        break;
      }
      tc_fence_after();
      uint32_t v[2][32];
      const uint32_t src = tmem + ((uint32_t)(sp * 32) << 16) + u * C::BN + col0;
      tmem_ld32(src, v[0]);
      tmem_ld32(src + 32, v[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&acc_empty[u]);
#pragma unroll
      for (int c = 0; c < 64; c += 2)
        fma2(acc[c], acc[c + 1], __uint_as_float(v[c >> 5][c & 31]), __uint_as_float(v[c >> 5][(c & 31) + 1]), s);
    }
    // the last block's sums were read, so every MMA has completed and with it
    // every use of the ring
    consumer_barrier();
    float* out = reinterpret_cast<float*>(smem) + rl * C::kRowFloats + col0;
#pragma unroll
    for (int c = 0; c < 64; c += 4) *reinterpret_cast<float4*>(out + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
  }
  if (S > 1)
    cluster_sync_all();  // every partial tile is in its CTA's shared memory
  else
    __syncthreads();
  if (warp >= 4 && !abort_sh) {
    const int valid = min(C::BM, a.T - mt * C::BM);
    const int per = (valid + S - 1) / S;
    const int r1 = min(valid, (rank + 1) * per);
    const uint32_t base = smem_u32(smem) + lane * 16;
    for (int r = rank * per + warp - 4; r < r1; r += 8) {
      float4 v;
      if (S == 1) {
        v = *reinterpret_cast<const float4*>(smem + (size_t)r * C::kRowFloats * 4 + lane * 16);
      } else {
        v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = 0; p < S; ++p) {
          const float4 o = ld_shared_cluster_f4(mapa_shared(base + r * C::kRowFloats * 4, (uint32_t)p));
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
      }
      store_cols4(a, mt * C::BM + r, nt * C::BN + lane * 4, v);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync_all();  // no CTA leaves while a peer reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------- pair form ---
// Two CTAs of a cluster run each 256 x 256 output tile as one tensor-core unit
// (M = 256): CTA r holds rows 128 r .. of X and columns 128 r .. of W, so each
// operand byte crosses from L2 once per 256 rows or columns of the other.
//   both CTAs  producer (warp 0): its own two boxes per 128-k block; their
//              bytes count on the even CTA's barrier
//              consumers (warps 4-11): its own 128 rows, a thread holds one row
//              and 128 columns (one weight-scale block) in registers
//   even CTA   MMA issuer (warp 1), two 256-column TMEM buffers; its commits
//              arrive on both CTAs' barriers
// The consumers take 224 registers (setmaxnreg), the other four warps keep 56:
// 256 x 224 + 128 x 56 = 384 x 168, the launch's registers.

struct Pair {
  static constexpr int BM = 256, BN = 256;
  static constexpr int kStages = 6;
  static constexpr int kStageBytes = 2 * 16384;
  static constexpr int kBufs = 2;
  static constexpr int kThreads = 384;
  static constexpr int kRegsLaunch = 168, kRegsConsumer = 224, kRegsOther = 56;
  static constexpr int kOffStage = kStages * kStageBytes;  // 4 KB of output staging per consumer warp
  static constexpr int kSmemBytes = kOffStage + 8 * 4096 + 1024;
  static_assert(kSmemBytes <= 232448 - 1024, "shared memory overflow");
  static_assert(2 * kRegsConsumer + kRegsOther <= 3 * kRegsLaunch, "register split above the launch's share");
};
__device__ __forceinline__ void regs_consumer() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory"); }
__device__ __forceinline__ void regs_other() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory"); }

// 32 rows (row = lane) x 32 four-byte words held in registers -> Y through the
// warp's 4 KB of shared memory, so that a warp stores whole 128-byte lines.
// kWords: output elements per word (2 for bf16, 1 for float32).
template <int kPer>
__device__ __forceinline__ void store_rows(const LinearArgs& a, uint8_t* wst, const uint32_t (&v)[32], int row0,
                                           int rows, int col0, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(wst + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  constexpr int kEl = 4 / kPer;  // bytes per element
  uint8_t* y = static_cast<uint8_t*>(a.y);
  if (a.vec_y && col0 + 32 * kPer <= a.D) {
    const int rsub = lane >> 3, q = lane & 7;
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int r = 4 * it + rsub;
      if (r < rows)
        *reinterpret_cast<uint4*>(y + ((size_t)(row0 + r) * a.ldy + col0) * kEl + 16 * q) =
            *reinterpret_cast<const uint4*>(wst + r * 128 + ((q ^ (r & 7)) << 4));
    }
  } else {
    for (int r = 0; r < rows && r < 32; ++r) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int c = lane + 32 * e;  // element of the row's 32 * kPer
        const int byte = c * kEl;
        const uint8_t* src = wst + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
        if (col0 + c < a.D) {
          uint8_t* dst = y + ((size_t)(row0 + r) * a.ldy + col0 + c) * kEl;
          if (kPer == 2)
            *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
          else
            *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
        }
      }
    }
  }
  __syncwarp();
}

__global__ void __launch_bounds__(Pair::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap mapx, const __grid_constant__ CUtensorMap mapw,
                    const LinearArgs a) {
  using C = Pair;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::kStages];   // even CTA: both CTAs' boxes have landed
  __shared__ __align__(8) uint64_t empty_bar[C::kStages];  // each CTA: its slot has been read
  __shared__ __align__(8) uint64_t acc_full[C::kBufs];     // each CTA
  __shared__ __align__(8) uint64_t acc_empty[C::kBufs];    // even CTA: both CTAs' consumers took the buffer
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nkb = blocks_of(a.K);
  const int m_tiles = (a.T + C::BM - 1) / C::BM, n_tiles = (a.D + C::BN - 1) / C::BN;
  const int ntiles = m_tiles * n_tiles;
  // the smaller operand is walked fastest, so that it stays in L2 while the
  // larger one streams past it once
  const bool m_fast = a.T <= a.D;
  auto coords = [&](int tile, int& mt, int& nt) {
    if (m_fast) {
      nt = tile / m_tiles;
      mt = tile - nt * m_tiles;
    } else {
      mt = tile / n_tiles;
      nt = tile - mt * n_tiles;
    }
  };

  pdl_trigger();
  if (threadIdx.x == 0) {
    tma_prefetch_map(&mapx);
    tma_prefetch_map(&mapw);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);  // 8 consumer warps of each CTA
    }
    fence_mbar_init();
    abort_sh = 0;
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers and TMEM exist before any pair traffic
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  pdl_wait();

  if (warp < 4) {
    regs_other();
    if (warp == 0 && lane == 0) {
      const uint32_t full_lead = mapa_shared(smem_u32(&full_bar[0]), 0);
      int i = 0;
      for (int tile = pair; tile < ntiles && !abort_sh; tile += npairs) {
        int mt, nt;
        coords(tile, mt, nt);
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        for (int b = 0; b < nkb; ++b, ++i) {
          const int s = i % C::kStages;
          if (i >= C::kStages && !mbar_wait_cluster(&empty_bar[s], ((i / C::kStages) & 1) ^ 1, deadline, &abort_sh)) {
            record_error_word(a.err, kErrTimeoutWord);
            abort_sh = 1;
            break;
          }
          uint8_t* st = smem + s * C::kStageBytes;
          if (leader) mbar_arrive_expect_tx(&full_bar[s], 2 * C::kStageBytes);  // both CTAs' boxes
          const uint32_t fb = full_lead + (uint32_t)(s * sizeof(uint64_t));
          tma_2d_pair(st, &mapx, b * kBlock, mt * C::BM + (int)rank * 128, fb);
          tma_2d_pair(st + 16384, &mapw, b * kBlock, nt * C::BN + (int)rank * 128, fb);
        }
      }
      // every slot's last use has been released (so its copies landed and the
      // commit's arrival on this CTA's barrier is in) before the CTA may leave
      const uint64_t lim = globaltimer_ns() + kWaitNs;
      for (int j = i > C::kStages ? i - C::kStages : 0; j < i; ++j)
        while (!mbar_try_wait_cluster(&empty_bar[j % C::kStages], (j / C::kStages) & 1) && globaltimer_ns() < lim) {
        }
    } else if (warp == 1 && lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_e4m3(C::BM, C::BN);
      int i = 0;
      for (int tile = pair; tile < ntiles && !abort_sh; tile += npairs) {
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        for (int b = 0; b < nkb; ++b, ++i) {
          const int s = i % C::kStages, u = i % C::kBufs;
          if (!mbar_wait_cluster(&full_bar[s], (i / C::kStages) & 1, deadline, &abort_sh) ||
              (i >= C::kBufs && !mbar_wait_cluster(&acc_empty[u], ((i / C::kBufs) & 1) ^ 1, deadline, &abort_sh))) {
            record_error_word(a.err, kErrTimeoutWord);
            abort_sh = 1;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * C::kStageBytes);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f8_pair(tmem + u * C::BN, smem_desc(st + 32 * j, 16, 1024, kSw128),
                        smem_desc(st + 16384 + 32 * j, 16, 1024, kSw128), idesc, j > 0);
          tc_commit_pair_mc(&empty_bar[s], 0x3);
          tc_commit_pair_mc(&acc_full[u], 0x3);
        }
      }
    }
  } else {
    regs_consumer();
    const int sp = warp & 3, half = (warp - 4) >> 2;
    const uint32_t acc_empty_lead = mapa_shared(smem_u32(&acc_empty[0]), 0);
    uint8_t* wst = smem + C::kOffStage + (size_t)(warp - 4) * 4096;
    const int d_blocks = blocks_of(a.D);
    int i = 0;
    for (int tile = pair; tile < ntiles && !abort_sh; tile += npairs) {
      int mt, nt;
      coords(tile, mt, nt);
      const uint64_t deadline = globaltimer_ns() + kWaitNs;
      const int row0 = mt * C::BM + (int)rank * 128 + sp * 32;
      const int nb = nt * 2 + half;  // this thread's weight-scale block
      const float* xs = a.xs + min(row0 + lane, a.T - 1);
      const float* ws = a.ws + (size_t)min(nb, d_blocks - 1) * nkb;
      float acc[128] = {};
      float s_next = xs[0] * ws[0];
      for (int b = 0; b < nkb; ++b, ++i) {
        const int u = i % C::kBufs;
        const float s = s_next;
        if (b + 1 < nkb) s_next = xs[(size_t)(b + 1) * a.lds] * ws[b + 1];
        if (!mbar_wait_cluster(&acc_full[u], (i / C::kBufs) & 1, deadline, &abort_sh)) {
          record_error_word(a.err, kErrTimeoutWord);
          abort_sh = 1;
          break;
        }
        tc_fence_after();
        const uint32_t src = tmem + ((uint32_t)(sp * 32) << 16) + u * C::BN + half * 128;
        uint32_t v[2][32];
        tmem_ld32(src, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // the next quarter loads while this one is added
          tmem_ld_wait();
          if (c < 3) tmem_ld32(src + 32 * (c + 1), v[(c + 1) & 1]);
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_lead + (uint32_t)(u * sizeof(uint64_t)));
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            fma2(acc[32 * c + e], acc[32 * c + e + 1], __uint_as_float(v[c & 1][e]), __uint_as_float(v[c & 1][e + 1]),
                 s);
        }
      }
      if (abort_sh) break;
      const int rows = a.T - row0;
      const int col0 = nt * C::BN + half * 128;
      if (rows > 0 && col0 < a.D) {
        if (a.out_f32) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(acc[32 * c + e]);
            store_rows<1>(a, wst, o, row0, rows, col0 + 32 * c, lane);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = pack_bf16x2(acc[64 * c + 2 * e], acc[64 * c + 2 * e + 1]);
            store_rows<2>(a, wst, o, row0, rows, col0 + 64 * c, lane);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA frees its TMEM or leaves while the pair's work may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The register split needs the launch to hold 384 x 168 registers; a build
// that was allotted fewer would wait for registers that never come.
bool pair_regs_ok() {
  static int ok = 0;  // 0 unknown, 1 yes, -1 no: a property of the build
  if (ok == 0) {
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, fp8_pair_kernel) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    ok = fa.numRegs >= Pair::kRegsLaunch ? 1 : -1;
  }
  return ok > 0;
}

}  // namespace

cudaError_t launch_linear(const uint8_t* x, const float* xs, int lds, int T, int K, const uint8_t* w, const float* ws,
                          int D, void* y, long long ldy, int out_f32, int* err, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const Device* dev = device();
  if (!dev) return cudaErrorInvalidDevice;
  LinearArgs a;
  a.x = x;
  a.xs = xs;
  a.w = w;
  a.ws = ws;
  a.y = y;
  a.ldy = ldy;
  a.err = err;
  a.T = T;
  a.K = K;
  a.D = D;
  a.lds = lds;
  a.out_f32 = out_f32;
  a.vec_y = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (ldy * (out_f32 ? 4 : 2)) % 16 == 0;
  a.splits = 1;
  if (T <= 16) {
    static bool done1[64] = {}, done2[64] = {};
    const bool one = T <= 8;
    const void* k = one ? (const void*)fp8_stream_kernel<1> : (const void*)fp8_stream_kernel<2>;
    const int smem = one ? Stream<1>::kSmemBytes : Stream<2>::kSmemBytes;
    cudaError_t e = opt_in_smem(k, smem, one ? done1 : done2);
    if (e != cudaSuccess) return e;
    void* args[] = {&a};
    const int items = (D + 15) / 16, most = 2 * dev->sms;
    return launch_pdl(k, dim3(items < most ? items : most), dim3(32 * kStreamWarps), smem, 1, stream, args);
  }
  CUtensorMap mx, mw;
  if (!byte_map(&mx, x, (uint64_t)T, (uint64_t)K, 128) || !byte_map(&mw, w, (uint64_t)D, (uint64_t)K, 128))
    return cudaErrorInvalidValue;
  void* args[] = {&mx, &mw, &a};
  const int nkb = blocks_of(K);
  const long long pair_tiles = (long long)((T + 255) / 256) * ((D + 255) / 256);
  if (pair_tiles * 2 >= dev->sms && pair_regs_ok()) {
    static bool done[64] = {};
    cudaError_t e = opt_in_smem((const void*)fp8_pair_kernel, Pair::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    const int pairs = (int)(pair_tiles < dev->sms / 2 ? pair_tiles : dev->sms / 2);
    return launch_pdl((const void*)fp8_pair_kernel, dim3(2 * pairs), dim3(Pair::kThreads), Pair::kSmemBytes, 2, stream,
                      args);
  }
  static bool done[64] = {};
  cudaError_t e = opt_in_smem((const void*)fp8_tile_kernel, Tile::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((T + 127) / 128) * ((D + 127) / 128);
  int s = (int)(dev->sms / tiles);
  s = s < 1 ? 1 : (s > 8 ? 8 : s);
  a.splits = s < nkb ? s : nkb;
  return launch_pdl((const void*)fp8_tile_kernel, dim3(a.splits, (D + 127) / 128, (T + 127) / 128),
                    dim3(Tile::kThreads), Tile::kSmemBytes, a.splits, stream, args);
}

}  // namespace fp8
}  // namespace sharq
