// fp8_linear.cu - Y = X W of E4M3 operands with float32 scales per row and 128
// k of X and per 128 x 128 block of W:
//
//   Y[t][d] = sum_b xs[t][b] ws[d / 128][b] sum_{k in block b} x[t][k] w[d][k]
//
// The tensor cores sum the products of one 128-k block exactly as they are;
// each block's sum is then scaled and added in float32 registers.  Three
// kernels, chosen by shape (launch_linear):
//   skinny  up to 64 rows: 128 weight rows are the MMA's M and the rows of X its
//           N (fp8_skinny.cuh), K split over a cluster.
//   tile    128 x 128 output tiles on tcgen05, K split over a cluster when the
//           tiles alone cannot fill the SMs.
//   pair    256 x 256 output tiles on CTA pairs (tcgen05 cta_group::2), a
//           persistent grid.
#include "fp8_skinny.cuh"

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

// four consecutive columns of a row
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

// Sum in rank order of four floats at the same place of S <= 8 CTAs' shared
// memory; every load is on its way before the first sum.
__device__ __forceinline__ float4 sum_over_cluster(uint32_t addr, int S) {
  float4 o[8], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int p = 0; p < 8; ++p)
    if (p < S) o[p] = ld_shared_cluster_f4(mapa_shared(addr, (uint32_t)p));
#pragma unroll
  for (int p = 0; p < 8; ++p)
    if (p < S) {
      v.x += o[p].x;
      v.y += o[p].y;
      v.z += o[p].z;
      v.w += o[p].w;
    }
  return v;
}

// ------------------------------------------------------------ skinny form ---
// 128 weight rows per CTA (or per cluster of S CTAs that share its K) against
// all rows of X at once, as fp8_skinny.cuh describes.
//   warps 0-3  sums: a thread holds one weight row and every row of X
//   warp 4     one thread copies: the weight's box, X's box and the rows'
//              scales of the block
//   warp 5     TMEM allocation; one thread issues the MMAs
// Two CTAs reside on an SM, so one's start and end hide behind the other's
// copies.  A cluster joins its partial sums in rank order over distributed
// shared memory (the ring, free by then).

template <int kN>
struct Skinny {
  static constexpr int kStages = kN == 16 ? 6 : (kN == 32 ? 5 : 4);
  static constexpr int kStageBytes = kUnitBytes + kN * kBlock;
  static constexpr int kThreads = 192;
  static constexpr int kTmem = tmem_cols(kN * kStages);
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
  static_assert(kN * kUnitRows * 4 <= kStages * kStageBytes, "the sums must fit the ring");
  static_assert(2 * kTmem <= 512, "two CTAs share the SM's TMEM");
};

__device__ __forceinline__ void store_one(const LinearArgs& a, size_t o, float v) {
  if (a.out_f32)
    static_cast<float*>(a.y)[o] = v;
  else
    static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
}

template <int kN>
__global__ void __launch_bounds__(Skinny<kN>::kThreads, 2)
    fp8_skinny_kernel(const __grid_constant__ CUtensorMap mapx, const __grid_constant__ CUtensorMap mapw,
                      const LinearArgs a) {
  using C = Skinny<kN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) SkinnyBars<C::kStages> bars;
  __shared__ __align__(16) float xs_sh[C::kStages][kN];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.splits;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / S, step = (int)gridDim.x / S;
  const int tiles = (a.D + kUnitRows - 1) / kUnitRows, nkb = blocks_of(a.K);
  const int b0 = (int)((long long)rank * nkb / S), b1 = (int)((long long)(rank + 1) * nkb / S);

  if (threadIdx.x == 128) {
    tma_prefetch_map(&mapx);
    tma_prefetch_map(&mapw);
    bars.init(1, 1);
    for (int i = 0; i < C::kStages && b0 + i < b1; ++i)
      tma_prefetch_2d(&mapw, (b0 + i) * kBlock, first * kUnitRows);
  }
  if (warp == 5) {
    tmem_alloc(&bars.tmem, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // after the allocation: the next grid's CTAs wait for this one with TMEM in hand
  pdl_wait();
  const uint32_t tmem = bars.tmem;
  const uint64_t deadline = globaltimer_ns() + kWaitNs;
  float acc[kN];

  if (warp == 4) {
    if (elect_one()) {
      // scales are read in whole 16-byte groups of a column, whose length is a multiple of 4
      const uint32_t xs_bytes = (uint32_t)(a.T + 3) / 4 * 16;
      RingPos<C::kStages> p;
      int n = 0;
      for (int tile = first; tile < tiles && !bars.abort; tile += step)
        for (int b = b0; b < b1; ++b, ++n, p.next()) {
          if (!wait_empty(bars, p, deadline)) {
            bars.give_up(a.err);
            break;
          }
          uint8_t* st = smem + p.s * C::kStageBytes;
          mbar_arrive_expect_tx(&bars.full[p.s], C::kStageBytes + xs_bytes);
          tma_2d(st, &mapw, b * kBlock, tile * kUnitRows, &bars.full[p.s]);
          tma_2d(st + kUnitBytes, &mapx, b * kBlock, 0, &bars.full[p.s]);
          bulk_g2s(xs_sh[p.s], a.xs + (size_t)b * a.lds, xs_bytes, &bars.full[p.s]);
        }
      if (bars.abort) drain_copies(bars, n);
    }
  } else if (warp == 5) {
    if (elect_one()) {
      RingPos<C::kStages> p;
      bool ready = false;  // the next unit had landed when it was asked for, before the MMAs ahead of it
      for (int tile = first; tile < tiles && !bars.abort; tile += step)
        for (int b = b0; b < b1; ++b) {
          if (!ready && !mbar_wait(&bars.full[p.s], p.phase, deadline, &bars.abort)) {
            bars.give_up(a.err);
            break;
          }
          const int s = p.s;
          p.next();
          ready = mbar_test(&bars.full[p.s], p.phase);
          tc_fence_after();
          unit_mma(tmem + s * kN, smem_u32(smem + s * C::kStageBytes), idesc_e4m3(kUnitRows, kN));
          tc_commit(&bars.done[s]);
        }
    }
  } else {
    RingPos<C::kStages> p;
    for (int tile = first; tile < tiles && !warp_stopped(&bars.abort); tile += step) {
      ScaleRow ws;
      ws.start(a.ws + (size_t)tile * nkb, nkb, b0, lane);
#pragma unroll
      for (int n = 0; n < kN; ++n) acc[n] = 0.0f;
      for (int b = b0; b < b1; ++b, p.next()) {
        const float s_w = ws.at(b, lane);
        if (!wait_done(bars, p, deadline)) {
          bars.give_up(a.err);
          break;
        }
        uint32_t v[kN];
        tmem_read(tmem + ((uint32_t)(warp * 32) << 16) + p.s * kN, v);
        tmem_ld_wait();
#pragma unroll
        for (int n = 0; n < kN; n += 4) {
          const float4 x = *reinterpret_cast<const float4*>(&xs_sh[p.s][n]);
          acc[n] = fmaf(__uint_as_float(v[n]), x.x * s_w, acc[n]);
          acc[n + 1] = fmaf(__uint_as_float(v[n + 1]), x.y * s_w, acc[n + 1]);
          acc[n + 2] = fmaf(__uint_as_float(v[n + 2]), x.z * s_w, acc[n + 2]);
          acc[n + 3] = fmaf(__uint_as_float(v[n + 3]), x.w * s_w, acc[n + 3]);
        }
        release_unit(bars, p, lane);
      }
      const int d = tile * kUnitRows + threadIdx.x;
      if (S == 1 && d < a.D && !bars.abort) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
          if (n < a.T) store_one(a, (size_t)n * a.ldy + d, acc[n]);
      }
    }
    if (S > 1) {  // one tile per cluster; its last sums were read, so the ring is free
      asm volatile("bar.sync 1, 128;" ::: "memory");
      float* out = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int n = 0; n < kN; ++n)
        if (n < a.T) out[n * kUnitRows + threadIdx.x] = acc[n];
    }
  }
  if (S > 1) {
    cluster_sync_all();  // every partial tile is in its CTA's shared memory
    const uint32_t base = smem_u32(smem);
    const int total = a.T * (kUnitRows / 4);
    const int i1 = (rank + 1) * total / S;
    for (int i = rank * total / S + (int)threadIdx.x; i < i1 && !bars.abort; i += C::kThreads) {
      const float4 v = sum_over_cluster(base + i * 16, S);
      store_cols4(a, i / (kUnitRows / 4), first * kUnitRows + i % (kUnitRows / 4) * 4, v);
    }
    cluster_sync_all();  // no CTA leaves while a peer reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

template <int kN>
cudaError_t launch_skinny(LinearArgs& a, const Device* dev, cudaStream_t stream) {
  using C = Skinny<kN>;
  CUtensorMap mx, mw;
  if (!byte_map(&mx, a.x, (uint64_t)a.T, (uint64_t)a.K, kN) ||
      !byte_map(&mw, a.w, (uint64_t)a.D, (uint64_t)a.K, kUnitRows))
    return cudaErrorInvalidValue;
  static bool done[64] = {};
  cudaError_t e = opt_in_smem((const void*)fp8_skinny_kernel<kN>, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const int tiles = (a.D + kUnitRows - 1) / kUnitRows, most = 2 * dev->sms, nkb = blocks_of(a.K);
  // The widest cluster with which all reside at once: a CTA per SM, or a second one where each then still has 16
  // units or more.  Measured: 28 tiles of 148 blocks 15.8 us at one, 14.5 at two; 36 tiles of 28 blocks 6.5 and 9.9.
  static Resident known;
  int s = 8;
  for (; s > 1; --s) {
    if (s > nkb || s * tiles > (nkb >= 16 * s ? most : dev->sms)) continue;
    if (2 * resident_clusters((const void*)fp8_skinny_kernel<kN>, C::kThreads, C::kSmemBytes, s, known) >= tiles) break;
  }
  a.splits = s;
  void* args[] = {&mx, &mw, &a};
  const int grid = a.splits > 1 ? tiles * a.splits : (tiles < most ? tiles : most);
  return launch_pdl((const void*)fp8_skinny_kernel<kN>, dim3(grid), dim3(C::kThreads), C::kSmemBytes, a.splits, stream,
                    args);
}

// Scales of a row's next four blocks, on their way while four are added:
// everything that goes through the load path is slow beside the MMAs' operand
// reads, and a load (and a shuffle) per block took 300 cycles of it.
struct ScaleGroup {
  static constexpr int kBlocks = 4;
  const float *xs, *ws;  // the row's column of X's scales, the tile's row of W's
  int lds, end;
  float nx[kBlocks], nw[kBlocks];
  __device__ __forceinline__ void load(int b0) {
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const int b = min(b0 + j, end - 1);
      nx[j] = xs[(size_t)b * lds];
      nw[j] = ws[b];
    }
  }
  // blocks b0 .. b1 - 1, at least one
  __device__ __forceinline__ void start(const float* x, int ld, const float* w, int b0, int b1) {
    xs = x, ws = w, lds = ld, end = b1;
    load(b0);
  }
  // the products of blocks b .. b + 3; the next four are asked for
  __device__ __forceinline__ void take(float (&s)[kBlocks], int b) {
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) s[j] = nx[j] * nw[j];
    if (b + kBlocks < end) load(b + kBlocks);
  }
};

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
  pdl_trigger();  // after the allocation: the next grid's CTAs wait for this one with TMEM in hand
  pdl_wait();
  const uint64_t deadline = globaltimer_ns() + kWaitNs;

  if (warp == 0) {
    if (elect_one()) {
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
    if (elect_one()) {
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
    ScaleGroup sg;
    sg.start(a.xs + min(row, a.T - 1), a.lds, a.ws + (size_t)nt * nkb, b0, b1);
    float acc[64] = {};
    bool seen = false;  // the next buffer was full when it was asked for
    int i = 0;
    for (int g0 = b0; g0 < b1; g0 += ScaleGroup::kBlocks) {
      float s[ScaleGroup::kBlocks];
      sg.take(s, g0);
#pragma unroll
      for (int j = 0; j < ScaleGroup::kBlocks; ++j) {
        if (g0 + j >= b1) break;
        const int u = i % C::kBufs;
        // where a wait runs out the warp goes on as one, with sums that nobody stores
        if (!seen && !mbar_wait_short(&acc_full[u], (i / C::kBufs) & 1, &abort_sh)) {
          record_error_word(a.err, kErrTimeoutWord);
          abort_sh = 1;
        }
        ++i;
        __syncwarp();
        tc_fence_after();
        uint32_t v[64];
        const uint32_t src = tmem + ((uint32_t)(sp * 32) << 16) + u * C::BN + col0;
        tmem_read(src, v);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&acc_empty[u]);
        seen = mbar_test(&acc_full[i % C::kBufs], (i / C::kBufs) & 1);  // answered while these are added
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          fma2(acc[c], acc[c + 1], __uint_as_float(v[c]), __uint_as_float(v[c + 1]), s[j]);
      }
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
        v = sum_over_cluster(base + r * C::kRowFloats * 4, S);
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
//   warps 4-11  sums of the CTA's own 128 rows: a thread holds one row and 128
//               columns (one weight-scale block)
//   warp 0      one thread copies: the CTA's own two boxes per 128-k block; their
//               bytes count on the even CTA's barrier
//   warp 1      TMEM allocation; in the even CTA one thread issues the MMAs into
//               four 128-column TMEM buffers, half a tile's columns each; its
//               commits arrive on both CTAs' barriers
// The MMAs of a block take 575 cycles by themselves.  Adding its 256 columns
// takes each warp scheduler 256 cycles of the FMA pipe, and the plain loop below
// (wait, read 64 columns, add them) 390 in all, two warps taking turns.  (Reading
// the next piece while one is added spills.)  Together they take 800 a block, and
// each tile 2650 more: 2100 for its store, 550 until the next tile's first buffer
// is full.  8192 x 3584 x 37888: 64 tiles a pair, 1.61 million cycles, 1008 us.
// A buffer's way round (sums' release, across the pair, MMAs, commit, read) takes
// more than 1200 cycles, so there are four of them.
// Waits acquire at CTA scope: what they guard is TMEM (ordered by the tcgen05
// fences) and bytes of the copy engine.  (At cluster scope a wait that need not
// wait takes 250 cycles.)
// The sum warps take 224 registers (setmaxnreg), the other four keep 56:
// 256 x 224 + 128 x 56 = 384 x 168, the launch's registers.
// Output goes through 8 KB of shared memory per warp and leaves by a tensor-map
// store, so the next tile's sums start at once.

struct Pair {
  static constexpr int BM = 256, BN = 256;
  static constexpr int kStages = 5;
  static constexpr int kStageBytes = 2 * 16384;
  static constexpr int kBufs = 4, kBufCols = 128;
  static constexpr int kSums = 8;  // warps
  static constexpr int kThreads = 32 * (kSums + 4);
  static constexpr int kRegsLaunch = 168, kRegsSum = 224, kRegsOther = 56;
  static constexpr int kOffStage = kStages * kStageBytes;
  static constexpr int kSmemBytes = kOffStage + kSums * 8192 + 1024;
  static_assert(kSmemBytes <= 232448 - 1024, "shared memory overflow");
  static_assert(2 * kRegsSum + kRegsOther <= 3 * kRegsLaunch, "register split above the launch's share");
};
__device__ __forceinline__ void regs_sum() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory"); }
__device__ __forceinline__ void regs_other() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory"); }

// 32 rows (row = lane) x 128 bytes in registers -> the warp's staging area, with
// the 128-byte swizzle of the output's tensor map
__device__ __forceinline__ void stage_rows(uint8_t* wst, const uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(wst + codes_chunk_off((uint32_t)lane, (uint32_t)j)) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
// The staged rows to rows of Y that no tensor map describes.  kPer: output
// elements per four bytes (2 for bf16, 1 for float32).
template <int kPer>
__device__ __forceinline__ void copy_rows(const LinearArgs& a, const uint8_t* wst, int row0, int col0, int lane) {
  constexpr int kEl = 4 / kPer;  // bytes per element
  uint8_t* y = static_cast<uint8_t*>(a.y);
  const int rows = min(32, a.T - row0);
  for (int r = 0; r < rows; ++r) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int c = lane + 32 * e, byte = c * kEl;  // element of the row's 32 * kPer
      const uint8_t* src = wst + codes_chunk_off((uint32_t)r, (uint32_t)byte >> 4) + (byte & 15);
      if (col0 + c < a.D) {
        uint8_t* dst = y + ((size_t)(row0 + r) * a.ldy + col0 + c) * kEl;
        if (kPer == 2)
          *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
        else
          *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
      }
    }
  }
  __syncwarp();
}
// Two staged pieces of 32 rows x 128 bytes, the second kSpan columns on, to Y
template <int kPer, int kSpan>
__device__ __forceinline__ void put_rows(const LinearArgs& a, const CUtensorMap* mapy, uint8_t* wst, int row0, int col0,
                                         int lane) {
  if (a.vec_y) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(mapy, wst, col0, row0);
      if (col0 + kSpan < a.D) tma_store_2d(mapy, wst + 4096, col0 + kSpan, row0);
      bulk_commit_group();
    }
  } else {
    __syncwarp();
    copy_rows<kPer>(a, wst, row0, col0, lane);
    if (col0 + kSpan < a.D) copy_rows<kPer>(a, wst + 4096, row0, col0 + kSpan, lane);
  }
}

__global__ void __launch_bounds__(Pair::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap mapx, const __grid_constant__ CUtensorMap mapw,
                    const __grid_constant__ CUtensorMap mapy, const LinearArgs a) {
  using C = Pair;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::kStages];   // even CTA: both CTAs' boxes have landed
  __shared__ __align__(8) uint64_t empty_bar[C::kStages];  // each CTA: its slot has been read
  __shared__ __align__(8) uint64_t acc_full[C::kBufs];     // each CTA
  __shared__ __align__(8) uint64_t acc_empty[C::kBufs];    // even CTA: both CTAs' sum warps took the buffer
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
  const int inner = m_fast ? m_tiles : n_tiles;
  // a role's walk over this pair's tiles; the division is done once
  struct Walk {
    int tile, in, out;
  };
  const int step_out = npairs / inner, step_in = npairs - step_out * inner;
  auto first_tile = [&]() { return Walk{pair, pair % inner, pair / inner}; };
  auto next_tile = [&](Walk& w) {
    w.tile += npairs;
    w.in += step_in;
    w.out += step_out;
    if (w.in >= inner) {
      w.in -= inner;
      ++w.out;
    }
  };
  auto row_tile = [&](const Walk& w) { return m_fast ? w.in : w.out; };
  auto col_tile = [&](const Walk& w) { return m_fast ? w.out : w.in; };

  if (threadIdx.x == 0) {
    tma_prefetch_map(&mapx);
    tma_prefetch_map(&mapw);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::kSums);
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
  pdl_trigger();  // after the allocation: the next grid's CTAs wait for this one with TMEM in hand
  pdl_wait();

  if (warp < 4) {
    regs_other();
    if (warp == 0 && elect_one()) {
      const uint32_t full_lead = mapa_shared(smem_u32(&full_bar[0]), 0);
      int i = 0, s = 0;
      uint32_t phase = 1;  // of the slot's previous use
      for (Walk w = first_tile(); w.tile < ntiles && !abort_sh; next_tile(w)) {
        const int mt = row_tile(w), nt = col_tile(w);
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        for (int b = 0; b < nkb; ++b, ++i) {
          if (i >= C::kStages && !mbar_wait(&empty_bar[s], phase, deadline, &abort_sh)) {
            record_error_word(a.err, kErrTimeoutWord);
            abort_sh = 1;
            break;
          }
          uint8_t* st = smem + s * C::kStageBytes;
          if (leader) mbar_arrive_expect_tx(&full_bar[s], 2 * C::kStageBytes);  // both CTAs' boxes
          const uint32_t fb = full_lead + (uint32_t)(s * sizeof(uint64_t));
          tma_2d_pair(st, &mapx, b * kBlock, mt * C::BM + (int)rank * 128, fb);
          tma_2d_pair(st + 16384, &mapw, b * kBlock, nt * C::BN + (int)rank * 128, fb);
          if (++s == C::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // every slot's last use has been released (so its copies landed and the
      // commit's arrival on this CTA's barrier is in) before the CTA may leave
      const uint64_t lim = globaltimer_ns() + kWaitNs;
      for (int j = i > C::kStages ? i - C::kStages : 0; j < i; ++j)
        while (!mbar_try_wait_cluster(&empty_bar[j % C::kStages], (j / C::kStages) & 1) && globaltimer_ns() < lim) {
        }
    }
    if (warp == 1 && leader && elect_one()) {
      constexpr uint32_t idesc = idesc_e4m3(C::BM, C::kBufCols);
      int i = 0, s = 0;
      uint32_t phase = 0;
      for (int tile = pair; tile < ntiles && !abort_sh; tile += npairs) {
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        for (int b = 0; b < nkb; ++b, ++i) {
          const int u = (i & 1) * 2;
          const uint32_t taken = ((i >> 1) & 1) ^ 1;
          // the three answers are asked for at once; what is not there yet is waited for
          const bool f = mbar_test(&full_bar[s], phase);
          const bool e0 = mbar_test(&acc_empty[u], taken), e1 = mbar_test(&acc_empty[u + 1], taken);
          bool ok = f || mbar_wait(&full_bar[s], phase, deadline, &abort_sh);
          const uint32_t st = smem_u32(smem + s * C::kStageBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 64 of each CTA's columns of W
            ok = ok && (i < 2 || (h ? e1 : e0) || mbar_wait(&acc_empty[u + h], taken, deadline, &abort_sh));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f8_pair(tmem + (u + h) * C::kBufCols, smem_desc(st + 32 * j, 16, 1024, kSw128),
                          smem_desc(st + 16384 + 8192 * h + 32 * j, 16, 1024, kSw128), idesc, j > 0);
            tc_commit_pair_mc(&acc_full[u + h], 0x3);
          }
          if (!ok) {
            record_error_word(a.err, kErrTimeoutWord);
            abort_sh = 1;
            break;
          }
          tc_commit_pair_mc(&empty_bar[s], 0x3);
          if (++s == C::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else {
    regs_sum();
    const int sp = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quarter; column half
    const uint32_t acc_empty_lead = mapa_shared(smem_u32(&acc_empty[0]), 0);
    uint8_t* wst = smem + C::kOffStage + (size_t)(warp - 4) * 8192;
    const int d_blocks = blocks_of(a.D);
    const uint32_t src = tmem + ((uint32_t)(sp * 32) << 16) + half * 64;
    int n = 0;  // buffers taken
    ScaleGroup sg;
    auto scales = [&](const Walk& w) {
      const int mt = row_tile(w), nt = col_tile(w);
      sg.start(a.xs + min(mt * C::BM + (int)rank * 128 + sp * 32 + lane, a.T - 1), a.lds,
               a.ws + (size_t)min(nt * 2 + half, d_blocks - 1) * nkb, 0, nkb);
    };
    bool seen = false;  // the next buffer was full when it was asked for
    Walk w = first_tile();
    if (w.tile < ntiles) scales(w);
    while (w.tile < ntiles) {
      const int row0 = row_tile(w) * C::BM + (int)rank * 128 + sp * 32, col0 = col_tile(w) * C::BN + half * 128;
      float acc[128] = {};
      for (int b0 = 0; b0 < nkb; b0 += ScaleGroup::kBlocks) {
        float s[ScaleGroup::kBlocks];
        sg.take(s, b0);
#pragma unroll
        for (int j = 0; j < ScaleGroup::kBlocks; ++j) {
          if (b0 + j >= nkb) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int u = n & 3;
            // where a wait runs out the warp goes on as one, with sums that nobody stores
            if (!seen && !mbar_wait_short(&acc_full[u], (n >> 2) & 1, &abort_sh)) {
              record_error_word(a.err, kErrTimeoutWord);
              abort_sh = 1;
            }
            ++n;
            __syncwarp();
            tc_fence_after();
            uint32_t v[64];
            tmem_ld32(src + u * C::kBufCols, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
            tmem_ld32(src + u * C::kBufCols + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_lead + (uint32_t)(u * sizeof(uint64_t)));
            seen = mbar_test(&acc_full[n & 3], (n >> 2) & 1);  // answered while these are added
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              fma2(acc[64 * h + e], acc[64 * h + e + 1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]), s[j]);
          }
        }
      }
      next_tile(w);
      if (warp_stopped(&abort_sh)) break;
      if (w.tile < ntiles) scales(w);  // on their way while this tile is stored
      if (row0 < a.T && col0 < a.D) {
        uint32_t o[32];
        if (lane == 0) bulk_wait_read_all();  // the last tile's stores have left the staging area
        __syncwarp();
        if (a.out_f32) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c == 2) {
              if (col0 + 64 >= a.D) break;
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(acc[32 * c + e]);
            stage_rows(wst + (c & 1) * 4096, o, lane);
            if (c & 1) put_rows<1, 32>(a, &mapy, wst, row0, col0 + 32 * (c - 1), lane);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = pack_bf16x2(acc[64 * c + 2 * e], acc[64 * c + 2 * e + 1]);
            stage_rows(wst + c * 4096, o, lane);
          }
          put_rows<2, 64>(a, &mapy, wst, row0, col0, lane);
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // the stores are complete before the grid is
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
  if (T <= 16) return launch_skinny<16>(a, dev, stream);
  if (T <= 32) return launch_skinny<32>(a, dev, stream);
  if (T <= 64) return launch_skinny<64>(a, dev, stream);
  CUtensorMap mx, mw;
  if (!byte_map(&mx, x, (uint64_t)T, (uint64_t)K, 128) || !byte_map(&mw, w, (uint64_t)D, (uint64_t)K, 128))
    return cudaErrorInvalidValue;
  void* args[] = {&mx, &mw, &a};
  const int nkb = blocks_of(K);
  const long long pair_tiles = (long long)((T + 255) / 256) * ((D + 255) / 256);
  const long long tiles = (long long)((T + 127) / 128) * ((D + 127) / 128);
  // Pairs once 128 x 128 tiles need a second wave.  Measured, pair against tile: 768 x 4096 x 4096 (192 tiles) 21 and
  // 30 us, 4096 x 1024 x 600 (160) 8.6 and 12.4; 600 x 8192 x 3000 (120) 35 and 28, 512 x 4096 x 4096 (128) 20 and 16.
  if (tiles > dev->sms && pair_regs_ok()) {
    static bool done[64] = {};
    cudaError_t e = opt_in_smem((const void*)fp8_pair_kernel, Pair::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    CUtensorMap my = mx;  // not used unless rows of Y start on 16-byte boundaries
    if (a.vec_y && !rows_map(&my, y, (uint64_t)T, (uint64_t)D, (uint64_t)ldy, out_f32 ? 4 : 2, 32))
      return cudaErrorInvalidValue;
    void* pair_args[] = {&mx, &mw, &my, &a};
    const int pairs = (int)(pair_tiles < dev->sms / 2 ? pair_tiles : dev->sms / 2);
    return launch_pdl((const void*)fp8_pair_kernel, dim3(2 * pairs), dim3(Pair::kThreads), Pair::kSmemBytes, 2, stream,
                      pair_args);
  }
  static bool done[64] = {};
  cudaError_t e = opt_in_smem((const void*)fp8_tile_kernel, Tile::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // the widest cluster with which all reside at once
  static Resident known;
  int s = 8;
  for (; s > 1; --s) {
    if (s > nkb || s * tiles > dev->sms) continue;
    if (resident_clusters((const void*)fp8_tile_kernel, Tile::kThreads, Tile::kSmemBytes, s, known) >= tiles) break;
  }
  a.splits = s;
  return launch_pdl((const void*)fp8_tile_kernel, dim3(a.splits, (D + 127) / 128, (T + 127) / 128),
                    dim3(Tile::kThreads), Tile::kSmemBytes, a.splits, stream, args);
}

}  // namespace fp8
}  // namespace sharq
