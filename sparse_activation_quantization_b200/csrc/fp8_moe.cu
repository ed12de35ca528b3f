// fp8_moe.cu - a whole mixture-of-experts layer for a few tokens, two kernels.
//
//   chosen(t) = the k largest router logits of token t (ties: lower index)
//   p(t, j)   = softmax of the logits over the chosen (or over all) experts
//   h(t, j)   = silu(W_gate[e] x_t) * (W_up[e] x_t),        e = chosen(t)[j]
//   y_t       = sum_j p(t, j) W_down[e] h(t, j)
//
// Weights are E4M3 with a float32 scale per 128 x 128 block, activations bf16.
// With a few tokens the layer is bound by reading each chosen expert's weights
// once, so both kernels stream weights from HBM straight into registers, 16
// weight rows x 128 k per warp step, and multiply them with warp-level f16 MMAs
// (m16n8k16): E4M3 converts to f16 exactly, and each activation's 128-k block
// is scaled by a power of two that puts its largest value in [2^14, 2^15), so
// the conversion of a bf16 activation is exact down to 2^-28 of that value
// (and 2^-39 of it in absolute terms below).  The power of two and the weight
// scale are applied to the block's sum in float32.
//   gate-up  item = (chosen expert, 8 columns of h): MMA rows 0-7 are the gate
//            rows, rows 8-15 the up rows of the same columns, so one thread
//            ends with both and forms silu(gate) * up.  K is split over the
//            warps and joined in shared memory.
//   down     item = 16 columns of y for all tokens: each warp takes a share of
//            the (expert, k range) units, adds p * result to its own sums in
//            shared memory, and the warps' sums are joined in warp order.
// Neither uses atomics on results; the sums' order is fixed by the routing.
#include "fp8.cuh"

namespace sharq {
namespace fp8 {

constexpr int kMoeMaxTokens = 64, kMoeMaxTopk = 16, kMoeMaxExperts = 512;

namespace {

constexpr int kMoeWarps = 8;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopk;

struct MoeArgs {
  const __nv_bfloat16* x;   // [T][H]
  const float* logits;      // [T][E]
  const uint8_t* w13;       // [E][2 I][H]: gate rows, then up rows
  const float* s13;         // [E][blocks(2 I)][blocks(H)]
  const uint8_t* w2;        // [E][H][I]
  const float* s2;          // [E][blocks(H)][blocks(I)]
  __nv_bfloat16* y;         // [T][H]
  int* ids;                 // [T][topk] or nullptr
  float* weights;           // [T][topk] or nullptr
  int* route;               // workspace: the routing that the down kernel reads
  float* h;                 // workspace: [T * topk][I]
  long long ldx, ldl, ldy;
  int T, E, topk, H, I, renorm;
};

// The routing in shared memory: experts with at least one token, and per
// expert the (token, choice) pairs t * topk + j that chose it.
struct Routing {
  int n_active;
  int n_pairs;
  short active[kMoeMaxExperts];        // expert of each active slot, ascending
  short first[kMoeMaxExperts + 1];     // first pair of each active slot
  short pairs[kMaxPairs];              // pair ids, expert by expert
  float p[kMaxPairs];                  // by pair id
};
constexpr int kRouteInts = (int)((sizeof(Routing) + 3) / 4);

// Order-preserving key of a logit: larger logit, larger key; -0 equals +0; a
// NaN sorts below everything, so an index is always valid.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// exp(l - max), 0 for a logit of -inf (also where the maximum is -inf) or NaN
__device__ __forceinline__ float logit_exp(float l, float mx) {
  if (!(l > -INFINITY)) return 0.0f;
  return l == mx ? 1.0f : expf(l - mx);
}

// Every CTA derives the same routing from the logits.  expert_of: scratch
// [kMaxPairs]; cnt: scratch [kMoeMaxExperts].
__device__ void build_routing(const MoeArgs& a, Routing& r, short* expert_of, int* cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += kMoeThreads) cnt[e] = 0;
  __syncthreads();
  for (int t = warp; t < a.T; t += kMoeWarps) {
    const float* lg = a.logits + (size_t)t * a.ldl;
    constexpr int kPer = kMoeMaxExperts / 32;
    uint32_t key[kPer];
    float lmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      key[i] = 0u;
      if (32 * i < a.E && e < a.E) {
        const float l = lg[e];
        // keys start at 1, so 0 marks a taken or absent expert
        key[i] = max(logit_key(l), 1u);
        if (l > lmax) lmax = l;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    float sum = 0.0f;
    if (!a.renorm) {
      for (int e = lane; e < a.E; e += 32) sum += logit_exp(lg[e], lmax);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    float mine = 0.0f;
    int my_e = 0;
    for (int j = 0; j < a.topk; ++j) {
      uint32_t best = 0u;
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (32 * i < a.E && key[i] > best) {
          best = key[i];
          be = lane + 32 * i;
        }
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int e = __reduce_min_sync(0xffffffffu, best == top ? be : 0x7fffffff);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i == e) key[i] = 0u;
      const float v = logit_exp(lg[e], lmax);
      if (a.renorm) sum += v;
      if (lane == j) {
        mine = v;
        my_e = e;
      }
    }
    if (lane < a.topk) {
      const int pr = t * a.topk + lane;
      const float p = sum > 0.0f ? __fdiv_rn(mine, sum) : 0.0f;  // all logits -inf or NaN: no expert counts
      r.p[pr] = p;
      expert_of[pr] = (short)my_e;
      atomicAdd(&cnt[my_e], 1);
      if (blockIdx.x == 0) {
        if (a.ids) a.ids[pr] = my_e;
        if (a.weights) a.weights[pr] = p;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {  // compact the experts in use, with the start of each one's pairs
    int na = 0, np = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < a.E ? cnt[e] : 0;
      const uint32_t m = __ballot_sync(0xffffffffu, c > 0);
      int pre = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += n;
      }
      if (c > 0) {
        const int slot = na + __popc(m & ((1u << lane) - 1u));
        r.active[slot] = (short)e;
        r.first[slot] = (short)(np + pre - c);
        cnt[e] = np + pre - c;  // now the expert's next free place
      }
      na += __popc(m);
      np += __shfl_sync(0xffffffffu, pre, 31);
    }
    if (lane == 0) {
      r.n_active = na;
      r.n_pairs = np;
      r.first[na] = (short)np;
    }
  }
  __syncthreads();
  // which place a pair takes among its expert's decides only the MMA column it
  // is computed in
  for (int i = threadIdx.x; i < a.T * a.topk; i += kMoeThreads) r.pairs[atomicAdd(&cnt[expert_of[i]], 1)] = (short)i;
  __syncthreads();
}

// One token's share of a 128-k block: this lane's 2 x 16 values (16 q + 64 h),
// scaled by a power of two and converted to f16 pairs.
struct ActBlock {
  uint32_t v[16];
  float scale;  // what the f16 values are to be multiplied by
};
__device__ __forceinline__ void scale_block(const float (&f)[32], ActBlock& o) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(f[i]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  // 2^(14 - floor(log2 m)) from the exponent field; the clamp keeps both it
  // and its inverse normal numbers
  const uint32_t ef = max(__float_as_uint(m) >> 23, 15u);
  const float up = __uint_as_float((268u - ef) << 23);
  o.scale = __uint_as_float((ef - 14u) << 23);
#pragma unroll
  for (int i = 0; i < 16; ++i) o.v[i] = f16x2_of(f[2 * i] * up, f[2 * i + 1] * up);
}
__device__ __forceinline__ void load_act(const __nv_bfloat16* row, int k0, int K, int q, float (&f)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = k0 + 64 * h + 16 * q;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float e[8] = {};
      if (row && k < K) unpack_bf16x8(*reinterpret_cast<const uint4*>(row + k + 8 * j), e);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[16 * h + 8 * j + i] = e[i];
    }
  }
}
__device__ __forceinline__ void load_act(const float* row, int k0, int K, int q, float (&f)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = k0 + 64 * h + 16 * q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 e = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (row && k < K) e = *reinterpret_cast<const float4*>(row + k + 4 * j);
      f[16 * h + 4 * j] = e.x;
      f[16 * h + 4 * j + 1] = e.y;
      f[16 * h + 4 * j + 2] = e.z;
      f[16 * h + 4 * j + 3] = e.w;
    }
  }
}

// 16 weight rows x one 128-k block in registers: [h][row half], 16 bytes each
struct WeightBlock {
  uint4 v[2][2];
};
__device__ __forceinline__ void load_weights(const uint8_t* r0, const uint8_t* r1, int k0, int K, int q,
                                             WeightBlock& w) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = k0 + 64 * h + 16 * q;
    const bool in = k < K;
    w.v[h][0] = in ? ld_stream(r0 + k) : make_uint4(0u, 0u, 0u, 0u);
    w.v[h][1] = in ? ld_stream(r1 + k) : make_uint4(0u, 0u, 0u, 0u);
  }
}
// c (16 x 8) = weights x activations over one 128-k block
__device__ __forceinline__ void block_product(const WeightBlock& w, const ActBlock& x, float (&c)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a0[4] = {w.v[h][0].x, w.v[h][0].y, w.v[h][0].z, w.v[h][0].w};
    const uint32_t a1[4] = {w.v[h][1].x, w.v[h][1].y, w.v[h][1].z, w.v[h][1].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t l0, h0, l1, h1;
      e4m3x4_to_f16(a0[j], l0, h0);
      e4m3x4_to_f16(a1[j], l1, h1);
      mma_f16(c, l0, l1, h0, h1, x.v[8 * h + 2 * j], x.v[8 * h + 2 * j + 1]);
    }
  }
}

__global__ void __launch_bounds__(kMoeThreads) moe_gate_up_kernel(const MoeArgs a) {
  __shared__ Routing r;
  __shared__ float red[kMoeWarps][16][9];
  __shared__ int cnt[kMoeMaxExperts];
  __shared__ short expert_of[kMaxPairs];
  pdl_wait();
  build_routing(a, r, expert_of, cnt);
  pdl_trigger();
  if (blockIdx.x == 0) {
    const int* src = reinterpret_cast<const int*>(&r);
    for (int i = threadIdx.x; i < kRouteInts; i += kMoeThreads) a.route[i] = src[i];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int nkb = blocks_of(a.H), cols = a.I / 8;
  const int rb = blocks_of(2 * a.I);
  const int items = r.n_active * cols;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int slot = it / cols, i0 = (it - slot * cols) * 8;
    const int e = r.active[slot];
    const int p0 = r.first[slot], np = r.first[slot + 1] - p0;
    const uint8_t* wg = a.w13 + ((size_t)e * 2 * a.I + i0 + g) * a.H;
    const uint8_t* wu = wg + (size_t)a.I * a.H;
    const float* sg = a.s13 + ((size_t)e * rb + i0 / kBlock) * nkb;
    const float* su = a.s13 + ((size_t)e * rb + (a.I + i0) / kBlock) * nkb;
    for (int n0 = 0; n0 < np; n0 += 8) {  // eight tokens at a time
      const int pr = n0 + g < np ? r.pairs[p0 + n0 + g] : -1;
      const __nv_bfloat16* row = pr >= 0 ? a.x + (size_t)(pr / a.topk) * a.ldx : nullptr;
      float acc[4] = {};
      for (int b = warp; b < nkb; b += kMoeWarps) {
        WeightBlock w;
        load_weights(wg, wu, b * kBlock, a.H, q, w);
        float f[32];
        load_act(row, b * kBlock, a.H, q, f);
        ActBlock x;
        scale_block(f, x);
        float c[4] = {};
        block_product(w, x, c);
        const float x0 = __shfl_sync(0xffffffffu, x.scale, (2 * q) * 4), x1 = __shfl_sync(0xffffffffu, x.scale, (2 * q + 1) * 4);
        const float g_s = sg[b], u_s = su[b];
        acc[0] = fmaf(c[0] * x0, g_s, acc[0]);
        acc[1] = fmaf(c[1] * x1, g_s, acc[1]);
        acc[2] = fmaf(c[2] * x0, u_s, acc[2]);
        acc[3] = fmaf(c[3] * x1, u_s, acc[3]);
      }
      red[warp][g][2 * q] = acc[0];
      red[warp][g][2 * q + 1] = acc[1];
      red[warp][g + 8][2 * q] = acc[2];
      red[warp][g + 8][2 * q + 1] = acc[3];
      __syncthreads();
      if (threadIdx.x < 64) {
        const int i = threadIdx.x & 7, n = threadIdx.x >> 3;
        if (n0 + n < np) {
          float gs = 0.0f, us = 0.0f;
#pragma unroll
          for (int v = 0; v < kMoeWarps; ++v) {
            gs += red[v][i][n];
            us += red[v][i + 8][n];
          }
          a.h[(size_t)r.pairs[p0 + n0 + n] * a.I + i0 + i] = silu_mul(gs, us);
        }
      }
      __syncthreads();
    }
  }
}

__global__ void __launch_bounds__(kMoeThreads) moe_down_kernel(const MoeArgs a) {
  __shared__ Routing r;
  extern __shared__ float sums[];  // [warp][T][16]
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int nkb = blocks_of(a.I), rb = blocks_of(a.H);
  for (int i = threadIdx.x; i < kMoeWarps * a.T * 16; i += kMoeThreads) sums[i] = 0.0f;
  pdl_wait();
  {
    int* dst = reinterpret_cast<int*>(&r);
    for (int i = threadIdx.x; i < kRouteInts; i += kMoeThreads) dst[i] = a.route[i];
  }
  __syncthreads();
  const int d0 = blockIdx.x * 16;
  float* mine = sums + (size_t)warp * a.T * 16;
  const int units = r.n_active * nkb;
  const int u0 = (int)((long long)warp * units / kMoeWarps), u1 = (int)((long long)(warp + 1) * units / kMoeWarps);
  for (int u = u0; u < u1;) {
    const int slot = u / nkb, b0 = u - slot * nkb;
    const int b1 = min(nkb, b0 + (u1 - u));
    u += b1 - b0;
    const int e = r.active[slot];
    const int p0 = r.first[slot], np = r.first[slot + 1] - p0;
    const uint8_t* w0 = a.w2 + ((size_t)e * a.H + d0 + g) * a.I;
    const uint8_t* w1 = w0 + (size_t)8 * a.I;
    const float* s = a.s2 + ((size_t)e * rb + d0 / kBlock) * nkb;
    for (int n0 = 0; n0 < np; n0 += 8) {
      const int pr = n0 + g < np ? r.pairs[p0 + n0 + g] : -1;
      const float* row = pr >= 0 ? a.h + (size_t)pr * a.I : nullptr;
      float acc[4] = {};
      for (int b = b0; b < b1; ++b) {
        WeightBlock w;
        load_weights(w0, w1, b * kBlock, a.I, q, w);
        float f[32];
        load_act(row, b * kBlock, a.I, q, f);
        ActBlock x;
        scale_block(f, x);
        float c[4] = {};
        block_product(w, x, c);
        const float x0 = __shfl_sync(0xffffffffu, x.scale, (2 * q) * 4), x1 = __shfl_sync(0xffffffffu, x.scale, (2 * q + 1) * 4);
        const float sw = s[b];
        acc[0] = fmaf(c[0] * x0, sw, acc[0]);
        acc[1] = fmaf(c[1] * x1, sw, acc[1]);
        acc[2] = fmaf(c[2] * x0, sw, acc[2]);
        acc[3] = fmaf(c[3] * x1, sw, acc[3]);
      }
      // an expert appears once in a token's choices, so the eight columns are
      // eight different tokens: no two lanes add to one place
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int m = n0 + 2 * q + n;
        if (m < np) {
          const int pc = r.pairs[p0 + m];
          float* dst = mine + (pc / a.topk) * 16;
          const float p = r.p[pc];
          dst[g] = fmaf(p, acc[n], dst[g]);
          dst[g + 8] = fmaf(p, acc[2 + n], dst[g + 8]);
        }
      }
      __syncwarp();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += kMoeThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeWarps; ++w) v += sums[(size_t)w * a.T * 16 + i];
    a.y[(size_t)(i >> 4) * a.ldy + d0 + (i & 15)] = __float2bfloat16_rn(v);
  }
}

}  // namespace

size_t moe_workspace(int T, int topk, int I) {
  return ((size_t)kRouteInts * 4 + 255) / 256 * 256 + (size_t)T * topk * I * sizeof(float);
}

cudaError_t launch_moe(const void* x, long long ldx, const float* logits, long long ldl, int T, int E, int topk,
                       int renorm, int H, int I, const uint8_t* w13, const float* s13, const uint8_t* w2,
                       const float* s2, void* y, long long ldy, int* ids, float* weights, void* ws,
                       cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const Device* dev = device();
  if (!dev) return cudaErrorInvalidDevice;
  MoeArgs a;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.logits = logits;
  a.w13 = w13;
  a.s13 = s13;
  a.w2 = w2;
  a.s2 = s2;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.ids = ids;
  a.weights = weights;
  a.route = static_cast<int*>(ws);
  a.h = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ((size_t)kRouteInts * 4 + 255) / 256 * 256);
  a.ldx = ldx;
  a.ldl = ldl;
  a.ldy = ldy;
  a.T = T;
  a.E = E;
  a.topk = topk;
  a.H = H;
  a.I = I;
  a.renorm = renorm;
  void* args[] = {&a};
  const long long most = (long long)(T * topk < E ? T * topk : E) * (I / 8);
  const long long grid = most < dev->sms * 2 ? most : dev->sms * 2;
  cudaError_t e = launch_pdl((const void*)moe_gate_up_kernel, dim3((unsigned)grid), dim3(kMoeThreads), 0, 1, stream, args);
  if (e != cudaSuccess) return e;
  const int smem = kMoeWarps * T * 16 * (int)sizeof(float);
  return launch_pdl((const void*)moe_down_kernel, dim3(H / 16), dim3(kMoeThreads), smem, 1, stream, args);
}

}  // namespace fp8
}  // namespace sharq
