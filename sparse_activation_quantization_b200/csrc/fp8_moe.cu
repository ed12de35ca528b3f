// fp8_moe.cu - a whole mixture-of-experts layer for a few tokens, two kernels.
//
//   chosen(t) = the k largest router logits of token t (ties: lower index)
//   p(t, j)   = softmax of the logits over the chosen (or over all) experts
//   h(t, j)   = silu(W_gate[e] x_t) * (W_up[e] x_t),        e = chosen(t)[j]
//   y_t       = sum_j p(t, j) W_down[e] h(t, j)
//
// Weights are E4M3 with a float32 scale per 128 x 128 block, activations bf16.
// With a few tokens the layer is bound by reading each chosen expert's weights
// once, so both kernels stream them (fp8_stream.cuh) against up to 32 tokens.
// Activations enter the E4M3 MMAs without being quantized to E4M3: a value v of
// a 128-k block, scaled by a power of two that puts the block's largest into
// [128, 256), is written as v1 + v2 / 16 (+ v3 / 256), each an E4M3 number, the
// rounded remainder of the one before.  Each term is a column of the MMA's B
// operand of its own, with its power of two in the column's scale, and the
// columns of a token are added at the end.  Four bits a term: two terms hold a
// bf16 activation exactly where it is at least 2^-13 of the block's largest,
// and to 2^-21 of that largest below; three hold h to 2^-12 of itself.
// (f16 MMAs need 8 conversions per 16 weights and half the MMA rate, and are no
// faster: 322 us against 307 on the 128-expert layer, T = 64.)
//   gate-up  item = (group of tokens of one expert, 8 CG columns of h): MMA
//            rows 0-7 are gate rows, rows 8-15 the up rows of the same columns,
//            so a thread ends with both and forms silu(gate) * up.  With few
//            items, KS = 8 / CG warps share a column tile's K and join their
//            sums in shared memory.
//   down     a cluster of CTAs owns 128 rows of W_down (16 per warp) for all
//            tokens; each CTA takes a share of the (group, k block) units and
//            sums p * result per token in shared memory; the CTAs' sums are
//            joined in rank order over distributed shared memory.
// No atomics touch results; the order of every sum follows from the routing.
#include "fp8_stream.cuh"

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

// The routing in shared memory: per expert the (token, choice) pairs
// t * topk + j that chose it, cut into groups of at most 32.
constexpr int kGroup = 32;
constexpr int kMaxGroups = kMoeMaxExperts + kMaxPairs / kGroup;
struct Routing {
  int n_groups;
  short expert[kMaxGroups];  // ascending
  short first[kMaxGroups];   // first of the group's pairs
  short count[kMaxGroups];
  short pairs[kMaxPairs];    // pair ids, expert by expert
  float p[kMaxPairs];        // by pair id
};
static_assert(sizeof(Routing) % 4 == 0, "copied as ints");
constexpr int kRouteInts = (int)(sizeof(Routing) / 4);

// Order-preserving key of a logit: larger logit, larger key; -0 equals +0; a
// NaN sorts below everything, so an index is always valid.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {  // the logit of a key (NaN: -inf)
  if (k <= 1u) return -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// exp(l - max), 0 for a logit of -inf (also where the maximum is -inf) or NaN
__device__ __forceinline__ float logit_exp(float l, float mx) {
  if (!(l > -INFINITY)) return 0.0f;
  return l == mx ? 1.0f : expf(l - mx);
}

// Every CTA derives the same routing from the logits.  expert_of: scratch
// [kMaxPairs]; cnt: scratch [kMoeMaxExperts].  kPer: logits per lane.
template <int kPer>
__device__ void choose_experts(const MoeArgs& a, Routing& r, short* expert_of, int* cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int t = warp; t < a.T; t += kMoeWarps) {
    const float* lg = a.logits + (size_t)t * a.ldl;
    uint32_t key[kPer];
    float l[kPer], lmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < a.E ? lg[e] : -INFINITY;
      key[i] = e < a.E ? max(logit_key(l[i]), 1u) : 0u;  // 0: absent, or taken
      if (l[i] > lmax) lmax = l[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    float sum = 0.0f;
    if (!a.renorm) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += logit_exp(l[i], lmax);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    uint32_t my_key = 0u;
    int my_e = 0;
    for (int j = 0; j < a.topk; ++j) {
      uint32_t best = key[0];
      int be = lane;
#pragma unroll
      for (int i = 1; i < kPer; ++i)
        if (key[i] > best) {
          best = key[i];
          be = lane + 32 * i;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int e = __reduce_min_sync(0xffffffffu, best == top ? be : 0x7fffffff);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i == e) key[i] = 0u;
      if (lane == j) {
        my_key = top;
        my_e = e;
      }
    }
    const float mine = lane < a.topk ? logit_exp(key_logit(my_key), lmax) : 0.0f;
    if (a.renorm) {
      sum = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < a.topk) {
      const int pr = t * a.topk + lane;
      const float p = sum > 0.0f ? __fdiv_rn(mine, sum) : 0.0f;  // no logit above -inf: no expert counts
      r.p[pr] = p;
      expert_of[pr] = (short)my_e;
      atomicAdd(&cnt[my_e], 1);
      if (blockIdx.x == 0) {
        if (a.ids) a.ids[pr] = my_e;
        if (a.weights) a.weights[pr] = p;
      }
    }
  }
}

__device__ void build_routing(const MoeArgs& a, Routing& r, short* expert_of, int* cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += kMoeThreads) cnt[e] = 0;
  __syncthreads();
  if (a.E <= 128)
    choose_experts<4>(a, r, expert_of, cnt);
  else
    choose_experts<kMoeMaxExperts / 32>(a, r, expert_of, cnt);
  __syncthreads();
  if (warp == 0) {  // lay the experts' pairs out one after another, in groups
    int ng = 0, np = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < a.E ? cnt[e] : 0;
      const int g = (c + kGroup - 1) / kGroup;
      int pc = c, pg = g;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int c1 = __shfl_up_sync(0xffffffffu, pc, o), g1 = __shfl_up_sync(0xffffffffu, pg, o);
        if (lane >= o) {
          pc += c1;
          pg += g1;
        }
      }
      for (int i = 0; i < g; ++i) {
        const int at = ng + pg - g + i;
        r.expert[at] = (short)e;
        r.first[at] = (short)(np + pc - c + i * kGroup);
        r.count[at] = (short)min(kGroup, c - i * kGroup);
      }
      if (e < a.E) cnt[e] = np + pc - c;  // now the expert's next free place
      ng += __shfl_sync(0xffffffffu, pg, 31);
      np += __shfl_sync(0xffffffffu, pc, 31);
    }
    if (lane == 0) r.n_groups = ng;
  }
  __syncthreads();
  // A pair's place among its expert's is its rank by pair id: every CTA cuts
  // the groups alike.  One warp, 32 pairs a step.
  if (warp == 0) {
    for (int i0 = 0; i0 < a.T * a.topk; i0 += 32) {
      const int i = i0 + lane;
      const int e = i < a.T * a.topk ? expert_of[i] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int base = e >= 0 ? cnt[e] : 0;
      __syncwarp();
      if (e >= 0) {
        r.pairs[base + before] = (short)i;
        if (before == 0) cnt[e] = base + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
}

// ----------------------------------------------------- staged activations ---
// Columns of the MMA's B operand.  A token's terms lie so that one lane's
// accumulators hold them all: two terms in neighbouring columns, three in the
// same column of three tiles.  Rows are padded by 16 bytes so that the 8 x 4
// lanes of an operand read distinct banks.

template <int J>
__device__ __forceinline__ int term_column(int n, int j) {
  return J == 2 ? 2 * n + j : 8 * (J * (n >> 3) + j) + (n & 7);
}

__host__ __device__ constexpr int stage_window(int bytes, int nt) {  // 128-k blocks that fit
  const int w = (bytes / (8 * nt) - 16) / kBlock;
  return w > 32 ? 32 : w;
}
constexpr int kStageScales = 272;  // columns x window of the largest form, rounded up

struct Stage {
  uint8_t* v;    // [column][row_bytes]
  float* scale;  // [block][columns]
  int cols, row_bytes;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Columns of np tokens, blocks [b0, b0 + nb).  rows(n): token n's row.  Half a
// warp per (token, block), eight values a lane.  Columns of no token keep what
// they held: their sums are not used.
template <int J, class T, class Rows>
__device__ __forceinline__ void stage_tokens(const Stage& st, int np, int b0, int nb, int K, Rows rows) {
  const int l16 = threadIdx.x & 15;
  const int n_items = np * nb;
  for (int i0 = (threadIdx.x >> 5) * 2; i0 < n_items; i0 += 2 * kMoeWarps) {  // uniform over the warp
    const int i = i0 + ((threadIdx.x >> 4) & 1);
    const int n = i / nb, b = i - n * nb;
    const int k = (b0 + b) * kBlock + l16 * 8;
    float f[8] = {};
    if (i < n_items && k < K) load8(static_cast<const T*>(rows(n)) + k, f);
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // 2^(7 - floor(log2 m)) from the exponent field; the clamp keeps it and its
    // inverse normal numbers (16^-2 of the inverse included)
    const uint32_t ef = max(__float_as_uint(m) >> 23, 20u);
    const float up = __uint_as_float((261u - ef) << 23);
    // an infinity saturates in E4M3: it is in the scale
    float s = ef == 255u ? INFINITY : __uint_as_float((ef - 7u) << 23);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= up;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t c0 = e4m3x4(f[0], f[1], f[2], f[3]), c1 = e4m3x4(f[4], f[5], f[6], f[7]);
      if (i < n_items) {
        const int col = term_column<J>(n, j);
        *reinterpret_cast<uint2*>(st.v + (size_t)col * st.row_bytes + b * kBlock + l16 * 8) = make_uint2(c0, c1);
        if (l16 == 0) st.scale[b * st.cols + col] = s;
      }
      if (j + 1 < J) {
        const float2 d0 = e4m3x2_to_float(c0), d1 = e4m3x2_to_float(c0 >> 16);
        const float2 d2 = e4m3x2_to_float(c1), d3 = e4m3x2_to_float(c1 >> 16);
        f[0] = (f[0] - d0.x) * 16.0f, f[1] = (f[1] - d0.y) * 16.0f;
        f[2] = (f[2] - d1.x) * 16.0f, f[3] = (f[3] - d1.y) * 16.0f;
        f[4] = (f[4] - d2.x) * 16.0f, f[5] = (f[5] - d2.y) * 16.0f;
        f[6] = (f[6] - d3.x) * 16.0f, f[7] = (f[7] - d3.y) * 16.0f;
        s *= 0.0625f;
      }
    }
  }
}

// ------------------------------------------------------------- ring units ---

constexpr int kUnitBytes = kWeightUnit + 16;  // 16 rows x 128 bytes, and the unit's scales

__device__ __forceinline__ void unit_load(uint32_t slot, const uint8_t* p0, const uint8_t* p1, int left,
                                          const float* s0, const float* s1, int lane) {
  rows16_load(slot, p0, p1, left, lane);
  if (lane < 2) copy4(slot + kWeightUnit + lane * 4, lane ? s1 : s0);
}

// acc += unit x staged block b, for NT tiles of eight columns: rows g take
// weight scale s.x, rows g + 8 scale s.y
template <int NT>
__device__ __forceinline__ void unit_product(uint32_t slot, const Stage& st, int b, int lane, float (&acc)[NT][4]) {
  const int g = lane >> 2, q = lane & 3;
  WeightUnit w;
  w.read(slot, lane);
  const float2 s = lds_f2(slot + kWeightUnit);
  const uint32_t x = smem_u32(st.v) + g * st.row_bytes + b * kBlock + q * 16;
  const uint32_t xs = smem_u32(st.scale) + (b * st.cols + 2 * q) * 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float c[4];
    const uint32_t p = x + 8 * n * st.row_bytes;
    w.times(lds128(p), lds128(p + 64), c);
    const float2 t = lds_f2(xs + 32 * n);
    acc[n][0] = fmaf(c[0], t.x * s.x, acc[n][0]);
    acc[n][1] = fmaf(c[1], t.y * s.x, acc[n][1]);
    acc[n][2] = fmaf(c[2], t.x * s.y, acc[n][2]);
    acc[n][3] = fmaf(c[3], t.y * s.y, acc[n][3]);
  }
}

// ---------------------------------------------------------------- gate-up ---

constexpr int kUpTerms = 2;
constexpr int kUpRing = 4;
struct UpSmem {  // offsets in dynamic shared memory
  static constexpr int kStageBytes = 34816;
  static constexpr int kRing = 0;
  static constexpr int kStage = kRing + kMoeWarps * kUpRing * kUnitBytes;
  static constexpr int kScale = kStage + kStageBytes;
  static constexpr int kBytes = kScale + kStageScales * 4;
};
__host__ __device__ constexpr int join_row(int nt) { return 4 * nt + 1; }
static_assert(kMoeWarps * 16 * join_row(kGroup * kUpTerms / 8) * 4 <= UpSmem::kStageBytes, "join buffer");
static_assert(8 * 8 * stage_window(UpSmem::kStageBytes, 8) <= kStageScales &&
              8 * stage_window(UpSmem::kStageBytes, 1) <= kStageScales, "column scales");

struct UpWalk {  // one warp's sequence of units
  const MoeArgs& a;
  const Routing& r;
  int it, end, kb, ks, KS, CG, cg, tiles, nkb, rb;
  const uint8_t *wg, *wu;
  const float *sg, *su;
  bool on;
  __device__ __forceinline__ void item(int lane) {
    if (it >= end) return;
    const int grp = it / tiles, i0 = ((it - grp * tiles) * CG + cg) * 8;
    on = i0 < a.I;
    if (!on) return;
    const int e = r.expert[grp];
    wg = a.w13 + ((size_t)e * 2 * a.I + i0 + (lane >> 2)) * a.H + 16 * (lane & 3);
    wu = wg + (size_t)a.I * a.H;
    sg = a.s13 + ((size_t)e * rb + i0 / kBlock) * nkb;
    su = a.s13 + ((size_t)e * rb + (a.I + i0) / kBlock) * nkb;
  }
  __device__ __forceinline__ void issue(uint32_t slot, int lane) {
    if (it < end) {
      const int k = kb * kBlock;
      if (on) unit_load(slot, wg + k, wu + k, a.H - k - 16 * (lane & 3), sg + kb, su + kb, lane);
      kb += KS;
      if (kb >= nkb) {
        kb = ks;
        ++it;
        item(lane);
      }
    }
    copies_commit();
  }
};

template <int NT>
__device__ __forceinline__ void up_item(const MoeArgs& a, const Routing& r, UpWalk& walk, int it, uint8_t* smem,
                                        uint32_t ring, uint32_t& slot, int& staged) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int grp = it / walk.tiles, base = (it - grp * walk.tiles) * walk.CG * 8;
  const bool on = base + walk.cg * 8 < a.I;
  const int p0 = r.first[grp], np = r.count[grp];
  constexpr int kWin = stage_window(UpSmem::kStageBytes, NT);
  const Stage st{smem + UpSmem::kStage, reinterpret_cast<float*>(smem + UpSmem::kScale), 8 * NT, kWin * kBlock + 16};
  float acc[NT][4] = {};
  int kb = walk.ks;
  for (int b0 = 0; b0 < walk.nkb; b0 += kWin) {
    const int nb = min(kWin, walk.nkb - b0);
    if (staged != grp) {  // otherwise the previous item left the same tokens here
      __syncthreads();
      stage_tokens<kUpTerms, __nv_bfloat16>(st, np, b0, nb, a.H, [&](int n) {
        return a.x + (size_t)(r.pairs[p0 + n] / a.topk) * a.ldx;
      });
      __syncthreads();
    }
    for (; kb < b0 + nb; kb += walk.KS) {
      copies_wait<kUpRing - 1>();
      __syncwarp();  // the scales come from other lanes' copies
      if (on) unit_product<NT>(slot, st, kb - b0, lane, acc);
      __syncwarp();
      walk.issue(slot, lane);
      slot = slot == ring + (kUpRing - 1) * kUnitBytes ? ring : slot + kUnitBytes;
    }
  }
  staged = walk.nkb <= kWin ? grp : -1;
  // columns 2 q, 2 q + 1 of tile n are the two terms of token 4 n + q
  if (walk.KS == 1) {
    if (on) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = 4 * n + q;
        if (m < np)
          a.h[(size_t)r.pairs[p0 + m] * a.I + base + walk.cg * 8 + g] =
              silu_mul(acc[n][0] + acc[n][1], acc[n][2] + acc[n][3]);
      }
    }
    return;
  }
  __syncthreads();  // the stage has been read: the warps' sums take its place
  staged = -1;
  float* red = reinterpret_cast<float*>(smem + UpSmem::kStage);
  constexpr int kRow = join_row(NT);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    red[(warp * 16 + g) * kRow + 4 * n + q] = acc[n][0] + acc[n][1];
    red[(warp * 16 + g + 8) * kRow + 4 * n + q] = acc[n][2] + acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < walk.CG * 8 * np; i += kMoeThreads) {
    const int m = i / (walk.CG * 8), col = i - m * walk.CG * 8;
    if (base + col >= a.I) continue;
    float gs = 0.0f, us = 0.0f;
    for (int k = 0; k < walk.KS; ++k) {
      const float* row = red + (((col >> 3) * walk.KS + k) * 16 + (col & 7)) * kRow + m;
      gs += row[0];
      us += row[8 * kRow];
    }
    a.h[(size_t)r.pairs[p0 + m] * a.I + base + col] = silu_mul(gs, us);
  }
}

__global__ void __launch_bounds__(kMoeThreads, 2) moe_gate_up_kernel(const MoeArgs a) {
  __shared__ Routing r;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  {  // scratch of the routing: the ring, not in use yet
    int* cnt = reinterpret_cast<int*>(smem);
    build_routing(a, r, reinterpret_cast<short*>(cnt + kMoeMaxExperts), cnt);
  }
  pdl_trigger();
  if (blockIdx.x == 0) {
    const int* src = reinterpret_cast<const int*>(&r);
    for (int i = threadIdx.x; i < kRouteInts; i += kMoeThreads) a.route[i] = src[i];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nkb = blocks_of(a.H), cols = a.I / 8;
  // The most warps per column tile that still leave every CTA at most one
  // item: with few experts all their weights are then in flight at once; with
  // many items each warp keeps a tile to itself.
  int KS = 1;
  while (KS < kMoeWarps && 2 * KS <= nkb &&
         r.n_groups * ((cols + kMoeWarps / (2 * KS) - 1) / (kMoeWarps / (2 * KS))) <= (int)gridDim.x)
    KS *= 2;
  const int CG = kMoeWarps / KS, tiles = (cols + CG - 1) / CG;
  const int items = r.n_groups * tiles;
  const int it0 = (int)((long long)blockIdx.x * items / gridDim.x);
  const int it1 = (int)((long long)(blockIdx.x + 1) * items / gridDim.x);
  UpWalk walk{a, r, it0, it1, warp % KS, warp % KS, KS, CG, warp / KS, tiles, nkb, blocks_of(2 * a.I),
              nullptr, nullptr, nullptr, nullptr, false};
  walk.item(lane);
  const uint32_t ring = smem_u32(smem + UpSmem::kRing) + warp * kUpRing * kUnitBytes;
  for (int i = 0; i < kUpRing; ++i) walk.issue(ring + i * kUnitBytes, lane);
  uint32_t slot = ring;
  int staged = -1;
  for (int it = it0; it < it1; ++it) {
    const int c = r.count[it / tiles] * kUpTerms;
    if (c <= 8)
      up_item<1>(a, r, walk, it, smem, ring, slot, staged);
    else if (c <= 16)
      up_item<2>(a, r, walk, it, smem, ring, slot, staged);
    else if (c <= 32)
      up_item<4>(a, r, walk, it, smem, ring, slot, staged);
    else
      up_item<8>(a, r, walk, it, smem, ring, slot, staged);
  }
  copies_wait<0>();
}

// ------------------------------------------------------------------- down ---

constexpr int kDownTerms = 3;
constexpr int kDownRing = 3;
constexpr int kDownRows = 16 * kMoeWarps;
struct DownSmem {
  static constexpr int kStageBytes = 18944;
  static constexpr int kRing = 0;
  static constexpr int kStage = kRing + kMoeWarps * kDownRing * kUnitBytes;
  static constexpr int kScale = kStage + kStageBytes;
  static constexpr int kSums = kScale + kStageScales * 4;  // [T][128]
  static constexpr int bytes(int T) { return kSums + T * kDownRows * 4; }
};
static_assert(stage_window(DownSmem::kStageBytes, kGroup * kDownTerms / 8) >= 1, "a block of a full group must fit");

template <int N>
struct Int {
  static constexpr int value = N;
};
__device__ __forceinline__ float2 ld_shared_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kMoeThreads, 2) moe_down_kernel(const MoeArgs a, int C) {
  __shared__ Routing r;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int d0 = (int)(blockIdx.x / C) * kDownRows;
  const int nkb = blocks_of(a.I), rb = blocks_of(a.H);
  float* sums = reinterpret_cast<float*>(smem + DownSmem::kSums);
  for (int i = threadIdx.x; i < a.T * kDownRows; i += kMoeThreads) sums[i] = 0.0f;
  pdl_wait();
  {
    int* dst = reinterpret_cast<int*>(&r);
    for (int i = threadIdx.x; i < kRouteInts; i += kMoeThreads) dst[i] = a.route[i];
  }
  __syncthreads();
  const int units = r.n_groups * nkb;
  const int u0 = (int)((long long)rank * units / C), u1 = (int)((long long)(rank + 1) * units / C);
  const int row = d0 + warp * 16;
  const bool on = row < a.H;  // H is a multiple of 16
  const uint32_t ring = smem_u32(smem + DownSmem::kRing) + warp * kDownRing * kUnitBytes;
  int lu = u0, lg = u0 / nkb, lb = u0 - lg * nkb;  // the next unit to load: group, block
  auto issue = [&](uint32_t slot) {
    if (lu < u1) {
      if (on) {
        const int e = r.expert[lg], k = lb * kBlock;
        const uint8_t* w = a.w2 + ((size_t)e * a.H + row + g) * a.I + k + 16 * q;
        const float* s = a.s2 + ((size_t)e * rb + row / kBlock) * nkb + lb;
        unit_load(slot, w, w + (size_t)8 * a.I, a.I - k - 16 * q, s, s, lane);
      }
      ++lu;
      if (++lb == nkb) {
        lb = 0;
        ++lg;
      }
    }
    copies_commit();
  };
  for (int i = 0; i < kDownRing; ++i) issue(ring + i * kUnitBytes);
  uint32_t slot = ring;
  for (int u = u0; u < u1;) {
    const int grp = u / nkb, b0 = u - grp * nkb;
    const int np = r.count[grp], p0 = r.first[grp];
    auto run = [&](auto tag) {
      constexpr int NT = decltype(tag)::value;
      constexpr int kWin = stage_window(DownSmem::kStageBytes, NT);
      static_assert(8 * NT * kWin <= kStageScales, "column scales");
      const int nb = min(min(kWin, nkb - b0), u1 - u);
      const Stage st{smem + DownSmem::kStage, reinterpret_cast<float*>(smem + DownSmem::kScale), 8 * NT,
                     kWin * kBlock + 16};
      __syncthreads();  // the stage has been read
      stage_tokens<kDownTerms, float>(st, np, b0, nb, a.I, [&](int n) { return a.h + (size_t)r.pairs[p0 + n] * a.I; });
      __syncthreads();
      float acc[NT][4] = {};
      for (int b = 0; b < nb; ++b) {
        copies_wait<kDownRing - 1>();
        __syncwarp();
        if (on) unit_product<NT>(slot, st, b, lane, acc);
        __syncwarp();
        issue(slot);
        slot = slot == ring + (kDownRing - 1) * kUnitBytes ? ring : slot + kUnitBytes;
      }
      // An expert appears once in a token's choices, so the columns are
      // different tokens: no two lanes add to one place, no two warps share a row.
      if (on) {
#pragma unroll
        for (int n = 0; n < NT; n += kDownTerms)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int m = (n / kDownTerms) * 8 + 2 * q + c;
            if (m < np) {
              const int pc = r.pairs[p0 + m];
              float* dst = sums + (size_t)(pc / a.topk) * kDownRows + warp * 16 + g;
              const float p = r.p[pc];
              dst[0] = fmaf(p, acc[n][c] + acc[n + 1][c] + acc[n + 2][c], dst[0]);
              dst[8] = fmaf(p, acc[n][2 + c] + acc[n + 1][2 + c] + acc[n + 2][2 + c], dst[8]);
            }
          }
        __syncwarp();
      }
      u += nb;
    };
    if (np <= 8)
      run(Int<3>{});
    else if (np <= 16)
      run(Int<6>{});
    else
      run(Int<12>{});
  }
  copies_wait<0>();
  if (C > 1)
    cluster_sync_all();  // every CTA's sums are complete
  else
    __syncthreads();
  // this CTA's share of the outputs, two neighbouring rows a thread
  const int pairs_of = a.T * (kDownRows / 2);
  const int i1 = (int)((long long)(rank + 1) * pairs_of / C);
  const uint32_t base = smem_u32(sums);
  for (int i = (int)((long long)rank * pairs_of / C) + threadIdx.x; i < i1; i += kMoeThreads) {
    const int t = i / (kDownRows / 2), d = d0 + 2 * (i - t * (kDownRows / 2));
    if (d >= a.H) continue;
    float2 v = make_float2(0.0f, 0.0f);
    for (int c = 0; c < C; ++c) {
      const float2 o = ld_shared_cluster_f2(C > 1 ? mapa_shared(base + i * 8, (uint32_t)c) : base + i * 8);
      v.x += o.x;
      v.y += o.y;
    }
    __nv_bfloat16* y = a.y + (size_t)t * a.ldy + d;
    y[0] = __float2bfloat16_rn(v.x);
    y[1] = __float2bfloat16_rn(v.y);
  }
  if (C > 1) cluster_sync_all();  // no CTA leaves while a peer reads its sums
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
  static bool up_done[64] = {}, down_done[64] = {};
  cudaError_t e = opt_in_smem((const void*)moe_gate_up_kernel, UpSmem::kBytes, up_done);
  if (e == cudaSuccess)
    e = opt_in_smem((const void*)moe_down_kernel, DownSmem::bytes(kMoeMaxTokens), down_done);
  if (e != cudaSuccess) return e;
  // as many CTAs as reside at once, or one per column group if that is less
  const long long most = (long long)T * topk * (I / 8);
  const long long grid = most < dev->sms * 2 ? most : dev->sms * 2;
  void* up_args[] = {&a};
  e = launch_pdl((const void*)moe_gate_up_kernel, dim3((unsigned)grid), dim3(kMoeThreads), UpSmem::kBytes, 1, stream,
                 up_args);
  if (e != cudaSuccess) return e;
  // the widest cluster with which every CTA has an SM of its own
  const int row_tiles = (H + kDownRows - 1) / kDownRows;
  int C = 8;
  while (C > 1 && row_tiles * C > dev->sms) C /= 2;
  void* down_args[] = {&a, &C};
  return launch_pdl((const void*)moe_down_kernel, dim3((unsigned)(row_tiles * C)), dim3(kMoeThreads),
                    DownSmem::bytes(T), C, stream, down_args);
}

}  // namespace fp8
}  // namespace sharq
