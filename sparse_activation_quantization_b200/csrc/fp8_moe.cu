// fp8_moe.cu - a whole mixture-of-experts layer for a few tokens: two kernels up to
// 8 tokens, one more that chooses the experts above, and with more than 4 tokens
// an expert on average one that prepares h between the two.
//
//   chosen(t) = the k largest router logits of token t (ties: lower index)
//   p(t, j)   = softmax of the logits over the chosen (or over all) experts
//   h(t, j)   = silu(W_gate[e] x_t) * (W_up[e] x_t),        e = chosen(t)[j]
//   y_t       = sum_j p(t, j) W_down[e] h(t, j)
//
// Weights are E4M3 with a float32 scale per 128 x 128 block, activations bf16.
// With a few tokens the layer is bound by reading each chosen expert's weights
// once, so both kernels stream them through tcgen05 (fp8_skinny.cuh) against up
// to 32 tokens.  Activations enter the E4M3 MMAs without being quantized to E4M3:
// a value v of a 128-k block, scaled by a power of two that puts the block's
// largest into [128, 256), is written as v1 + v2 / 16 (+ v3 / 256), each an E4M3
// number, the rounded remainder of the one before.  Each term is a column of the
// MMA's B operand of its own, and the columns of a token are added at the end
// with its power of two.  Four bits a term: two terms hold a bf16 activation
// exactly where it is at least 2^-13 of the block's largest, and to 2^-21 of that
// largest below; three hold h to 2^-12 of itself or 2^-25 of its block's largest,
// whichever is more (half the spacing of the last term's smallest numbers).
//   gate-up  item = (group of tokens of one expert, 64 columns of h): the unit's
//            128 rows are 16 gate rows, the 16 up rows of the same columns, and so
//            on, so gate and up of a column meet in one warp.  Each CTA walks a
//            share of the items; with few of them a cluster shares an item's K
//            and joins its sums over distributed shared memory.
//   down     a cluster of CTAs owns 128 rows of W_down for all tokens; each CTA
//            takes a share of the (group, k block) units and sums p * result per
//            token in shared memory; the CTAs' sums are joined in rank order over
//            distributed shared memory.  Where there are few row tiles several
//            clusters share one, and the last of them adds their parts in order.
// Warps of a CTA: 0-3 sums, 4 copies (one thread), 5 MMAs (one thread) and TMEM,
// 6-9 form the columns, a unit each in turn.  Up to 8 tokens every CTA chooses their
// experts itself, a warp per token; above that a small kernel does it before (64
// tokens on ten warps took 15 us of gate-up).  Down does not wait for gate-up to
// derive the routing and to fill its ring with weights.
// No atomics touch results; the order of every sum follows from the routing.
#include "fp8_skinny.cuh"

namespace sharq {
namespace fp8 {

constexpr int kMoeMaxTokens = 64, kMoeMaxTopk = 16, kMoeMaxExperts = 512;

namespace {

constexpr int kFormWarps = 4, kFirstFormWarp = kSumWarps + 2;
constexpr int kMoeWarps = kFirstFormWarp + kFormWarps;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopk;
constexpr int kUpTerms = 2, kDownTerms = 3;  // E4M3 terms of a value of x and of h

struct MoeArgs {
  const __nv_bfloat16* x;   // [T][H]
  const float* logits;      // [T][E]
  const float* s13;         // [E][blocks(2 I)][blocks(H)]: gate rows, then up rows
  const float* s2;          // [E][blocks(H)][blocks(I)]
  __nv_bfloat16* y;         // [T][H]
  int* ids;                 // [T][topk] or nullptr
  float* weights;           // [T][topk] or nullptr
  int* err;                 // workspace: the error word
  int* choice;              // workspace: [T * topk] experts and weights of the choice kernel
  float* choice_p;
  int* arrived;             // workspace: down's arrivals [tile][8], zero between calls
  float* partial;           // workspace: down's partial sums [tile][parts][T][128]
  float* h;                 // workspace: [T * topk][I]
  uint8_t* x_terms;         // workspace, groups of 32 only: terms of x and h and their scales (Terms)
  uint8_t* h_terms;
  float* x_scale;
  float* h_scale;
  long long ldx, ldl, ldy;
  int T, E, topk, H, I, renorm;
  int splits;               // CTAs of a cluster
  int parts;                // down: clusters that share a tile
};

// The routing in shared memory: per expert the (token, choice) pairs
// t * topk + j that chose it, cut into groups of at most G tokens.  G = 8 for
// calls of up to 8 tokens, whose groups never hold more.
constexpr int kSmallGroup = 8, kGroup = 32;
// n experts that P pairs chose are at most n + (P - n) / G groups: one each, and one more for every G further tokens.
// That grows with n and is largest for the smaller G, with every expert chosen.
constexpr int kMaxGroups = kMoeMaxExperts + (kMaxPairs - kMoeMaxExperts) / kSmallGroup;
static_assert(kSmallGroup <= kGroup && kMoeMaxExperts <= kMaxPairs, "the bound above");
struct Group {
  short expert, first, count, form;  // first of its pairs, their number, tokens_form of it
};
struct Routing {
  int n_groups, n_pairs;
  float p[kMaxPairs];        // by pair id
  short pairs[kMaxPairs];    // pair ids, expert by expert, by token
  short token[kMaxPairs];    // their tokens
  Group groups[kMaxGroups];  // experts ascending
};
struct __align__(8) RoutingScratch {
  uint32_t chose[2 * kMoeMaxExperts];  // two words an expert, bit t: token t chose it
  short first[kMoeMaxExperts];
  short expert_of[kMaxPairs];
};

// the form that takes a group of np tokens
__device__ __forceinline__ int tokens_form(int np) { return np <= 8 ? 8 : (np <= 16 ? 16 : 32); }

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

// The k largest logits of a token and their weights, by one warp: lane j < topk
// gets the j-th.  kPer: logits per lane.  A round is two warp reductions (the
// largest key, then the lowest expert that has it) and no branch: about 100
// cycles.
template <int kPer>
__device__ __forceinline__ void choose(const MoeArgs& a, int t, int& my_e, float& my_p) {
  const int lane = threadIdx.x & 31;
  const float* lg = a.logits + (size_t)t * a.ldl;
  float l[kPer];
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) l[i] = lane + 32 * i < a.E ? __ldcg(lg + lane + 32 * i) : -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < a.E ? max(logit_key(l[i]), 1u) : 0u;  // 0: absent, or taken
  uint32_t my_key = 0u, first = 0u;
  my_e = 0;
  for (int j = 0; j < a.topk; ++j) {
    uint32_t k[kPer];
    int at[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      k[i] = key[i];
      at[i] = lane + 32 * i;
    }
#pragma unroll
    for (int w = 1; w < kPer; w *= 2)  // equal keys: the lower expert stays
#pragma unroll
      for (int i = 0; i + w < kPer; i += 2 * w) {
        const bool up = k[i + w] > k[i];
        k[i] = up ? k[i + w] : k[i];
        at[i] = up ? at[i + w] : at[i];
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, k[0]);
    const int e = __reduce_min_sync(0xffffffffu, k[0] == top ? at[0] : 0x7fffffff);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i == e ? 0u : key[i];
    if (j == 0) first = top;
    my_key = lane == j ? top : my_key;
    my_e = lane == j ? e : my_e;
  }
  const float lmax = key_logit(first);
  const float mine = lane < a.topk ? logit_exp(key_logit(my_key), lmax) : 0.0f;
  float sum = mine;
  if (!a.renorm) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += logit_exp(l[i], lmax);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  my_p = sum > 0.0f ? __fdiv_rn(mine, sum) : 0.0f;  // no logit above -inf: no expert counts
}
__device__ __forceinline__ void choose_any(const MoeArgs& a, int t, int& e, float& p) {
  if (a.E <= 128)
    choose<4>(a, t, e, p);
  else
    choose<kMoeMaxExperts / 32>(a, t, e, p);
}
__device__ __forceinline__ void publish_choice(const MoeArgs& a, int pr, int e, float p) {
  if (a.ids) a.ids[pr] = e;
  if (a.weights) a.weights[pr] = p;
}

__device__ __forceinline__ unsigned long long tokens_of(const RoutingScratch& sc, int e) {
  return *reinterpret_cast<const unsigned long long*>(&sc.chose[2 * e]);
}

// The whole routing, from the logits (kChoose: at most a token per warp) or from
// the choice kernel's list.  Every CTA derives the same.  Ends with a barrier.
template <int G, bool kChoose>
__device__ void build_routing(const MoeArgs& a, Routing& r, RoutingScratch& sc, bool publish) {
  if (kChoose && a.T == 1) {  // every choice is a group of its own, in the order of choice
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int e;
      float p;
      choose_any(a, 0, e, p);
      const bool in = lane < a.topk && p > 0.0f;
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      const int at = __popc(all & ((1u << lane) - 1u));
      if (in) {
        r.groups[at] = Group{(short)e, (short)at, 1, (short)tokens_form(1)};
        r.pairs[at] = (short)lane;
        r.token[at] = 0;
        r.p[lane] = p;
      }
      if (lane == 0) r.n_groups = r.n_pairs = __popc(all);
      if (publish && lane < a.topk) publish_choice(a, lane, e, p);
    }
    __syncthreads();
    return;
  }
  const int pairs = a.T * a.topk;
  constexpr int kList = (kMaxPairs + kMoeThreads - 1) / kMoeThreads;
  int le[kList];
  float lp[kList];
  if (!kChoose) {
#pragma unroll
    for (int j = 0; j < kList; ++j) {
      const int i = j * kMoeThreads + (int)threadIdx.x;
      le[j] = i < pairs ? __ldcg(a.choice + i) : 0;
      lp[j] = i < pairs ? __ldcg(a.choice_p + i) : 0.0f;
    }
  }
  for (int i = threadIdx.x; i < 2 * a.E; i += kMoeThreads) sc.chose[i] = 0u;
  __syncthreads();
  auto enter = [&](int pr, int t, int e, float p) {
    r.p[pr] = p;
    sc.expert_of[pr] = p > 0.0f ? (short)e : (short)-1;  // weight 0: the expert is not evaluated
    if (p > 0.0f) atomicOr(&sc.chose[2 * e + (t >> 5)], 1u << (t & 31));
  };
  if (kChoose) {
    static_assert(!kChoose || kSmallGroup <= kMoeWarps, "a token per warp");
    const int t = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (t < a.T) {
      int e;
      float p;
      choose_any(a, t, e, p);
      if (lane < a.topk) {
        enter(t * a.topk + lane, t, e, p);
        if (publish) publish_choice(a, t * a.topk + lane, e, p);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kList; ++j) {
      const int i = j * kMoeThreads + (int)threadIdx.x;
      if (i < pairs) enter(i, i / a.topk, le[j], lp[j]);
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // lay the experts' pairs out one after another, in groups; a run of experts per lane
    const int per = (a.E + 31) / 32, e0 = threadIdx.x * per, e1 = min(a.E, e0 + per);
    int sum = 0;  // pairs in the low half, groups in the high
    for (int e = e0; e < e1; ++e) {
      const int c = __popcll(tokens_of(sc, e));
      sum += c + ((c + G - 1) / G << 16);
    }
    int at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if ((int)threadIdx.x >= o) at += v;
    }
    if (threadIdx.x == 31) {
      r.n_groups = at >> 16;
      r.n_pairs = at & 0xffff;
    }
    at -= sum;
    int np = at & 0xffff, ng = at >> 16;
    for (int e = e0; e < e1; ++e) {
      const int c = __popcll(tokens_of(sc, e));
      sc.first[e] = (short)np;
      for (int i = 0; i < c; i += G) {
        const int n = min(G, c - i);
        r.groups[ng++] = Group{(short)e, (short)(np + i), (short)n, (short)tokens_form(n)};
      }
      np += c;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.topk; i += kMoeThreads) {
    const int e = sc.expert_of[i], t = i / a.topk;
    if (e >= 0) {
      const int at = sc.first[e] + __popcll(tokens_of(sc, e) & ((1ull << t) - 1));
      r.pairs[at] = (short)i;
      r.token[at] = (short)t;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------ columns on the fly ---
// A form for P tokens (8, 16 or 32) has J P columns, term j of token t at j P + t.

// eight values as they lie in memory
template <class T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
      unpack_bf16x8(v[0], f);
    } else {
      const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
};

// The terms of eight values of a block whose largest is m, and their scale: the
// values times 2^(7 - floor(log2 m)), the factor from the exponent field, whose
// clamp keeps it and its inverse normal numbers.
template <int J>
__device__ __forceinline__ float split_terms(float (&v)[8], float m, uint2 (&term)[J]) {
  const uint32_t ef = max(__float_as_uint(m) >> 23, 20u);
  const float up = __uint_as_float((261u - ef) << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= up;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const uint32_t c0 = e4m3x4(v[0], v[1], v[2], v[3]), c1 = e4m3x4(v[4], v[5], v[6], v[7]);
    term[j] = make_uint2(c0, c1);
    if (j + 1 < J) {
      const float2 d0 = e4m3x2_to_float(c0), d1 = e4m3x2_to_float(c0 >> 16);
      const float2 d2 = e4m3x2_to_float(c1), d3 = e4m3x2_to_float(c1 >> 16);
      v[0] = (v[0] - d0.x) * 16.0f, v[1] = (v[1] - d0.y) * 16.0f;
      v[2] = (v[2] - d1.x) * 16.0f, v[3] = (v[3] - d1.y) * 16.0f;
      v[4] = (v[4] - d2.x) * 16.0f, v[5] = (v[5] - d2.y) * 16.0f;
      v[6] = (v[6] - d3.x) * 16.0f, v[7] = (v[7] - d3.y) * 16.0f;
    }
  }
  return ef == 255u ? INFINITY : __uint_as_float((ef - 7u) << 23);  // an infinity saturates in E4M3: it is in the scale
}

// Block b of np tokens into a stage's B operand (128-byte swizzle) and scales, by
// one warp: half a warp per token, eight values a lane, kBatch tokens of each half
// side by side.  rows(n): token n's row; weights(n): a factor of its scale.
// Columns of no token keep what they held: their sums are not used.  ready():
// returns once the stage is free.  It is asked only when the first terms are at
// hand, so that loads and arithmetic lie outside the ring's round trip (they are
// 2000 of its 3300 cycles at one token).
template <int J, class T, int kBatch, class Rows, class Weights, class Ready>
__device__ __forceinline__ void form_batch(uint8_t* dst, float* scale, int n0, int np, int P, int b, int K, Rows rows,
                                           Weights weights, Ready ready) {
  const int lane = threadIdx.x & 31, l16 = lane & 15, half = lane >> 4;
  const int k = b * kBlock + l16 * 8;
  Raw8<T> raw[kBatch];  // every load is on its way before the first value is used
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int n = n0 + 2 * i + half;
    raw[i].clear();
    if (n < np && k < K) raw[i].load(static_cast<const T*>(rows(n)) + k);
  }
  float f[kBatch][8], m[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    raw[i].floats(f[i]);
    m[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[i] = fmaxf(m[i], fabsf(f[i][e]));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
  float sc[kBatch];
  uint2 term[kBatch][J];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int n = n0 + 2 * i + half;
    sc[i] = split_terms<J>(f[i], m[i], term[i]) * (n < np ? weights(n) : 1.0f);
  }
  if (!ready()) return;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int n = n0 + 2 * i + half;
    if (n < np) {
      if (l16 == 0) scale[n] = sc[i];
#pragma unroll
      for (int j = 0; j < J; ++j)
        *reinterpret_cast<uint2*>(dst + codes_chunk_off((uint32_t)(j * P + n), l16 >> 1) + (l16 & 1) * 8) = term[i][j];
    }
  }
}
// Returns false if the stage did not become free.
template <int J, class T, class Rows, class Weights, class Wait>
__device__ __forceinline__ bool form_columns(uint8_t* dst, float* scale, int np, int P, int b, int K, Rows rows,
                                             Weights weights, Wait wait) {
  bool free = false;
  auto ready = [&]() {
    if (!free) free = __all_sync(0xffffffffu, wait());
    return free;
  };
  int n0 = 0;
  for (; np - n0 > 4; n0 += 8) form_batch<J, T, 4>(dst, scale, n0, np, P, b, K, rows, weights, ready);
  if (np - n0 > 2)
    form_batch<J, T, 2>(dst, scale, n0, np, P, b, K, rows, weights, ready);
  else if (np > n0)
    form_batch<J, T, 1>(dst, scale, n0, np, P, b, K, rows, weights, ready);
  return free;
}

// Where groups are large, every CTA would form the same columns for each of its
// tiles: 2000 cycles of a unit at 32 tokens, and the tiles' loads wait for it.
// Then the terms are formed once, as [row][block][term][128] with a scale per row
// and block, and only gathered here (measured at 16 experts of 2048 x 768, 64
// tokens with 8 choices: 84 us formed, 61 us gathered).
template <int J, class T>
__device__ __forceinline__ void store_terms(const T* src, long long ld, int rows, int K, uint8_t* codes, float* scale,
                                            int cta, int ctas) {
  const int nkb = blocks_of(K), total = rows * nkb, l16 = threadIdx.x & 15, per = (int)(blockDim.x >> 4);
  const int here = cta * per + (int)(threadIdx.x >> 4);
  for (int i0 = here; i0 - (int)((threadIdx.x >> 4) & 1) < total; i0 += ctas * per) {  // uniform over the warp
    const int i = min(i0, total - 1), row = i / nkb, b = i - row * nkb, k = b * kBlock + l16 * 8;
    Raw8<T> raw;
    raw.clear();
    if (k < K) raw.load(src + (size_t)row * ld + k);
    float f[8], m = 0.0f;
    raw.floats(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    uint2 term[J];
    const float s = split_terms<J>(f, m, term);
    if (i0 < total) {
      if (l16 == 0) scale[i] = s;
#pragma unroll
      for (int j = 0; j < J; ++j) *reinterpret_cast<uint2*>(codes + ((size_t)i * J + j) * kBlock + l16 * 8) = term[j];
    }
  }
}
template <int J, class Rows, class Weights, class Wait>
__device__ __forceinline__ bool gather_columns(uint8_t* dst, float* scale, int np, int P, int b, int nkb,
                                               const uint8_t* codes, const float* scales, Rows rows, Weights weights,
                                               Wait wait) {
  const int lane = threadIdx.x & 31;
  constexpr int kChunks = J * kBlock / 16, kBatch = 8;  // 16-byte chunks of a token's block; loads on their way
  const int total = np * kChunks;
  const float s = lane < np ? __ldcg(scales + (size_t)rows(lane) * nkb + b) * weights(lane) : 0.0f;
  bool free = false;
  for (int i0 = 0; i0 < total; i0 += 32 * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + 32 * q + lane, n = i / kChunks, c = i - n * kChunks;
      if (i < total)
        v[q] = __ldcg(reinterpret_cast<const uint4*>(codes + ((size_t)rows(n) * nkb + b) * (J * kBlock)) + c);
    }
    if (!free) {
      free = __all_sync(0xffffffffu, wait());
      if (!free) return false;
      if (lane < np) scale[lane] = s;
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + 32 * q + lane, n = i / kChunks, c = i - n * kChunks;
      if (i < total)
        *reinterpret_cast<uint4*>(dst + codes_chunk_off((uint32_t)((c >> 3) * P + n), (uint32_t)c & 7)) = v[q];
    }
  }
  return free;
}

__host__ __device__ constexpr int mma_n(int cols) { return (cols + 15) / 16 * 16; }

// One unit's MMAs, by the issuing thread, which has seen the stage's columns and
// scales arrive and therefore arrives on done itself as well: who waits for done
// then sees the scales too, and the sum warps need not wait on full.  `ready`:
// whether this unit was full when it was asked for; on return, whether the next
// one is.  (A question asked behind MMAs is answered when they are taken in, 200
// cycles later: it is asked before them.)
template <int kStages>
__device__ __forceinline__ bool issue_unit(SkinnyBars<kStages>& bars, RingPos<kStages>& p, bool& ready, uint32_t tmem,
                                           int stage_cols, const uint8_t* ring, int stage_bytes, uint32_t idesc,
                                           uint64_t deadline) {
  if (!ready && !mbar_wait(&bars.full[p.s], p.phase, deadline, &bars.abort)) return false;
  const int s = p.s;
  p.next();
  ready = mbar_test(&bars.full[p.s], p.phase);
  tc_fence_after();
  unit_mma(tmem + s * stage_cols, smem_u32(ring + s * stage_bytes), idesc);
  tc_commit(&bars.done[s]);
  mbar_arrive_cta(&bars.done[s]);
  return true;
}

// One unit's sums: acc[t] += (c1 + c2 / 16 (+ c3 / 256)) scale[t] s_w.  `seen`: the
// unit was done when it was asked for; on return, whether the next one is.  Where
// a wait runs out the flag is set and the warp goes on as one, with sums that
// nobody stores.
template <int J, int P, int kStages>
__device__ __forceinline__ void add_unit(SkinnyBars<kStages>& bars, RingPos<kStages>& pos, bool& seen,
                                         uint32_t tmem_lane, int stage_cols, const float* scale, float s_w,
                                         float (&acc)[P], int* err, int lane) {
  if (!seen && !mbar_wait_short(&bars.done[pos.s], pos.phase, &bars.abort)) bars.give_up(err);
  __syncwarp();
  tc_fence_after();
  float s[P];
#pragma unroll
  for (int t = 0; t < P; t += 4) {
    const float4 s4 = *reinterpret_cast<const float4*>(scale + t);
    s[t] = s4.x, s[t + 1] = s4.y, s[t + 2] = s4.z, s[t + 3] = s4.w;
  }
  uint32_t v[J * P];
  tmem_read(tmem_lane + pos.s * stage_cols, v);
  tmem_ld_wait();
  release_unit(bars, pos, lane);
  pos.next();
  seen = mbar_test(&bars.done[pos.s], pos.phase);  // answered while this unit is added
#pragma unroll
  for (int t = 0; t < P; ++t) {
    float c = __uint_as_float(v[(J - 1) * P + t]);
#pragma unroll
    for (int j = J - 2; j >= 0; --j) c = fmaf(c, 0.0625f, __uint_as_float(v[j * P + t]));
    acc[t] = fmaf(c, s[t] * s_w, acc[t]);
  }
}

// The weight scales of a unit whose 32 rows a warp are 16 gate rows and 16 up rows:
// each half of the warp holds its row's scales, 16 blocks at a time.
struct HalfScales {
  const float* p;
  int n, base;
  float cur, ahead;
  __device__ __forceinline__ float load(int b) const { return b < n ? p[b] : 0.0f; }
  __device__ __forceinline__ void start(const float* row, int blocks, int b0, int lane) {
    p = row;
    n = blocks;
    base = b0;
    cur = load(b0 + (lane & 15));
    ahead = load(b0 + 16 + (lane & 15));
  }
  __device__ __forceinline__ float at(int b, int lane) {  // b ascends
    if (b - base >= 16) {
      base += 16;
      cur = ahead;
      ahead = load(base + 16 + (lane & 15));
    }
    return __shfl_sync(0xffffffffu, cur, (lane & 16) | (b - base));
  }
};

template <int J, int G, int Stages>
struct MoeRing {
  static constexpr int kStages = Stages;
  static constexpr int kCols = mma_n(J * G);
  static constexpr int kStageBytes = kUnitBytes + kCols * kBlock;
  static constexpr int kTmem = tmem_cols(kCols * kStages);
  static constexpr int kBytes = kStages * kStageBytes;
  // Warps that form columns, a unit each in turn.  Never more than stages: a warp that comes to unit i has formed
  // unit i - kFormers, so every stage up to unit i - kFormers - kStages has been emptied, and the parity that it
  // waits for (unit i - kStages) can only be the next to come, not one two uses back.
  static constexpr int kFormers = kFormWarps < kStages ? kFormWarps : kStages;
  static_assert(kTmem <= 512 && kStageBytes % 1024 == 0, "ring");
};

// Where part i of n begins among `total`.  In 32 bits: at most kMaxGroups (576)
// groups of 2048 column tiles or 1024 k blocks, and a few hundred CTAs.
__device__ __forceinline__ int share_of(int i, int total, int n) {
  return (int)((uint32_t)i * (uint32_t)total / (uint32_t)n);
}

template <int P>
struct Tokens {
  static constexpr int value = P;
};

// start-up common to both kernels: barriers, TMEM
template <class R>
__device__ __forceinline__ void moe_setup(SkinnyBars<R::kStages>& bars, const CUtensorMap* map) {
  if (threadIdx.x == kSumWarps * 32) {
    tma_prefetch_map(map);
    bars.init(2, 2);  // full: the copy and the forming warp; done: the MMAs and the thread that issued them
  }
  if (threadIdx.x >> 5 == kSumWarps + 1) {
    tmem_alloc(&bars.tmem, R::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}
template <class R>
__device__ __forceinline__ void moe_teardown(uint32_t tmem) {
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x >> 5 == kSumWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, R::kTmem);
  }
}

// ---------------------------------------------- before gate-up and down ---

// The choices of every token, a warp each, where they do not fit the first wave of
// gate-up's own warps.
constexpr int kChooseWarps = 8;
__global__ void __launch_bounds__(32 * kChooseWarps) moe_choose_kernel(const MoeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int choosers = (a.T + kChooseWarps - 1) / kChooseWarps;
  if ((int)blockIdx.x >= choosers) {  // the other CTAs: the terms of x
    store_terms<kUpTerms>(a.x, a.ldx, a.T, a.H, a.x_terms, a.x_scale, (int)blockIdx.x - choosers,
                          (int)gridDim.x - choosers);
    return;
  }
  const int t = (int)(blockIdx.x * kChooseWarps + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (t >= a.T) return;
  int e;
  float p;
  choose_any(a, t, e, p);
  if (lane < a.topk) {
    const int pr = t * a.topk + lane;
    a.choice_p[pr] = p;
    a.choice[pr] = e;
    publish_choice(a, pr, e, p);
  }
}
// The terms of h, between gate-up and down.
__global__ void __launch_bounds__(256) moe_terms_kernel(const MoeArgs a) {
  pdl_trigger();
  pdl_wait();
  store_terms<kDownTerms>(a.h, (long long)a.I, a.T * a.topk, a.I, a.h_terms, a.h_scale, (int)blockIdx.x,
                          (int)gridDim.x);
}

// ---------------------------------------------------------------- gate-up ---

constexpr int kUpCols = 64;
template <int G>
struct Up : MoeRing<kUpTerms, G, G == kSmallGroup ? 5 : 8> {
  // several CTAs of the small form, and down's beside them, reside on an SM
  static constexpr int kSmemBytes = Up::kBytes + 1024;
};

template <int G, bool kChoose>
__global__ void __launch_bounds__(kMoeThreads, G == kSmallGroup ? 2 : 1)
    moe_gate_up_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
  using C = Up<G>;
  using Pos = RingPos<C::kStages>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routing r;
  __shared__ __align__(8) SkinnyBars<C::kStages> bars;
  __shared__ __align__(16) float scale[C::kStages][G];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  moe_setup<C>(bars, &map);
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  build_routing<G, kChoose>(a, r, *reinterpret_cast<RoutingScratch*>(smem), blockIdx.x == 0);
  pdl_trigger();  // after the allocation, and after the kernels before (logits, choices) are complete
  const int nkb = blocks_of(a.H), tiles = (a.I + kUpCols - 1) / kUpCols, items = r.n_groups * tiles;
  const int S = a.splits, rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int cl = (int)blockIdx.x / S, ncl = (int)gridDim.x / S;  // with S > 1 there are as many clusters as items
  const int it0 = share_of(cl, items, ncl), it1 = share_of(cl + 1, items, ncl);
  const int b0 = rank * nkb / S, b1 = (rank + 1) * nkb / S;
  const uint64_t deadline = globaltimer_ns() + kWaitNs;
  fence_proxy_async_smem();  // the scratch was written where copies land
  __syncthreads();

  if (warp == kSumWarps) {
    if (elect_one()) {
      Pos p;
      int n = 0;
      for (int it = it0; it < it1 && !bars.abort; ++it) {
        const int grp = it / tiles, i0 = (it - grp * tiles) * kUpCols, e = r.groups[grp].expert;
        for (int b = b0; b < b1; ++b, ++n, p.next()) {
          if (!wait_empty(bars, p, deadline)) {
            bars.give_up(a.err);
            break;
          }
          mbar_arrive_expect_tx(&bars.full[p.s], kUnitBytes);
          tma_5d(smem + p.s * C::kStageBytes, &map, b * kBlock, 0, 0, i0 / 16, e, &bars.full[p.s]);
        }
      }
      if (bars.abort) drain_copies(bars, n);
    }
  } else if (warp == kSumWarps + 1) {
    if (elect_one()) {
      Pos p;
      bool ready = false;
      for (int it = it0; it < it1 && !bars.abort; ++it) {
        const uint32_t idesc = idesc_e4m3(kUnitRows, mma_n(kUpTerms * r.groups[it / tiles].form));
        for (int b = b0; b < b1; ++b)
          if (!issue_unit(bars, p, ready, tmem, C::kCols, smem, C::kStageBytes, idesc, deadline)) {
            bars.give_up(a.err);
            break;
          }
      }
    }
  } else if (warp >= kFirstFormWarp) {
    Pos p;
    static_assert(C::kFormers == kFormWarps, "every former has a turn");
    int turn = warp - kFirstFormWarp;  // units until this warp's next
    for (int it = it0; it < it1 && !warp_stopped(&bars.abort); ++it) {
      const Group gr = r.groups[it / tiles];
      for (int b = b0; b < b1; ++b, p.next()) {
        if (turn-- > 0) continue;
        turn = C::kFormers - 1;
        uint8_t* dst = smem + p.s * C::kStageBytes + kUnitBytes;
        const auto one = [](int) { return 1.0f; };
        const auto wait = [&]() { return wait_empty(bars, p, deadline); };
        bool ok;
        if constexpr (G == kGroup)
          ok = gather_columns<kUpTerms>(dst, scale[p.s], gr.count, gr.form, b, nkb, a.x_terms, a.x_scale,
                                        [&](int n) { return (int)r.token[gr.first + n]; }, one, wait);
        else
          ok = form_columns<kUpTerms, __nv_bfloat16>(
              dst, scale[p.s], gr.count, gr.form, b, a.H,
              [&](int n) { return a.x + (size_t)r.token[gr.first + n] * a.ldx; }, one, wait);
        if (!ok) {
          bars.give_up(a.err);
          break;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&bars.full[p.s]);
      }
    }
  } else {
    Pos p;
    bool seen = false;
    const int rb = blocks_of(2 * a.I);
    const uint32_t tmem_lane = tmem + ((uint32_t)(warp * 32) << 16);
    // with S > 1 every sum warp has to come to its item's barrier
    for (int it = it0; it < it1 && (S > 1 || !warp_stopped(&bars.abort)); ++it) {
      const int grp = it / tiles, c0 = (it - grp * tiles) * kUpCols + 16 * warp;
      const int np = r.groups[grp].count, p0 = r.groups[grp].first;
      // the warp's 16 gate rows lie in one scale block, its up rows in another; rows past the last read zeros
      const float* s13 = a.s13 + (size_t)r.groups[grp].expert * rb * nkb;
      const int row = min(c0, a.I - 16);
      HalfScales sw;
      sw.start(s13 + (size_t)((lane < 16 ? row : a.I + row) / kBlock) * nkb, nkb, b0, lane);
      auto run = [&](auto form) {
        constexpr int P = decltype(form)::value;
        float acc[P] = {};
        for (int b = b0; b < b1; ++b) {
          const float s = sw.at(b, lane);
          add_unit<kUpTerms, P>(bars, p, seen, tmem_lane, C::kCols, scale[p.s], s, acc, a.err, lane);
        }
        if (S == 1) {
          const int col = c0 + (lane & 15);
#pragma unroll
          for (int t = 0; t < P; t += 2) {  // the lower lanes finish token t, the upper ones t + 1
            const float other = __shfl_xor_sync(0xffffffffu, lane < 16 ? acc[t + 1] : acc[t], 16);
            const int n = t + (lane >> 4);
            if (n < np && col < a.I && !bars.abort)
              a.h[(size_t)r.pairs[p0 + n] * a.I + col] =
                  lane < 16 ? silu_mul(acc[t], other) : silu_mul(other, acc[t + 1]);
          }
        } else {  // one item per cluster: the ring is free once every sum warp is here
          asm volatile("bar.sync 1, 128;" ::: "memory");
          float* out = reinterpret_cast<float*>(smem);
#pragma unroll
          for (int t = 0; t < P; ++t)
            if (t < np) out[t * kUnitRows + threadIdx.x] = acc[t];
        }
      };
      if (np <= 8)
        run(Tokens<8>{});
      else if (G > 8 && np <= 16)
        run(Tokens<G < 16 ? 8 : 16>{});
      else if (G > 16)
        run(Tokens<G < 32 ? 8 : 32>{});
    }
  }
  if (S > 1) {
    cluster_sync_all();  // every CTA's sums are in its shared memory
    if (it0 < it1 && !bars.abort) {
      const int grp = it0 / tiles, i0 = (it0 - grp * tiles) * kUpCols;
      const int np = r.groups[grp].count, p0 = r.groups[grp].first;
      const uint32_t base = smem_u32(smem);
      const int total = np * kUpCols;
      for (int i = rank * total / S + (int)threadIdx.x; i < (rank + 1) * total / S; i += kMoeThreads) {
        const int n = i / kUpCols, c = i - n * kUpCols;
        const uint32_t at = base + (n * kUnitRows + (c >> 4) * 32 + (c & 15)) * 4;
        float g = 0.0f, u = 0.0f;
        for (int q = 0; q < S; ++q) {
          const uint32_t peer = mapa_shared(at, (uint32_t)q);
          g += ld_shared_cluster_f(peer);
          u += ld_shared_cluster_f(peer + 64);
        }
        if (i0 + c < a.I) a.h[(size_t)r.pairs[p0 + n] * a.I + i0 + c] = silu_mul(g, u);
      }
    }
    cluster_sync_all();  // no CTA leaves while a peer reads its sums
  }
  moe_teardown<C>(tmem);
}

// ------------------------------------------------------------------- down ---

// kBeside: the form that fits an SM beside gate-up's (calls of up to 8 tokens).
template <int G, bool kBeside>
struct Down : MoeRing<kDownTerms, G, kBeside ? 4 : (G == kSmallGroup ? 3 : 5)> {
  static constexpr int kSums = Down::kBytes;  // [T][128]
  static constexpr int bytes(int T) { return kSums + T * kUnitRows * 4 + 1024; }
};
using BesideDown = Down<kSmallGroup, true>;
static_assert(Up<kSmallGroup>::kSmemBytes + BesideDown::bytes(kSmallGroup) + 2 * (int)sizeof(Routing) <= 226 * 1024 &&
              Up<kSmallGroup>::kTmem + BesideDown::kTmem <= 512, "both kernels' forms share an SM");
static_assert(2 * (Up<kSmallGroup>::kSmemBytes + (int)sizeof(Routing) + 2048) <= 226 * 1024 &&
              2 * (Down<kSmallGroup, false>::bytes(kMoeMaxTokens) + (int)sizeof(Routing) + 2048) <= 226 * 1024,
              "two CTAs of the small forms, with 2 KB of barriers and scales each, share an SM");

template <int G, bool kBeside>
__global__ void __launch_bounds__(kMoeThreads, G == kSmallGroup ? 2 : 1)
    moe_down_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
  using C = Down<G, kBeside>;
  using Pos = RingPos<C::kStages>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routing r;
  __shared__ __align__(8) SkinnyBars<C::kStages> bars;
  __shared__ __align__(16) float scale[C::kStages][G];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.splits, rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int cl = (int)blockIdx.x / S, tile = cl / a.parts, part = cl - tile * a.parts;
  const int d0 = tile * kUnitRows;
  const int nkb = blocks_of(a.I), rb = blocks_of(a.H);
  float* sums = reinterpret_cast<float*>(smem + C::kSums);
  moe_setup<C>(bars, &map);
  const uint32_t tmem = bars.tmem;
  pdl_trigger();  // after the allocation
  // Logits, choices and weights: complete before gate-up let this grid start.
  build_routing<G, kBeside>(a, r, *reinterpret_cast<RoutingScratch*>(smem), false);
  for (int i = threadIdx.x; i < a.T * kUnitRows; i += kMoeThreads) sums[i] = 0.0f;
  const int units = r.n_groups * nkb;
  const int share = part * S + rank, shares = a.parts * S;
  const int u0 = share_of(share, units, shares), u1 = share_of(share + 1, units, shares);
  const uint64_t deadline = globaltimer_ns() + 2 * kWaitNs;  // gate-up may still run
  fence_proxy_async_smem();  // the scratch was written where copies land
  __syncthreads();

  if (warp == kSumWarps) {
    if (elect_one()) {
      Pos p;
      int grp = u0 / nkb, b = u0 - grp * nkb, u = u0;
      for (; u < u1; ++u, p.next()) {
        if (!wait_empty(bars, p, deadline)) {
          bars.give_up(a.err);
          break;
        }
        mbar_arrive_expect_tx(&bars.full[p.s], kUnitBytes);
        tma_2d(smem + p.s * C::kStageBytes, &map, b * kBlock, r.groups[grp].expert * a.H + d0, &bars.full[p.s]);
        if (++b == nkb) {
          b = 0;
          ++grp;
        }
      }
      if (bars.abort) drain_copies(bars, u - u0);
    }
  } else if (warp == kSumWarps + 1) {
    if (elect_one()) {
      Pos p;
      bool ready = false;
      for (int u = u0; u < u1; ++u) {
        const uint32_t idesc = idesc_e4m3(kUnitRows, mma_n(kDownTerms * r.groups[u / nkb].form));
        if (!issue_unit(bars, p, ready, tmem, C::kCols, smem, C::kStageBytes, idesc, deadline)) {
          bars.give_up(a.err);
          break;
        }
      }
    }
  } else if (warp >= kFirstFormWarp) {
    pdl_wait();  // gate-up has ended: h is complete
    Pos p;
    for (int u = u0; u < u1; ++u, p.next()) {
      if ((u - u0) % C::kFormers != warp - kFirstFormWarp) continue;
      const int grp = u / nkb;
      const Group gr = r.groups[grp];
      uint8_t* dst = smem + p.s * C::kStageBytes + kUnitBytes;
      const auto weight = [&](int n) { return r.p[r.pairs[gr.first + n]]; };
      const auto wait = [&]() { return wait_empty(bars, p, deadline); };
      bool ok;
      if constexpr (G == kGroup)
        ok = gather_columns<kDownTerms>(dst, scale[p.s], gr.count, gr.form, u - grp * nkb, nkb, a.h_terms, a.h_scale,
                                        [&](int n) { return (int)r.pairs[gr.first + n]; }, weight, wait);
      else
        ok = form_columns<kDownTerms, float>(dst, scale[p.s], gr.count, gr.form, u - grp * nkb, a.I,
                                             [&](int n) { return a.h + (size_t)r.pairs[gr.first + n] * a.I; }, weight,
                                             wait);
      if (!ok) {
        bars.give_up(a.err);
        break;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars.full[p.s]);
    }
  } else {
    Pos p;
    bool seen = false;
    const uint32_t tmem_lane = tmem + ((uint32_t)(warp * 32) << 16);
    auto scales_of = [&](int grp, int b) {
      ScaleRow w;
      w.start(a.s2 + ((size_t)r.groups[grp].expert * rb + d0 / kBlock) * nkb, nkb, b, lane);
      return w;
    };
    ScaleRow ahead;
    if (u0 < u1) ahead = scales_of(u0 / nkb, u0 % nkb);
    for (int u = u0; u < u1 && !warp_stopped(&bars.abort);) {
      const int grp = u / nkb, bb = u - grp * nkb, be = min(nkb, bb + u1 - u);
      const int np = r.groups[grp].count, p0 = r.groups[grp].first;
      ScaleRow sw = ahead;
      if (grp + 1 < r.n_groups) ahead = scales_of(grp + 1, 0);  // read while this group is summed
      auto run = [&](auto form) {
        constexpr int P = decltype(form)::value;
        float acc[P] = {};
        for (int b = bb; b < be; ++b) {
          const float s = sw.at(b, lane);
          add_unit<kDownTerms, P>(bars, p, seen, tmem_lane, C::kCols, scale[p.s], s, acc, a.err, lane);
        }
        // This thread alone adds to its row's sums, and a group's tokens are different ones: an expert appears
        // once in a token's choices.
#pragma unroll
        for (int n0 = 0; n0 < P; n0 += 8) {
          float* at[8];
          float old[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + i < np) {
              at[i] = sums + (size_t)r.token[p0 + n0 + i] * kUnitRows + threadIdx.x;
              old[i] = *at[i];
            }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + i < np) *at[i] = old[i] + acc[n0 + i];
        }
      };
      if (np <= 8)
        run(Tokens<8>{});
      else if (G > 8 && np <= 16)
        run(Tokens<G < 16 ? 8 : 16>{});
      else if (G > 16)
        run(Tokens<G < 32 ? 8 : 32>{});
      u += be - bb;
    }
  }
  pdl_wait();  // y may be x: no store before gate-up has ended (a CTA without units comes here at once)
  if (S > 1)
    cluster_sync_all();  // every CTA's sums are complete
  else
    __syncthreads();
  // this CTA's share of the outputs, two neighbouring rows a thread
  const int pairs_of = a.T * (kUnitRows / 2);
  const int i0 = rank * pairs_of / S, i1 = (rank + 1) * pairs_of / S;
  const uint32_t base = smem_u32(sums);
  float2* mine = reinterpret_cast<float2*>(a.partial) + (size_t)(tile * a.parts) * pairs_of;
  auto store = [&](int i, float2 v) {
    const int t = i / (kUnitRows / 2), d = d0 + 2 * (i - t * (kUnitRows / 2));
    if (d >= a.H || bars.abort) return;
    __nv_bfloat16* y = a.y + (size_t)t * a.ldy + d;
    y[0] = __float2bfloat16_rn(v.x);
    y[1] = __float2bfloat16_rn(v.y);
  };
  for (int i = i0 + (int)threadIdx.x; i < i1; i += kMoeThreads) {
    float2 o[8], v = make_float2(0.0f, 0.0f);  // every load is on its way before the first sum
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < S) o[c] = ld_shared_cluster_f2(S > 1 ? mapa_shared(base + i * 8, (uint32_t)c) : base + i * 8);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < S) {
        v.x += o[c].x;
        v.y += o[c].y;
      }
    if (a.parts == 1)
      store(i, v);
    else
      __stcg(mine + (size_t)part * pairs_of + i, v);
  }
  if (a.parts > 1) {
    // The last of the tile's CTAs of this rank adds the parts, in their order.
    __shared__ int last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      int* arrived = a.arrived + tile * 8 + rank;
      last = atomicAdd(arrived, 1) == a.parts - 1;
      if (last) *arrived = 0;
    }
    __syncthreads();
    if (last) {
      __threadfence();
      for (int i = i0 + (int)threadIdx.x; i < i1; i += kMoeThreads) {
        float2 v = make_float2(0.0f, 0.0f);
        for (int q = 0; q < a.parts; ++q) {
          const float2 o = __ldcg(mine + (size_t)q * pairs_of + i);
          v.x += o.x;
          v.y += o.y;
        }
        store(i, v);
      }
    }
  }
  if (S > 1) cluster_sync_all();  // no CTA leaves while a peer reads its sums
  moe_teardown<C>(tmem);
}

constexpr int kMaxParts = 4, kMaxSharedTiles = 64;
// The workspace: error word and arrivals at fixed places (they keep their meaning between calls of other sizes), then
// the choices, h and the partial sums.
constexpr size_t kFixedBytes = 256 + kMaxSharedTiles * 8 * sizeof(int);
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int G, bool kFew>
cudaError_t launch_form(MoeArgs& a, const uint8_t* w13, const uint8_t* w2, const Device* dev, cudaStream_t stream) {
  using U = Up<G>;
  using D = Down<G, kFew>;
  CUtensorMap m13, m2;
  if (!halves_map(&m13, w13, (uint64_t)a.E, (uint64_t)a.I, (uint64_t)a.H, kUpCols) ||
      !byte_map(&m2, w2, (uint64_t)a.E * a.H, (uint64_t)a.I, kUnitRows))
    return cudaErrorInvalidValue;
  static bool up_done[64] = {}, down_done[64] = {};
  const void *up = (const void*)moe_gate_up_kernel<G, kFew>, *down = (const void*)moe_down_kernel<G, kFew>;
  cudaError_t e = opt_in_smem(up, U::kSmemBytes, up_done);
  if (e == cudaSuccess) e = opt_in_smem(down, D::bytes(kFew ? G : kMoeMaxTokens), down_done);
  if (e != cudaSuccess) return e;
  if (!kFew) {
    void* args[] = {&a};
    const int choosers = (a.T + kChooseWarps - 1) / kChooseWarps;
    const int terms = G == kGroup ? (a.T * blocks_of(a.H) + 2 * kChooseWarps - 1) / (2 * kChooseWarps) : 0;
    e = launch_pdl((const void*)moe_choose_kernel, dim3(choosers + terms), dim3(32 * kChooseWarps), 0, 1, stream, args);
    if (e != cudaSuccess) return e;
  }
  // Items if every choice were another expert; with few, clusters share them.
  // Otherwise as many CTAs as reside at once.
  const int pairs = a.T * a.topk, tiles = (a.I + kUpCols - 1) / kUpCols;
  const long long most = (long long)(pairs < a.E + pairs / G ? pairs : a.E + pairs / G) * tiles;
  const int nkb = blocks_of(a.H), resident = dev->sms * (G == kSmallGroup ? 2 : 1);
  a.splits = 1;
  while (a.splits < 8 && 2 * a.splits <= nkb && 2 * a.splits * most <= dev->sms) a.splits *= 2;
  void* up_args[] = {&m13, &a};
  e = launch_pdl(up, dim3((unsigned)((most < resident ? most : resident) * a.splits)), dim3(kMoeThreads),
                 U::kSmemBytes, a.splits, stream, up_args);
  if (e != cudaSuccess) return e;
  if (G == kGroup) {
    void* args[] = {&a};
    e = launch_pdl((const void*)moe_terms_kernel, dim3((pairs * blocks_of(a.I) + 15) / 16), dim3(256), 0, 1, stream,
                   args);
    if (e != cudaSuccess) return e;
  }
  // The widest cluster with which every CTA resides at once, and several to a tile where there are few tiles.  With
  // two CTAs on an SM clusters of at most 4: of 8 (and 16) fewer fit, and one that has to wait costs a second wave
  // (45 us at 64 tokens).
  const int row_tiles = (a.H + kUnitRows - 1) / kUnitRows, down_smem = D::bytes(kFew ? G : kMoeMaxTokens);
  const int room = kFew ? dev->sms : resident;
  static Resident known;
  int fit = 0;
  for (a.splits = kFew ? 8 : 4; a.splits > 1; a.splits /= 2) {
    fit = (G == kSmallGroup ? 2 : 1) * resident_clusters(down, kMoeThreads, down_smem, a.splits, known);
    if (fit > room / a.splits) fit = room / a.splits;
    if (fit >= row_tiles) break;
  }
  if (a.splits == 1) fit = room;
  a.parts = row_tiles <= kMaxSharedTiles ? fit / row_tiles : 1;
  a.parts = a.parts < 1 ? 1 : (a.parts > kMaxParts ? kMaxParts : a.parts);
  void* down_args[] = {&m2, &a};
  return launch_pdl(down, dim3((unsigned)(row_tiles * a.splits * a.parts)), dim3(kMoeThreads), D::bytes(a.T), a.splits,
                    stream, down_args);
}

}  // namespace

size_t moe_workspace(int T, int topk, int H, int I) {
  const size_t pairs = (size_t)T * topk, tiles = (size_t)(H + kUnitRows - 1) / kUnitRows;
  const size_t xb = (size_t)T * blocks_of(H), hb = pairs * blocks_of(I);
  return kFixedBytes + align256(8 * pairs) + align256(pairs * I * sizeof(float)) +
         align256(xb * (kUpTerms * kBlock + sizeof(float))) + align256(hb * (kDownTerms * kBlock + sizeof(float))) +
         (tiles <= kMaxSharedTiles ? kMaxParts * tiles * T * kUnitRows * sizeof(float) : 0);
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
  a.s13 = s13;
  a.s2 = s2;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.ids = ids;
  a.weights = weights;
  a.err = static_cast<int*>(ws);
  uint8_t* at = static_cast<uint8_t*>(ws);
  const size_t pairs = (size_t)T * topk;
  a.arrived = reinterpret_cast<int*>(at + 256);
  a.choice = reinterpret_cast<int*>(at += kFixedBytes);
  a.choice_p = reinterpret_cast<float*>(a.choice + pairs);
  a.h = reinterpret_cast<float*>(at += align256(8 * pairs));
  a.x_terms = at += align256(pairs * I * sizeof(float));
  const size_t xb = (size_t)T * blocks_of(H), hb = pairs * blocks_of(I);
  a.x_scale = reinterpret_cast<float*>(a.x_terms + xb * kUpTerms * kBlock);
  a.h_terms = at += align256(xb * (kUpTerms * kBlock + sizeof(float)));
  a.h_scale = reinterpret_cast<float*>(a.h_terms + hb * kDownTerms * kBlock);
  a.partial = reinterpret_cast<float*>(at += align256(hb * (kDownTerms * kBlock + sizeof(float))));
  a.parts = 1;
  a.ldx = ldx;
  a.ldl = ldl;
  a.ldy = ldy;
  a.T = T;
  a.E = E;
  a.topk = topk;
  a.H = H;
  a.I = I;
  a.renorm = renorm;
  if (T <= kSmallGroup) return launch_form<kSmallGroup, true>(a, w13, w2, dev, stream);
  // Groups of 8 while an expert has 4 tokens on average: two gate-up CTAs reside on an SM, and the few experts with
  // more than 8 tokens are read again from L2.
  if (T * topk <= 4 * E) return launch_form<kSmallGroup, false>(a, w13, w2, dev, stream);
  return launch_form<kGroup, false>(a, w13, w2, dev, stream);
}

}  // namespace fp8
}  // namespace sharq
