// fp8_prep.cu - activations and weights to E4M3 with float32 block scales.
//
// Per row and 128 columns:  s = max|v| / 448,  code = e4m3(v * f32(1/s)),
// where v is the row's RMS norm, its SwiGLU product or the row itself.
// Everything is bound by HBM: each input is read once into registers, the
// statistics are taken there and codes, scales and the new residual stream
// are written once.
#include "fp8.cuh"

namespace sharq {
namespace fp8 {

namespace {

enum { kPlain = 0, kResidual = 1, kSwiglu = 2 };

struct PrepArgs {
  const __nv_bfloat16* x;    // plain / residual: the input; SwiGLU: the gate
  const __nv_bfloat16* b;    // residual: the stream; SwiGLU: up
  __nv_bfloat16* h;          // residual: the new stream, or nullptr
  const __nv_bfloat16* gamma;
  uint8_t* codes;
  float* scales;
  long long ldx, ldb, ldh;
  int T, K, lds;
  float eps;
};

// 8 consecutive columns as they lie in memory
template <int kKind>
struct Raw {
  uint4 x, w;
  __device__ __forceinline__ void load(const PrepArgs& a, int t, int c) {
    x = *reinterpret_cast<const uint4*>(a.x + (size_t)t * a.ldx + c);
    if (kKind != kPlain) w = *reinterpret_cast<const uint4*>(a.b + (size_t)t * a.ldb + c);
  }
  __device__ __forceinline__ void clear() { x = w = make_uint4(0u, 0u, 0u, 0u); }
  // the residual form's sum, rounded to bf16; the other forms' x
  __device__ __forceinline__ uint4 stream() const {
    if (kKind != kResidual) return x;
    float v[8], u[8];
    unpack_bf16x8(x, v);
    unpack_bf16x8(w, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += u[i];
    return pack_bf16x8(v);
  }
};
__device__ __forceinline__ void store_stream(const PrepArgs& a, int t, int c, const uint4& h) {
  if (a.h) *reinterpret_cast<uint4*>(a.h + (size_t)t * a.ldh + c) = h;
}
// v of 8 consecutive columns before the norm; the residual form stores the sum
template <int kKind>
__device__ __forceinline__ void values8(const PrepArgs& a, int t, int c, const Raw<kKind>& raw, float (&v)[8]) {
  const uint4 h = raw.stream();
  if (kKind == kResidual) store_stream(a, t, c, h);
  unpack_bf16x8(h, v);
  if (kKind == kSwiglu) {
    float w[8];
    unpack_bf16x8(raw.w, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu_mul(v[i], w[i]);
  }
}
template <int kKind>
__device__ __forceinline__ void load8(const PrepArgs& a, int t, int c, float (&v)[8]) {
  Raw<kKind> raw;
  raw.load(a, t, c);
  values8<kKind>(a, t, c, raw, v);
}

// Scales and codes of R 128-blocks that 16 neighbouring lanes hold, 8 values of
// each a lane: block i is row t[i], this lane's columns c[i] .. c[i] + 7 (c >= K:
// zeros, nothing stored), its values v[i].  The maxima are reduced and
// handed out at once: in each step a lane gives away half of its blocks, so R - 1
// exchanges leave a block to every 16 / R lanes, whose scale and reciprocal are
// then computed once and not by every lane for every block.
template <int R>
__device__ __forceinline__ void quant_blocks(const PrepArgs& a, const int (&t)[R], const int (&c)[R],
                                             const float (&v)[R][8]) {
  static_assert(R == 1 || R == 2 || R == 4, "blocks");
  constexpr int kLanes = 16 / R;  // that share a block at the end
  const int l16 = threadIdx.x & 15;
  float m[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[i] = fmaxf(m[i], fabsf(v[i][e]));
  }
  int n = R;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = (l16 & o) ? m[i] : m[i + n], keep = (l16 & o) ? m[i + n] : m[i];
        m[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    } else {
      m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    }
  }
  const float s = block_scale_e4m3(m[0]);  // of block l16 / kLanes
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float k = R == 1 ? inv : __shfl_sync(0xffffffffu, inv, (threadIdx.x & 16) | (i * kLanes));
    if (c[i] < a.K) {
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = v[i][e] * k;
      *reinterpret_cast<uint2*>(a.codes + (size_t)t[i] * a.K + c[i]) =
          make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
    }
    const int b0 = c[i] - l16 * 8;  // the block's first column
    if (l16 == i * kLanes && b0 < a.K) a.scales[(size_t)(b0 / kBlock) * a.lds + t[i]] = s;
  }
}

// Without a norm every 128-block stands alone: half a warp per block, kUnroll
// blocks on their way at once.  A thread steps through (row, block) by the grid's
// step, split into rows and blocks once, so the loop divides nothing.
constexpr int kUnroll = 2, kQuantCtas = 6;
constexpr int kNoColumn = 1 << 30;  // of a block that is not there
template <int kKind>
__global__ void __launch_bounds__(256, kQuantCtas) fp8_quant_kernel(const PrepArgs a) {
  pdl_trigger();
  pdl_wait();
  const int kb = blocks_of(a.K);
  const int step = (int)gridDim.x * 16, dt = step / kb, db = step - dt * kb;
  const int i0 = (int)blockIdx.x * 16 + (int)(threadIdx.x >> 4);
  int t = i0 / kb, b = i0 - t * kb;
  const int lane_col = (threadIdx.x & 15) * 8;
  // the loop is uniform over the warp, so both halves take part in the shuffles
  while (__any_sync(0xffffffffu, t < a.T)) {
    Raw<kKind> raw[kUnroll];
    int rt[kUnroll], rc[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      rt[u] = t < a.T ? t : 0;
      rc[u] = t < a.T ? b * kBlock + lane_col : kNoColumn;
      raw[u].clear();
      if (rc[u] < a.K) raw[u].load(a, rt[u], rc[u]);
      t = t < a.T ? t + dt : t;  // stays past the end without overflowing
      b += db;
      if (b >= kb) {
        b -= kb;
        ++t;
      }
    }
    float v[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
      if (rc[u] < a.K) values8<kKind>(a, rt[u], rc[u], raw[u], v[u]);
    }
    quant_blocks<kUnroll>(a, rt, rc, v);
  }
}

// A row whose sum of squares float32 does not hold (an overflow, or squares
// below its smallest normal value) takes its 1/rms in float64.
__device__ __forceinline__ bool square_sum_fits(float ss) { return ss < 1e37f && ss > 1e-30f; }

template <bool kWarpRow>
__device__ __noinline__ double inv_rms_wide(double s2, const PrepArgs& a) {
  __shared__ double part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
  if (!kWarpRow) {
    if (lane == 0) part[warp] = s2;
    __syncthreads();
    s2 = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s2 += part[w];
  }
  return 1.0 / sqrt(s2 / (double)a.K + (double)a.eps);
}

// threads of the form for rows that fill more than half of an SM's threads at 4 vectors each
constexpr int kWideThreads = 640;

// With a norm, one CTA (or one warp) holds a row: R vectors of 8 columns per
// thread, as bf16.  kWarpRow: a warp per row, no barrier.  The products are
// taken from left to right, (x / rms) gamma: x gamma may leave float32 where
// neither x / rms nor the result does.
template <int kKind, int R, bool kWarpRow, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) fp8_norm_kernel(const PrepArgs a) {
  __shared__ float part[32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nthr = kWarpRow ? 32 : (int)blockDim.x;
  const int me = kWarpRow ? lane : (int)threadIdx.x;
  const int t = kWarpRow ? (int)(blockIdx.x * (blockDim.x >> 5)) + warp : (int)blockIdx.x;
  if (kWarpRow && t >= a.T) return;
  Raw<kKind> raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * nthr + me) * 8;
    raw[r].clear();
    if (c < a.K) raw[r].load(a, t, c);
  }
  uint4 h[R];
  float ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * nthr + me) * 8;
    h[r] = raw[r].stream();
    if (kKind == kResidual && c < a.K) store_stream(a, t, c, h[r]);
    float v[8];
    unpack_bf16x8(h[r], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (!kWarpRow) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = lane < (nthr >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float inv = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.K), a.eps));
  const bool fits = square_sum_fits(ss);  // the same for every thread of the row
  double inv2 = 0.0;
  if (!fits) {
    double s2 = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[8];
      unpack_bf16x8(h[r], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s2 += (double)v[i] * (double)v[i];
    }
    inv2 = inv_rms_wide<kWarpRow>(s2, a);
  }
  constexpr int G = R < 4 ? R : (kThreads == kWideThreads ? 2 : 4);
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += G) {
    int rt[G], rc[G];
    float v[G][8];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      rt[i] = t;
      rc[i] = ((r0 + i) * nthr + me) * 8;
      unpack_bf16x8(h[r0 + i], v[i]);
      if (rc[i] < a.K) {
        float g[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(a.gamma + rc[i]), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = (fits ? v[i][e] * inv : (float)((double)v[i][e] * inv2)) * g[e];
      }
    }
    quant_blocks<G>(a, rt, rc, v);
  }
}

// Rows longer than the registers of one CTA hold: the row is read twice.  The
// second pass reads the stored sum where there is one (the first pass may have
// overwritten the stream it was formed from).
template <int kKind>
__device__ __forceinline__ void reload8(const PrepArgs& a, int t, int c, float (&v)[8]) {
  if (kKind == kResidual && a.h)
    unpack_bf16x8(*reinterpret_cast<const uint4*>(a.h + (size_t)t * a.ldh + c), v);  // this thread's own store
  else
    load8<kKind>(a, t, c, v);
}
template <int kKind>
__global__ void __launch_bounds__(1024) fp8_norm_long_kernel(const PrepArgs a) {
  __shared__ float part[32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x;
  float ss = 0.0f;
  for (int c = threadIdx.x * 8; c < a.K; c += 8192) {
    float v[8];
    load8<kKind>(a, t, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = part[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  double inv = (double)__frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.K), a.eps));
  const bool fits = square_sum_fits(ss);
  if (!fits) {
    double s2 = 0.0;
    for (int c = threadIdx.x * 8; c < a.K; c += 8192) {
      float v[8];
      reload8<kKind>(a, t, c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s2 += (double)v[i] * (double)v[i];
    }
    inv = inv_rms_wide<false>(s2, a);
  }
  for (int c0 = 0; c0 < a.K; c0 += 8192) {
    const int c = c0 + threadIdx.x * 8;
    float v[8] = {};
    if (c < a.K) {
      reload8<kKind>(a, t, c, v);
      float g[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(a.gamma + c), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (fits ? v[i] * (float)inv : (float)((double)v[i] * inv)) * g[i];
    }
    quant_blocks<1>(a, {t}, {c}, reinterpret_cast<const float(&)[1][8]>(v));
  }
}

template <int kKind, int R, bool kWarpRow, int kThreads, int kCtas>
cudaError_t launch_norm(PrepArgs& a, int grid, int block, cudaStream_t stream) {
  void* args[] = {&a};
  return launch_pdl((const void*)fp8_norm_kernel<kKind, R, kWarpRow, kThreads, kCtas>, dim3(grid), dim3(block), 0, 1,
                    stream, args);
}

template <int kKind>
cudaError_t launch_quant(PrepArgs& a, const Device* d, cudaStream_t stream) {
  void* args[] = {&a};
  // 16 blocks a CTA and step; kQuantCtas CTAs reside on an SM
  const long long want = ((long long)a.T * blocks_of(a.K) + 15) / 16, most = (long long)d->sms * kQuantCtas;
  return launch_pdl((const void*)fp8_quant_kernel<kKind>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, 1,
                    stream, args);
}

template <int kKind>
cudaError_t launch_rows(PrepArgs& a, const Device* d, cudaStream_t stream) {
  if (!a.gamma) return launch_quant<kKind>(a, d, stream);
  void* args[] = {&a};
  const int vecs = (a.K + 7) / 8;
  // Short rows: a warp each, four to a CTA.
  if (vecs <= 128) {
    const int grid = (a.T + 3) / 4;
    if (vecs <= 32) return launch_norm<kKind, 1, true, 128, 8>(a, grid, 128, stream);
    if (vecs <= 64) return launch_norm<kKind, 2, true, 128, 8>(a, grid, 128, stream);
    return launch_norm<kKind, 4, true, 128, 8>(a, grid, 128, stream);
  }
  // A CTA per row: a vector per thread while the rows do not fill the GPU, else four, so that several rows are on
  // their way on an SM.  Measured at 8192 x 3584, residual: 43, 39, 38 and 50 us with 1, 2, 4 and 8 vectors, 55 with a
  // warp per row.
  auto block = [&](int r) { return ((vecs + r - 1) / r + 31) / 32 * 32; };
  if (vecs <= 1024 && a.T <= d->sms) return launch_norm<kKind, 1, false, 1024, 1>(a, a.T, block(1), stream);
  if (vecs <= 1024) return launch_norm<kKind, 4, false, 256, 4>(a, a.T, block(4), stream);
  if (vecs <= 4 * kWideThreads) return launch_norm<kKind, 4, false, kWideThreads, 2>(a, a.T, block(4), stream);
  if (vecs <= 4096) return launch_norm<kKind, 4, false, 1024, 1>(a, a.T, block(4), stream);
  return launch_pdl((const void*)fp8_norm_long_kernel<kKind>, dim3(a.T), dim3(1024), 0, 1, stream, args);
}

// --------------------------------------------------------------- weights ---

// One 128 x 128 block of W [K][D] per CTA: amax, then codes transposed to
// [D][K] through shared memory.  Thread (o, kg) holds rows 8 kg .. 8 kg + 7 and
// 8 columns of each, as 8 / kW loads of kW neighbouring columns (what D and the
// base allow to be aligned): column 16 kW p + kW o + i.  Shared memory holds row
// d as 16 chunks of 8 k-bytes, chunk kg at kg ^ (d / kW % 16), so that neither
// side meets bank conflicts.
template <int kW>
struct PackVec;
template <>
struct PackVec<8> {
  using type = uint4;
};
template <>
struct PackVec<4> {
  using type = uint2;
};
template <>
struct PackVec<2> {
  using type = uint32_t;
};
template <>
struct PackVec<1> {
  using type = uint16_t;
};
template <int kW>
__global__ void __launch_bounds__(256) fp8_pack_kernel(const __nv_bfloat16* W, int K, int D, uint8_t* codes,
                                                       float* scales) {
  using Vec = typename PackVec<kW>::type;
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ float part[8];
  pdl_trigger();
  pdl_wait();
  const int kb = blockIdx.x, db = blockIdx.y;
  const size_t e = blockIdx.z;
  const int o = threadIdx.x & 15, kg = threadIdx.x >> 4;
  const int d0 = db * 128, k0 = kb * 128 + kg * 8;
  const __nv_bfloat16* src = W + (e * K + k0) * (size_t)D + d0;
  union {
    Vec v[8 / kW];
    uint16_t b[8];
  } raw[8];  // [row]: bf16 of the thread's 8 columns
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int p = 0; p < 8 / kW; ++p) {
      const int c = (16 * p + o) * kW;
      raw[j].v[p] = Vec{};
      if (k0 + j < K && d0 + c < D) raw[j].v[p] = *reinterpret_cast<const Vec*>(src + (size_t)j * D + c);
    }
  auto value = [&](int j, int i) { return __uint_as_float((uint32_t)raw[j].b[i] << 16); };
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(value(j, i)));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  m = part[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = fmaxf(m, part[w]);
  const float s = block_scale_e4m3(m);
  const float inv = __frcp_rn(s);
  if (threadIdx.x == 0) scales[(e * gridDim.y + db) * gridDim.x + kb] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = (16 * (i / kW) + o) * kW + i % kW;
    uint2 q;
    q.x = e4m3x4(value(0, i) * inv, value(1, i) * inv, value(2, i) * inv, value(3, i) * inv);
    q.y = e4m3x4(value(4, i) * inv, value(5, i) * inv, value(6, i) * inv, value(7, i) * inv);
    *reinterpret_cast<uint2*>(tile + d * 128 + ((kg ^ o) << 3)) = q;
  }
  __syncthreads();
  const int q = threadIdx.x & 7;  // 16-byte chunk of the output row
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = it * 32 + (threadIdx.x >> 3);
    const int ro = (r / kW) & 15;
    uint4 w = *reinterpret_cast<const uint4*>(tile + r * 128 + (((2 * q) ^ (ro & ~1)) << 3));
    if (ro & 1) w = make_uint4(w.z, w.w, w.x, w.y);
    const int d = d0 + r, k = kb * 128 + q * 16;
    if (d < D && k < K) *reinterpret_cast<uint4*>(codes + (e * D + d) * (size_t)K + k) = w;
  }
}

}  // namespace

cudaError_t launch_prep(int kind, const void* x, long long ldx, const void* b, long long ldb, void* h, long long ldh,
                        const void* gamma, float eps, int T, int K, uint8_t* codes, float* scales, int lds,
                        cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  PrepArgs a;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.b = static_cast<const __nv_bfloat16*>(b);
  a.h = static_cast<__nv_bfloat16*>(h);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.codes = codes;
  a.scales = scales;
  a.ldx = ldx;
  a.ldb = ldb;
  a.ldh = ldh;
  a.T = T;
  a.K = K;
  a.lds = lds;
  a.eps = eps;
  const Device* d = device();
  if (!d) return cudaErrorInvalidDevice;
  if (kind == kSwiglu) return launch_quant<kSwiglu>(a, d, stream);  // has no norm
  if (kind == kResidual) return launch_rows<kResidual>(a, d, stream);
  return launch_rows<kPlain>(a, d, stream);
}

cudaError_t launch_pack(const void* W, int K, int D, int E, uint8_t* codes, float* scales, cudaStream_t stream) {
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(W);
  void* args[] = {&w, &K, &D, &codes, &scales};
  // the widest load that every row's start allows
  const uintptr_t at = reinterpret_cast<uintptr_t>(W) | (uintptr_t)D * 2;
  const void* k = at % 16 == 0  ? (const void*)fp8_pack_kernel<8>
                  : at % 8 == 0 ? (const void*)fp8_pack_kernel<4>
                  : at % 4 == 0 ? (const void*)fp8_pack_kernel<2>
                                : (const void*)fp8_pack_kernel<1>;
  return launch_pdl(k, dim3(blocks_of(K), blocks_of(D), E), dim3(256), 0, 1, stream, args);
}

}  // namespace fp8
}  // namespace sharq
