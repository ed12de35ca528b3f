// fp8_api.cu - the sharq_fp8_* entry points of include/sharq.h: size queries,
// views, argument checks and launches of fp8_prep.cu, fp8_linear.cu and
// fp8_moe.cu.  Nothing here allocates device memory.
#include "../../include/sharq.h"
#include "fp8.cuh"

namespace sharq {
namespace fp8 {

cudaError_t launch_prep(int kind, const void* x, long long ldx, const void* b, long long ldb, void* h, long long ldh,
                        const void* gamma, float eps, int T, int K, uint8_t* codes, float* scales, int lds,
                        cudaStream_t stream);
cudaError_t launch_pack(const void* W, int K, int D, int E, uint8_t* codes, float* scales, cudaStream_t stream);
cudaError_t launch_linear(const uint8_t* x, const float* xs, int lds, int T, int K, const uint8_t* w, const float* ws,
                          int D, void* y, long long ldy, int out_f32, int* err, cudaStream_t stream);
size_t moe_workspace(int T, int topk, int H, int I);
cudaError_t launch_moe(const void* x, long long ldx, const float* logits, long long ldl, int T, int E, int topk,
                       int renorm, int H, int I, const uint8_t* w13, const float* s13, const uint8_t* w2,
                       const float* s2, void* y, long long ldy, int* ids, float* weights, void* ws,
                       cudaStream_t stream);

namespace {
constexpr int kMaxDevices = 64;
}

// Values that do not change while the process lives; several threads may fill
// an entry at once and write the same.
const Device* device() {
  static Device table[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  Device& d = table[dev];
  if (d.sms == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return nullptr;
    d.sms = n;
  }
  return &d;
}

cudaError_t opt_in_smem(const void* kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

int resident_clusters(const void* kernel, int threads, int smem, int cluster, Resident& known) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices || cluster < 1 || cluster > 8) return 0;
  int& n = known.n[dev][cluster];
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int got = 0;
    if (cudaOccupancyMaxActiveClusters(&got, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    n = got;
  }
  return n;
}

cudaError_t launch_pdl(const void* kernel, dim3 grid, dim3 block, int smem, int cluster, cudaStream_t stream,
                       void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

namespace {
// tensor map with 128-byte swizzle; dims, strides (of all but the first axis) and box innermost first
bool tensor_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode encode = nullptr;  // a function's address: the same for every thread that looks it up
  if (!encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) !=
            cudaSuccess ||
        res != cudaDriverEntryPointSuccess || !f)
      return false;
    encode = reinterpret_cast<Encode>(f);
  }
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return encode(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, elem,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool byte_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
  const cuuint32_t box[2] = {128, box_rows};
  return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 2, dims, strides, box);
}

bool rows_map(CUtensorMap* map, void* base, uint64_t rows, uint64_t cols, uint64_t ld, int bytes, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * bytes};
  const cuuint32_t box[2] = {128u / (uint32_t)bytes, box_rows};
  return tensor_map(map, bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 2, dims,
                    strides, box);
}

bool halves_map(CUtensorMap* map, const void* base, uint64_t E, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const cuuint64_t dims[5] = {cols, 16, 2, rows / 16, E};
  const cuuint64_t strides[4] = {cols, rows * cols, 16 * cols, 2 * rows * cols};
  const cuuint32_t box[5] = {128, 16, 2, box_rows / 16, 1};
  return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 5, dims, strides, box);
}

}  // namespace fp8
}  // namespace sharq

namespace {

using sharq::fp8::blocks_of;

constexpr int kMaxT = 1 << 22;
constexpr int kMaxK = 1 << 17;
constexpr int kMaxD = 1 << 18;
constexpr int kMaxE = 4096;
constexpr size_t kAlign = 256;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ok_t(int T) { return T >= 0 && T <= kMaxT; }
bool ok_k(int K) { return K > 0 && K <= kMaxK && K % 16 == 0; }
bool ok_d(int D) { return D > 0 && D <= kMaxD; }
bool ok_e(int E) { return E > 0 && E <= kMaxE; }

// rows of `bytes`-wide elements that 16-byte loads read: null only when there are none
bool ok_rows(const void* p, int64_t ld, int cols, int rows) {
  return rows == 0 || (p && aligned(p, 16) && ld >= cols && ld % 8 == 0);
}
// [p, p + rows) x [0, cols) of two strided bf16 matrices share no byte
bool disjoint(const void* p, int64_t ldp, const void* q, int64_t ldq, int rows, int cols) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  const uintptr_t ea = a + 2 * ((uintptr_t)(rows - 1) * ldp + cols), eb = b + 2 * ((uintptr_t)(rows - 1) * ldq + cols);
  if (ea <= b || eb <= a) return true;
  if (ldp != ldq) return false;  // spans that interleave in different strides are refused
  // equal strides: the columns of one must lie beside the other's in every row
  const uintptr_t w = 2 * (uintptr_t)ldp, off = a >= b ? (a - b) % w : (w - (b - a) % w) % w;
  return off >= 2 * (uintptr_t)cols && off + 2 * (uintptr_t)cols <= w;
}

int arch_ok() {
  static int cached[64] = {};  // 0 unknown, 1 sm_100, -1 another
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SHARQ_ERR_CUDA;
  if (cached[dev] == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return SHARQ_ERR_CUDA;
    cached[dev] = major == 10 && minor == 0 ? 1 : -1;
  }
  return cached[dev] > 0 ? SHARQ_OK : SHARQ_ERR_ARCH;
}

int act_ok(const sharq_fp8_act* a) {
  if (!a) return SHARQ_ERR_INVALID_ARG;
  if (!ok_t(a->T) || !ok_k(a->K)) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  if (a->lds < a->T || a->lds % 4 != 0) return SHARQ_ERR_INVALID_ARG;
  if (a->T > 0 && (!a->codes || !a->scales)) return SHARQ_ERR_INVALID_ARG;
  if (!aligned(a->codes, 16) || !aligned(a->scales, 16)) return SHARQ_ERR_INVALID_ARG;
  return SHARQ_OK;
}

int weight_ok(const sharq_fp8_weight* w) {
  if (!w) return SHARQ_ERR_INVALID_ARG;
  if (!ok_k(w->K) || !ok_d(w->D) || !ok_e(w->E)) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  if (!w->codes || !w->scales || !aligned(w->codes, 16) || !aligned(w->scales, 4)) return SHARQ_ERR_INVALID_ARG;
  return SHARQ_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? SHARQ_OK : SHARQ_ERR_CUDA; }

// kind: 0 plain, 1 residual, 2 SwiGLU (fp8_prep.cu)
int prep(int kind, const void* x, int64_t ldx, const void* b, int64_t ldb, void* h, int64_t ldh, const void* gamma,
         float eps, const sharq_fp8_act* a, sharq_stream_t stream) {
  int st = act_ok(a);
  if (st) return st;
  if (!ok_rows(x, ldx, a->K, a->T)) return SHARQ_ERR_INVALID_ARG;
  if (kind != 0 && !ok_rows(b, ldb, a->K, a->T)) return SHARQ_ERR_INVALID_ARG;
  if (h && !ok_rows(h, ldh, a->K, a->T)) return SHARQ_ERR_INVALID_ARG;
  if (gamma && !aligned(gamma, 16)) return SHARQ_ERR_INVALID_ARG;
  if (gamma && !(eps >= 0.0f)) return SHARQ_ERR_INVALID_ARG;
  if (h && a->T > 0) {
    if (!disjoint(x, ldx, h, ldh, a->T, a->K)) return SHARQ_ERR_INVALID_ARG;
    if (!(h == b && ldh == ldb) && !disjoint(b, ldb, h, ldh, a->T, a->K)) return SHARQ_ERR_INVALID_ARG;
  }
  if ((st = arch_ok())) return st;
  return done(sharq::fp8::launch_prep(kind, x, ldx, b, ldb, h, ldh, gamma, eps, a->T, a->K,
                                      static_cast<uint8_t*>(a->codes), a->scales, a->lds,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t sharq_fp8_weight_bytes(int K, int D, int E) {
  if (!ok_k(K) || !ok_d(D) || !ok_e(E)) return 0;
  return round_up((size_t)E * D * K, kAlign) + round_up((size_t)E * blocks_of(D) * blocks_of(K) * sizeof(float), kAlign);
}

size_t sharq_fp8_act_bytes(int T, int K) {
  if (!ok_t(T) || !ok_k(K)) return 0;
  return round_up((size_t)T * K, kAlign) + round_up((size_t)blocks_of(K) * round_up((size_t)T, 4) * sizeof(float), kAlign) +
         kAlign;
}

int sharq_fp8_weight_view(void* d_buf, int K, int D, int E, sharq_fp8_weight* out) {
  if (!d_buf || !out) return SHARQ_ERR_INVALID_ARG;
  if (!ok_k(K) || !ok_d(D) || !ok_e(E)) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(d_buf, kAlign)) return SHARQ_ERR_INVALID_ARG;
  out->codes = d_buf;
  out->scales = reinterpret_cast<float*>(static_cast<uint8_t*>(d_buf) + round_up((size_t)E * D * K, kAlign));
  out->K = K;
  out->D = D;
  out->E = E;
  return SHARQ_OK;
}

int sharq_fp8_act_view(void* d_buf, int T, int K, sharq_fp8_act* out) {
  if (!d_buf || !out) return SHARQ_ERR_INVALID_ARG;
  if (!ok_t(T) || !ok_k(K)) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(d_buf, kAlign)) return SHARQ_ERR_INVALID_ARG;
  out->codes = d_buf;
  out->scales = reinterpret_cast<float*>(static_cast<uint8_t*>(d_buf) + round_up((size_t)T * K, kAlign));
  out->T = T;
  out->K = K;
  out->lds = (int)round_up((size_t)T, 4);
  return SHARQ_OK;
}

int sharq_fp8_pack_weight(const void* d_W, const sharq_fp8_weight* w, sharq_stream_t stream) {
  int st = weight_ok(w);
  if (st) return st;
  if (!d_W || !aligned(d_W, 2)) return SHARQ_ERR_INVALID_ARG;
  if ((st = arch_ok())) return st;
  return done(sharq::fp8::launch_pack(d_W, w->K, w->D, w->E, static_cast<uint8_t*>(w->codes), w->scales,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int sharq_fp8_prep(const void* d_X, int64_t ldx, const void* d_gamma, float eps, const sharq_fp8_act* a,
                   sharq_stream_t stream) {
  return prep(0, d_X, ldx, nullptr, 0, nullptr, 0, d_gamma, eps, a, stream);
}

int sharq_fp8_prep_residual(const void* d_X, int64_t ldx, const void* d_res, int64_t ldr, void* d_res_out, int64_t ldo,
                            const void* d_gamma, float eps, const sharq_fp8_act* a, sharq_stream_t stream) {
  return prep(1, d_X, ldx, d_res, ldr, d_res_out, ldo, d_gamma, eps, a, stream);
}

int sharq_fp8_prep_silu_mul(const void* d_gate, int64_t ldg, const void* d_up, int64_t ldu, const sharq_fp8_act* a,
                            sharq_stream_t stream) {
  return prep(2, d_gate, ldg, d_up, ldu, nullptr, 0, nullptr, 0.0f, a, stream);
}

size_t sharq_fp8_linear_workspace_bytes(int T, int K, int D) {
  if (!ok_t(T) || !ok_k(K) || !ok_d(D)) return 0;
  return kAlign;
}

int sharq_fp8_linear(const sharq_fp8_act* a, const sharq_fp8_weight* w, void* d_Y, int64_t ldy, int out_dtype,
                     void* d_ws, size_t ws_bytes, sharq_stream_t stream) {
  int st = act_ok(a);
  if (st) return st;
  if ((st = weight_ok(w))) return st;
  if (a->K != w->K) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  if (w->E != 1) return SHARQ_ERR_INVALID_ARG;
  if (out_dtype != SHARQ_OUT_BF16 && out_dtype != SHARQ_OUT_F32) return SHARQ_ERR_INVALID_ARG;
  if (a->T > 0 && (!d_Y || !aligned(d_Y, out_dtype == SHARQ_OUT_F32 ? 4 : 2) || ldy < w->D)) return SHARQ_ERR_INVALID_ARG;
  if (!d_ws || !aligned(d_ws, 16) || ws_bytes < sharq_fp8_linear_workspace_bytes(a->T, a->K, w->D))
    return SHARQ_ERR_WORKSPACE;
  if ((st = arch_ok())) return st;
  return done(sharq::fp8::launch_linear(static_cast<const uint8_t*>(a->codes), a->scales, a->lds, a->T, a->K,
                                        static_cast<const uint8_t*>(w->codes), w->scales, w->D, d_Y, ldy,
                                        out_dtype == SHARQ_OUT_F32, static_cast<int*>(d_ws),
                                        reinterpret_cast<cudaStream_t>(stream)));
}

size_t sharq_fp8_moe_workspace_bytes(int T, int topk, int H, int I, int E) {
  if (T < 0 || T > SHARQ_FP8_MOE_MAX_T || topk < 1 || topk > SHARQ_FP8_MOE_MAX_TOPK || topk > E || E < 1 ||
      E > SHARQ_FP8_MOE_MAX_E || !ok_k(H) || !ok_k(I))
    return 0;
  return sharq::fp8::moe_workspace(T, topk, H, I);
}

int sharq_fp8_moe(const void* d_X, int64_t ldx, const float* d_logits, int64_t ldl, int T, int topk, int renormalize,
                  const sharq_fp8_weight* w13, const sharq_fp8_weight* w2, void* d_Y, int64_t ldy, int32_t* d_topk_ids,
                  float* d_topk_weights, void* d_ws, size_t ws_bytes, sharq_stream_t stream) {
  int st = weight_ok(w13);
  if (st) return st;
  if ((st = weight_ok(w2))) return st;
  const int H = w13->K, I = w2->K, E = w13->E;
  if (w2->E != E || w2->D != H || w13->D != 2 * I) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  const size_t need = sharq_fp8_moe_workspace_bytes(T, topk, H, I, E);
  if (need == 0) return SHARQ_ERR_UNSUPPORTED_SHAPE;
  if (!ok_rows(d_X, ldx, H, T)) return SHARQ_ERR_INVALID_ARG;
  if (T > 0 && (!d_logits || !aligned(d_logits, 4) || ldl < E)) return SHARQ_ERR_INVALID_ARG;
  if (T > 0 && (!d_Y || !aligned(d_Y, 2) || ldy < H)) return SHARQ_ERR_INVALID_ARG;
  if (!aligned(d_topk_ids, 4) || !aligned(d_topk_weights, 4)) return SHARQ_ERR_INVALID_ARG;
  if (!d_ws || !aligned(d_ws, 16) || ws_bytes < need) return SHARQ_ERR_WORKSPACE;
  if ((st = arch_ok())) return st;
  return done(sharq::fp8::launch_moe(d_X, ldx, d_logits, ldl, T, E, topk, renormalize != 0, H, I,
                                     static_cast<const uint8_t*>(w13->codes), w13->scales,
                                     static_cast<const uint8_t*>(w2->codes), w2->scales, d_Y, ldy, d_topk_ids,
                                     d_topk_weights, d_ws,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
