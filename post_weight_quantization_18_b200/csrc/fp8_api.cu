// fp8_api.cu — the extern "C" entry points declared in include/fp8.h: argument checks on the
// host, then one kernel launch each.
#include <math.h>

#include <mutex>

#include "fp8.cuh"

namespace {

constexpr int64_t kMaxDim = 1 << 30;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool dtype_ok(int t) { return t == GPTQ_BF16 || t == GPTQ_F16 || t == GPTQ_F32; }
inline size_t dtype_bytes(int t) { return t == GPTQ_F32 ? 4 : 2; }
inline int64_t groups(int64_t k) { return (k + 127) / 128; }
inline bool size_ok(int64_t v) { return v >= 1 && v <= kMaxDim; }

// One operand of a product: e4m3 [rows, ld] with its scales.
inline bool pitch_ok(int64_t ld, int64_t lds, int64_t k) { return ld >= k && lds >= groups(k); }
inline bool operand_ok(const uint8_t* q, const float* s) {
  return q != nullptr && s != nullptr && aligned(s, 4);
}

int gemm_launch(const gptq_host::Fp8Gemm& a, cudaStream_t stream) {
  const int rc = !gptq_host::fp8_tma_takes(a) ? gptq_host::fp8_gemm_simt(a, stream)
                 : gptq_host::fp8_skinny_takes(a)  ? gptq_host::fp8_skinny(a, stream)
                 : gptq_host::fp8_wide_cost(a) < gptq_host::fp8_thin_cost(a)
                     ? gptq_host::fp8_gemm_wide(a, stream)
                     : gptq_host::fp8_thin(a, stream);
  return rc ? GPTQ_ERR_CUDA : GPTQ_OK;
}

}  // namespace

namespace {

// Never launched: a kernel for the occupancy calculator, which counts one CTA an SM for kernels that
// allocate tensor memory, however little (two of the streaming kernel's run together).
__global__ void __launch_bounds__(384) occupancy_kernel() {}

}  // namespace

namespace gptq_host {

int resident_clusters(int threads, int smem, int size) {
  struct Entry { int threads, smem, dev, size, count; };
  static Entry known[512];  // five kernels of few rows and one more, sizes 2 to 8, a device
  static int n_known = 0;
  static std::mutex mu;
  int dev = 0;
  if (size < 2 || cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_known; ++i)
    if (known[i].threads == threads && known[i].smem == smem && known[i].dev == dev &&
        known[i].size == size)
      return known[i].count;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int count = 0;
  if (ensure_smem_attr(reinterpret_cast<const void*>(occupancy_kernel), smem) != 0 ||
      cudaOccupancyMaxActiveClusters(&count, occupancy_kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    count = 0;
  }
  if (n_known < 512) known[n_known++] = Entry{threads, smem, dev, size, count};
  return count;
}

}  // namespace gptq_host

extern "C" {

int fp8_quantize(const void* X, int x_dtype, int64_t ldx, int64_t m, int64_t k, int block_rows,
                 uint8_t* Q, int64_t ldq, float* scales, int64_t lds, gptq_stream_t stream) {
  if (m < 0 || m > kMaxDim || !size_ok(k) || ldx < k || ldq < k || lds < groups(k))
    return GPTQ_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return GPTQ_ERR_INVALID_ARG;
  if (!dtype_ok(x_dtype)) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  if (X == nullptr || Q == nullptr || scales == nullptr) return GPTQ_ERR_INVALID_ARG;
  if (!aligned(X, dtype_bytes(x_dtype)) || !aligned(scales, 4)) return GPTQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = block_rows == 1
                     ? gptq_host::fp8_quantize_rows(X, x_dtype, ldx, (int)m, (int)k, Q, ldq,
                                                    scales, lds, s)
                     : gptq_host::fp8_quantize_blocks(X, x_dtype, ldx, (int)m, (int)k, Q, ldq,
                                                      scales, lds, s);
  return rc ? GPTQ_ERR_CUDA : GPTQ_OK;
}

int fp8_add_rmsnorm(const void* X, int64_t ldx, const void* R, int64_t ldr, int dtype,
                    const void* gamma, int gamma_dtype, float eps, int64_t m, int64_t k, void* H,
                    int64_t ldh, uint8_t* Q, int64_t ldq, float* scales, int64_t lds,
                    gptq_stream_t stream) {
  if (m < 0 || m > kMaxDim || !size_ok(k) || ldx < k || ldq < k || lds < groups(k))
    return GPTQ_ERR_INVALID_ARG;
  if ((R != nullptr && ldr < k) || (H != nullptr && ldh < k)) return GPTQ_ERR_INVALID_ARG;
  if (!isfinite(eps) || !(eps >= 0.f)) return GPTQ_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (gamma_dtype != dtype && gamma_dtype != GPTQ_F32))
    return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  if (X == nullptr || gamma == nullptr || Q == nullptr || scales == nullptr)
    return GPTQ_ERR_INVALID_ARG;
  const size_t b = dtype_bytes(dtype);
  if (!aligned(X, b) || (R != nullptr && !aligned(R, b)) || (H != nullptr && !aligned(H, b)) ||
      !aligned(gamma, dtype_bytes(gamma_dtype)) || !aligned(scales, 4))
    return GPTQ_ERR_INVALID_ARG;
  if ((H == X && H != nullptr && ldh != ldx) || (H == R && H != nullptr && ldh != ldr))
    return GPTQ_ERR_INVALID_ARG;
  return gptq_host::fp8_add_rmsnorm(X, ldx, R, ldr, dtype, gamma, gamma_dtype, eps, (int)m, (int)k,
                                    H, ldh, Q, ldq, scales, lds,
                                    reinterpret_cast<cudaStream_t>(stream))
             ? GPTQ_ERR_CUDA
             : GPTQ_OK;
}

int fp8_gemm(const uint8_t* X, int64_t ldx, const float* sx, int64_t ldsx, const uint8_t* W,
             int64_t ldw, const float* sw, int64_t ldsw, int64_t m, int64_t n, int64_t k, void* Y,
             int y_dtype, int64_t ldy, int32_t* dev_status, gptq_stream_t stream) {
  if (m < 0 || m > kMaxDim || !size_ok(n) || !size_ok(k)) return GPTQ_ERR_INVALID_ARG;
  if (!pitch_ok(ldx, ldsx, k) || !pitch_ok(ldw, ldsw, k) || ldy < n) return GPTQ_ERR_INVALID_ARG;
  if (!dtype_ok(y_dtype)) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  if (!operand_ok(X, sx) || !operand_ok(W, sw) || Y == nullptr ||
      !aligned(Y, dtype_bytes(y_dtype)) || !aligned(dev_status, 4))
    return GPTQ_ERR_INVALID_ARG;
  gptq_host::Fp8Gemm a{};
  a.x = X; a.ldx = ldx; a.sx = sx; a.ldsx = ldsx;
  a.w[0] = W; a.ldw[0] = ldw; a.sw[0] = sw; a.ldsw[0] = ldsw;
  a.m = (int)m; a.n = (int)n; a.k = (int)k;
  a.y = Y; a.y_dtype = y_dtype; a.ldy = ldy;
  a.status = dev_status;
  return gemm_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int fp8_gated_gemm(const uint8_t* X, int64_t ldx, const float* sx, int64_t ldsx,
                   const uint8_t* Wg, int64_t ldwg, const float* sg, int64_t ldsg,
                   const uint8_t* Wu, int64_t ldwu, const float* su, int64_t ldsu, int64_t m,
                   int64_t n, int64_t k, uint8_t* Q, int64_t ldq, float* scales, int64_t lds,
                   int32_t* dev_status, gptq_stream_t stream) {
  if (m < 0 || m > kMaxDim || !size_ok(n) || !size_ok(k)) return GPTQ_ERR_INVALID_ARG;
  if (!pitch_ok(ldx, ldsx, k) || !pitch_ok(ldwg, ldsg, k) || !pitch_ok(ldwu, ldsu, k) ||
      !pitch_ok(ldq, lds, n))
    return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!operand_ok(X, sx) || !operand_ok(Wg, sg) || !operand_ok(Wu, su) || !operand_ok(Q, scales) ||
      !aligned(dev_status, 4))
    return GPTQ_ERR_INVALID_ARG;
  gptq_host::Fp8Gemm a{};
  a.x = X; a.ldx = ldx; a.sx = sx; a.ldsx = ldsx;
  a.w[0] = Wg; a.ldw[0] = ldwg; a.sw[0] = sg; a.ldsw[0] = ldsg;
  a.w[1] = Wu; a.ldw[1] = ldwu; a.sw[1] = su; a.ldsw[1] = ldsu;
  a.m = (int)m; a.n = (int)n; a.k = (int)k;
  a.y = Q; a.ldy = ldq; a.sy = scales; a.ldsy = lds;
  a.status = dev_status;
  return gemm_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
