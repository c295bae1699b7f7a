// fp8_quant.cu — matrices into the e4m3 format with one scale per block of 128: activations
// (1 x 128), weights (128 x 128), and the root-mean-square norm with the residual's addition
// whose output goes straight into the format.
//
// All three read each input once and write each output once; a block's largest magnitude is
// found in registers before anything is written.
#include "fp8.cuh"

namespace {

using gptq::Vec8;

constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 2;  // groups per half warp

// Sixteen lanes hold one (row, group of 128), eight elements each: the largest magnitude of the
// group in every one of them.
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

__device__ __forceinline__ uint2 quantize8(const float (&f)[8], float inv) {
  return make_uint2(gptq::e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    gptq::e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// A warp takes 2 * kRowsUnroll consecutive groups of one row.
template <typename T>
__global__ void __launch_bounds__(kRowsThreads)
quantize_rows_kernel(const T* __restrict__ X, long long ldx, long long tiles, int tiles_row, int k,
                     uint8_t* __restrict__ Q, long long ldq, float* __restrict__ S, long long lds,
                     bool vec_x, bool vec_q) {
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  const long long tile = (long long)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 31;
  long long row;
  int t;
  if (tiles <= 0x7FFFFFFFll) {  // one 32-bit division a warp where the tiles' number allows it
    row = (int)tile / tiles_row;
    t = (int)tile % tiles_row;
  } else {
    row = tile / tiles_row;
    t = (int)(tile % tiles_row);
  }
  const T* x = X + row * ldx;
  Vec8<T> v[kRowsUnroll];
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    const long long c = ((long long)t * kRowsUnroll + u) * 256 + lane * 8;
    const int valid = (int)max(0ll, min(8ll, k - c));
    v[u] = gptq::load8(x + c, valid, vec_x);
  }
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    const long long c = ((long long)t * kRowsUnroll + u) * 256 + lane * 8;
    const int valid = (int)max(0ll, min(8ll, k - c));
    float f[8];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = v[u].get(i);
      mx = max(mx, gptq::mag_bits(f[i]));
    }
    float s, inv;
    gptq::block_scale(group_max(mx), s, inv);
    gptq::store_q8(Q + row * ldq + c, quantize8(f, inv), valid, vec_q);
    if ((lane & 15) == 0 && valid > 0) S[row * lds + c / 128] = s;
  }
}

// One CTA per block of 128 x 128, held in registers: thread (i, j) of 16 x 16 has columns
// 8 j .. 8 j + 7 of rows i, i + 16, ...
template <typename T>
__global__ void __launch_bounds__(256)
quantize_blocks_kernel(const T* __restrict__ X, long long ldx, int m, int k, int groups,
                       uint8_t* __restrict__ Q, long long ldq, float* __restrict__ S,
                       long long lds, bool vec_x, bool vec_q) {
  __shared__ uint32_t part[8];
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  const int br = blockIdx.x / groups, g = blockIdx.x % groups;
  const int i0 = threadIdx.x >> 4, c = g * 128 + (threadIdx.x & 15) * 8;
  const int valid = max(0, min(8, k - c));
  Vec8<T> v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const long long row = (long long)br * 128 + i0 + 16 * r;
    v[r] = gptq::load8(X + row * ldx + c, row < m ? valid : 0, vec_x);
  }
  uint32_t mx = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = max(mx, gptq::mag_bits(v[r].get(e)));
  mx = __reduce_max_sync(0xFFFFFFFFu, mx);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = part[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) mx = max(mx, part[w]);
  float s, inv;
  gptq::block_scale(mx, s, inv);
  if (threadIdx.x == 0) S[(long long)br * lds + g] = s;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const long long row = (long long)br * 128 + i0 + 16 * r;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[r].get(e);
    gptq::store_q8(Q + row * ldq + c, quantize8(f, inv), row < m ? valid : 0, vec_q);
  }
}

struct NormArgs {
  const void *x, *r, *gamma;
  void* h;
  uint8_t* q;
  float* s;
  long long ldx, ldr, ldh, ldq, lds;
  int m, k;
  float eps;
  bool vec, vec_g, vec_q;  // 16-byte rows of x, r and h; of gamma; 8-byte rows of q
};

__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void load_h(const NormArgs& a, long long row, int c, int valid,
                                       float (&h)[8]) {
  const Vec8<T> x = gptq::load8(reinterpret_cast<const T*>(a.x) + row * a.ldx + c, valid, a.vec);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = x.get(i);
  if (a.r != nullptr) {
    const Vec8<T> r = gptq::load8(reinterpret_cast<const T*>(a.r) + row * a.ldr + c, valid, a.vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += r.get(i);
  }
}

// One vector of eight: H, and y = h * rs * gamma in the format.
template <typename T, typename TG>
__device__ __forceinline__ void finish8(const NormArgs& a, long long row, int c, int valid,
                                        const float (&h)[8], float rs) {
  if (a.h != nullptr) {
    Vec8<T> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.set(i, h[i]);
    gptq::store8(reinterpret_cast<T*>(a.h) + row * a.ldh + c, o, valid, a.vec);
  }
  const Vec8<TG> gm = gptq::load8(reinterpret_cast<const TG*>(a.gamma) + c, valid, a.vec_g);
  float y[8];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = h[i] * rs * gm.get(i);
    mx = max(mx, i < valid ? gptq::mag_bits(y[i]) : 0u);
  }
  float s, inv;
  gptq::block_scale(group_max(mx), s, inv);
  gptq::store_q8(a.q + row * a.ldq + c, quantize8(y, inv), valid, a.vec_q);
  if ((threadIdx.x & 15) == 0 && valid > 0) a.s[row * a.lds + c / 128] = s;
}

// One CTA per row, the row in registers: V vectors of eight a thread.
template <typename T, typename TG, int V>
__global__ void add_rmsnorm_kernel(NormArgs a) {
  __shared__ float part[32];
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  const long long row = blockIdx.x;
  float h[V][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    load_h<T>(a, row, c, max(0, min(8, a.k - c)), h[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
  }
  sum = block_sum(sum, part);
  const float rs = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)a.k) + a.eps));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    finish8<T, TG>(a, row, c, max(0, min(8, a.k - c)), h[i], rs);
  }
}

// Rows too long for registers: x and r are read a second time (from L2 mostly).
template <typename T, typename TG>
__global__ void __launch_bounds__(1024) add_rmsnorm_wide_kernel(NormArgs a) {
  __shared__ float part[32];
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  const long long row = blockIdx.x;
  const int steps = (a.k + 8191) / 8192;  // whole warps in every step
  float sum = 0.f;
  for (int t = 0; t < steps; ++t) {
    const long long cl = ((long long)t * 1024 + threadIdx.x) * 8;
    const int valid = (int)max(0ll, min(8ll, a.k - cl));
    float h[8];
    load_h<T>(a, row, valid > 0 ? (int)cl : 0, valid, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[e], h[e], sum);
  }
  sum = block_sum(sum, part);
  const float rs = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)a.k) + a.eps));
  for (int t = 0; t < steps; ++t) {
    const long long cl = ((long long)t * 1024 + threadIdx.x) * 8;
    const int valid = (int)max(0ll, min(8ll, a.k - cl));
    const int c = valid > 0 ? (int)cl : 0;
    float h[8];
    load_h<T>(a, row, c, valid, h);
    finish8<T, TG>(a, row, c, valid, h, rs);
  }
}

inline bool rows_aligned(const void* p, long long ld, int elem, int to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && ld * elem % to == 0;
}

template <typename T>
int launch_rows(const void* x, long long ldx, int m, int k, uint8_t* q, long long ldq, float* s,
                long long lds, cudaStream_t stream) {
  const int tiles_row = (k + 256 * kRowsUnroll - 1) / (256 * kRowsUnroll);
  const long long tiles = (long long)m * tiles_row;
  const long long ctas = (tiles + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  return gptq_host::fp8_launch(quantize_rows_kernel<T>, ctas, kRowsThreads, 0, 1, stream,
                               static_cast<const T*>(x), ldx, tiles, tiles_row, k, q, ldq, s, lds,
                               rows_aligned(x, ldx, sizeof(T), 16), rows_aligned(q, ldq, 1, 8));
}

template <typename T>
int launch_blocks(const void* x, long long ldx, int m, int k, uint8_t* q, long long ldq, float* s,
                  long long lds, cudaStream_t stream) {
  const int groups = (k + 127) / 128;
  const long long ctas = (long long)groups * ((m + 127) / 128);
  return gptq_host::fp8_launch(quantize_blocks_kernel<T>, ctas, 256, 0, 1, stream,
                               static_cast<const T*>(x), ldx, m, k, groups, q, ldq, s, lds,
                               rows_aligned(x, ldx, sizeof(T), 16), rows_aligned(q, ldq, 1, 8));
}

template <typename T, typename TG>
int launch_norm(NormArgs a, cudaStream_t stream) {
  a.vec = rows_aligned(a.x, a.ldx, sizeof(T), 16) &&
          (a.r == nullptr || rows_aligned(a.r, a.ldr, sizeof(T), 16)) &&
          (a.h == nullptr || rows_aligned(a.h, a.ldh, sizeof(T), 16));
  a.vec_g = rows_aligned(a.gamma, 0, sizeof(TG), 16);
  a.vec_q = rows_aligned(a.q, a.ldq, 1, 8);
  const int vecs = (a.k + 7) / 8;
  auto threads = [&](int v) { return ((vecs + v - 1) / v + 31) / 32 * 32; };
  using gptq_host::fp8_launch;
  if (vecs <= 512)
    return fp8_launch(add_rmsnorm_kernel<T, TG, 1>, a.m, threads(1), 0, 1, stream, a);
  if (vecs <= 1024)
    return fp8_launch(add_rmsnorm_kernel<T, TG, 2>, a.m, threads(2), 0, 1, stream, a);
  if (vecs <= 2048)
    return fp8_launch(add_rmsnorm_kernel<T, TG, 4>, a.m, threads(4), 0, 1, stream, a);
  return fp8_launch(add_rmsnorm_wide_kernel<T, TG>, a.m, 1024, 0, 1, stream, a);
}

}  // namespace

namespace gptq_host {

int fp8_quantize_rows(const void* x, int dtype, long long ldx, int m, int k, uint8_t* q,
                      long long ldq, float* s, long long lds, cudaStream_t stream) {
  if (dtype == GPTQ_BF16)
    return launch_rows<__nv_bfloat16>(x, ldx, m, k, q, ldq, s, lds, stream);
  if (dtype == GPTQ_F16) return launch_rows<__half>(x, ldx, m, k, q, ldq, s, lds, stream);
  return launch_rows<float>(x, ldx, m, k, q, ldq, s, lds, stream);
}

int fp8_quantize_blocks(const void* x, int dtype, long long ldx, int m, int k, uint8_t* q,
                        long long ldq, float* s, long long lds, cudaStream_t stream) {
  if (dtype == GPTQ_BF16)
    return launch_blocks<__nv_bfloat16>(x, ldx, m, k, q, ldq, s, lds, stream);
  if (dtype == GPTQ_F16) return launch_blocks<__half>(x, ldx, m, k, q, ldq, s, lds, stream);
  return launch_blocks<float>(x, ldx, m, k, q, ldq, s, lds, stream);
}

int fp8_add_rmsnorm(const void* x, long long ldx, const void* r, long long ldr, int dtype,
                    const void* gamma, int gamma_dtype, float eps, int m, int k, void* h,
                    long long ldh, uint8_t* q, long long ldq, float* s, long long lds,
                    cudaStream_t stream) {
  NormArgs a{};
  a.x = x; a.r = r; a.gamma = gamma; a.h = h; a.q = q; a.s = s;
  a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldq = ldq; a.lds = lds;
  a.m = m; a.k = k; a.eps = eps;
  const bool g32 = gamma_dtype == GPTQ_F32;
  if (dtype == GPTQ_BF16)
    return g32 ? launch_norm<__nv_bfloat16, float>(a, stream)
               : launch_norm<__nv_bfloat16, __nv_bfloat16>(a, stream);
  if (dtype == GPTQ_F16)
    return g32 ? launch_norm<__half, float>(a, stream) : launch_norm<__half, __half>(a, stream);
  return launch_norm<float, float>(a, stream);
}

}  // namespace gptq_host
