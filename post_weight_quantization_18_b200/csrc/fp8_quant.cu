// fp8_quant.cu — matrices into the e4m3 format with one scale per block of 128: activations
// (1 x 128), weights (128 x 128), and the root-mean-square norm with the residual's addition
// whose output goes straight into the format.
//
// All three read each input once and write each output once; a block's largest magnitude is
// found in registers before anything is written. They are bound by HBM, and next by the number of
// instructions (issue slots 60 to 75 % busy). Measured (B200, measured copy rate 6.44 TB/s), in a graph of
// calls over inputs larger than L2 and, behind the stroke, called one after the other from Python:
// weights 8192 x 28672 bf16 in 102 / 107 us (6.9 TB/s), rows 4096 x 11008 fp16 in 22.9 / 24.8 us (5.9),
// norm 8192 x 5120 bf16 in 51.3 / 54.4 us (5.7; its registers allow three CTAs of 320 threads an SM).
#include "fp8.cuh"

namespace {

using gptq::Vec8;

constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 4;  // groups per half warp

// Sixteen lanes hold one (row, group of 128), eight elements each: the largest magnitude of the
// group in every one of them.
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// The scales of the half warp's U groups, whose largest magnitudes all its lanes hold: lane u of it
// finds the scale of group u, so that U groups cost one reciprocal, and passes on 1 / s.
template <int U>
__device__ __forceinline__ void group_scales(const uint32_t (&mx)[U], float& s, float (&inv)[U]) {
  static_assert(U == 1 || U == 2 || U == 4, "selected by two bits of the lane");
  const int lane = threadIdx.x & 31;
  uint32_t m = (lane & 1) ? mx[1 % U] : mx[0];
  if (U == 4 && (lane & 2)) m = (lane & 1) ? mx[3 % U] : mx[2 % U];
  float i;
  gptq::block_scale(m, s, i);
#pragma unroll
  for (int u = 0; u < U; ++u) inv[u] = __shfl_sync(0xFFFFFFFFu, i, (lane & 16) + u);
}

__device__ __forceinline__ uint2 quantize8(const float (&f)[8], float inv) {
  return make_uint2(gptq::e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    gptq::e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}
template <typename T>
__device__ __forceinline__ uint2 quantize8(const Vec8<T>& v, float inv) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = v.get(i);
  return quantize8(f, inv);
}

// A half warp takes a group, a warp 2 * kRowsUnroll consecutive ones, all loaded before the first is
// looked at. IN_ROW: of one row, whose last warp may have fewer. Otherwise the groups are dealt out
// through the rows' ends, so that no half warp is idle where rows are short; finding each
// group's row costs 8 % at 4096 x 11008 (28 instead of 26 us) and halves 8192 x 128 (3.6
// instead of 7.4 us), so rows of eight groups and more are not split.
template <typename T, bool IN_ROW>
__global__ void __launch_bounds__(kRowsThreads)
quantize_rows_kernel(const T* X, long long ldx, long long items, int groups, int k,
                     uint8_t* Q, long long ldq, float* S, long long lds,
                     bool vec_x, bool vec_q) {
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, col = (lane & 15) * 8;
  const long long warp = (long long)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  const int half = lane >> 4;
  // IN_ROW: items counts rows, each padded to whole warps
  const int per_row = IN_ROW ? (groups + 2 * kRowsUnroll - 1) / (2 * kRowsUnroll) : groups;
  const long long item = IN_ROW ? warp : warp * (2 * kRowsUnroll) + half;
  if (IN_ROW ? item >= items : item - half >= items) return;  // whole warps
  long long row0;
  int g0;
  if (items <= 0x7FFFFFF0ll) {  // one 32-bit division where the groups' number allows it
    row0 = (int)item / per_row;
    g0 = (int)item % per_row;
  } else {
    row0 = item / per_row;
    g0 = (int)(item % per_row);
  }
  if (IN_ROW) g0 = g0 * (2 * kRowsUnroll) + half;
  // Group u of the half warp is 2 u groups on; a group that does not exist has no valid columns.
  auto place = [&](int u, long long& row, int& g) {
    row = row0;
    g = g0 + 2 * u;
    if (!IN_ROW) {
      while (g >= groups) {
        g -= groups;
        ++row;
      }
      if (item + 2 * u >= items) return 0;
    }
    return max(0, min(8, k - (g * 128 + col)));
  };
  Vec8<T> v[kRowsUnroll];
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    long long row;
    int g;
    const int valid = place(u, row, g);
    v[u] = gptq::load8(X + row * ldx + g * 128 + col, valid, vec_x);
  }
  uint32_t mx[kRowsUnroll];
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) mx[u] = group_max(gptq::max_mag(v[u]));
  float s, inv[kRowsUnroll];
  group_scales(mx, s, inv);
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    long long row;
    int g;
    const int valid = place(u, row, g);
    gptq::store_q8(Q + row * ldq + g * 128 + col, quantize8(v[u], inv[u]), valid, vec_q);
    if ((lane & 15) == u && (IN_ROW ? g < groups : item + 2 * u < items)) S[row * lds + g] = s;
  }
}

// One CTA per block of 128 x 128, held in registers: thread (i, j) of 16 x 16 has columns
// 8 j .. 8 j + 7 of rows i, i + 16, ...
template <typename T>
__global__ void __launch_bounds__(256)
quantize_blocks_kernel(const T* X, long long ldx, int m, int k, int groups,
                       uint8_t* Q, long long ldq, float* S,
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
  for (int r = 0; r < 8; ++r) mx = max(mx, gptq::max_mag(v[r]));
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
    gptq::store_q8(Q + row * ldq + c, quantize8(v[r], inv), row < m ? valid : 0, vec_q);
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// part: one array of 32 per call in flight (a second barrier would protect a single one).
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f);
}

template <typename T>
__device__ __forceinline__ void add8(const Vec8<T>& x, const Vec8<T>& r, bool with_r, float (&h)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = with_r ? x.get(i) + r.get(i) : x.get(i);
}
template <typename T>
__device__ __forceinline__ void load_h(const NormArgs& a, long long row, int c, int valid,
                                       float (&h)[8]) {
  const Vec8<T> x = gptq::load8(reinterpret_cast<const T*>(a.x) + row * a.ldx + c, valid, a.vec);
  Vec8<T> r = x;
  if (a.r != nullptr)
    r = gptq::load8(reinterpret_cast<const T*>(a.r) + row * a.ldr + c, valid, a.vec);
  add8(x, r, a.r != nullptr, h);
}

// V vectors of eight, `step` columns apart: H, and y = (h * rs) * gamma(v) in the format. The factors in
// this order and 1 / s apart, although rs could join it: h rs is at most sqrt(k), while h gamma, and
// rs / s for a block of small values (1 / s is up to 2^126), leave fp32's range though y does not. (The
// third product takes 8192 x 5120 of bf16 from 50.5 to 51.3 us, 8192 x 8704 from 97.2 to 98.8.)
template <typename T, int V, typename F>
__device__ __forceinline__ void finish(const NormArgs& a, long long row, int c0, int step,
                                       float (&h)[V][8], F gamma, float rs) {
  uint32_t mx[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = c0 + v * step, valid = max(0, min(8, a.k - c));
    if (a.h != nullptr)
      gptq::store8(reinterpret_cast<T*>(a.h) + row * a.ldh + c, gptq::pack8<T>(h[v]), valid, a.vec);
    const auto gm = gamma(v);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[v][i] = h[v][i] * rs * gm.get(i);  // h and gamma are zero behind the row's end
      m = gptq::max_abs(m, h[v][i]);
    }
    mx[v] = group_max(gptq::mag_bits(m));
  }
  float s, inv[V];
  group_scales(mx, s, inv);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = c0 + v * step, valid = max(0, min(8, a.k - c));
    gptq::store_q8(a.q + row * a.ldq + c, quantize8(h[v], inv[v]), valid, a.vec_q);
    if ((threadIdx.x & 15) == v && c - 8 * v < a.k) a.s[row * a.lds + c / 128] = s;
  }
}

__device__ __forceinline__ float inv_rms(float sum, const NormArgs& a) {
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)a.k) + a.eps));
}

// Rows in registers, V vectors of eight a thread; a team of threads per row: a warp (TEAM_WARP) or the
// CTA. Persistent for 16-bit rows: every thread keeps its part of gamma, and copies its part of the next row
// of x and r into shared memory of its own (cp.async) while it works on this one, because with plain
// loads a row's latency, the reduction and the stores followed one another and DRAM was idle
// for a third of the time. Rows that 16-byte copies cannot address are loaded when they are due,
// and so are rows of fp32, of whose sectors a thread's two copies would each fetch all (67 us
// at 4096 x 5120, loaded 55).
template <typename T, typename TG, int V, bool TEAM_WARP>
__global__ void __launch_bounds__(512, 2) add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  constexpr bool AHEAD = sizeof(T) == 2;
  // gamma before the row's sum, but not where registers are short: with four vectors they are better
  // spent on a second CTA (8192 x 8704 of bf16: 137 us, so 99)
  constexpr bool EARLY = (AHEAD && V < 4) || V == 1;
  extern __shared__ __align__(16) uint8_t next_row[];  // [x, r][V][threads] of 16 bytes
  __shared__ float part[2][32];
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  const int team = TEAM_WARP ? 32 : blockDim.x;
  const int teams = TEAM_WARP ? blockDim.x / 32 : 1;
  const int c0 = (threadIdx.x % team) * 8, step = team * 8;
  const long long row0 = (long long)blockIdx.x * teams + threadIdx.x / team;
  const long long stride = (long long)gridDim.x * teams;
  const bool ahead = AHEAD && a.vec;
  const uint32_t mine = gptq::smem_u32(next_row) + threadIdx.x * 16;
  auto slot_at = [&](int which, int v) { return mine + (uint32_t)((which * V + v) * blockDim.x) * 16; };
  auto fetch = [&](long long row) {
    if (!ahead || row >= a.m) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which == 1 && a.r == nullptr) continue;
      const T* p = reinterpret_cast<const T*>(which ? a.r : a.x) + row * (which ? a.ldr : a.ldx);
#pragma unroll
      for (int v = 0; v < V; ++v) {  // zeros behind the row's end, which is not read
        const int c = c0 + v * step, n = max(0, min(8, a.k - c));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot_at(which, v)),
                     "l"(p + (n > 0 ? c : 0)), "r"(n * 2)
                     : "memory");
      }
    }
  };
  auto taken = [&](int which, int v) {
    Vec8<T> o;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(o.w[0]), "=r"(o.w[1]), "=r"(o.w[2]), "=r"(o.w[3])
                 : "r"(slot_at(which, v))
                 : "memory");
    return o;
  };
  fetch(row0);
  auto load_gamma = [&](int v) {
    const int c = c0 + v * step;
    return gptq::load8(reinterpret_cast<const TG*>(a.gamma) + c, max(0, min(8, a.k - c)), a.vec_g);
  };
  Vec8<TG> gamma[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (EARLY) gamma[v] = load_gamma(v);
  int flip = 0;
  for (long long row = row0; row < a.m; row += stride) {
    float h[V][8];
    float sum = 0.f;
    if (ahead) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + v * step;
      if (AHEAD && ahead) {
        const Vec8<T> x = taken(0, v);
        add8(x, a.r != nullptr ? taken(1, v) : x, a.r != nullptr, h[v]);
      } else {
        load_h<T>(a, row, c, max(0, min(8, a.k - c)), h[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(h[v][e], h[v][e], sum);
    }
    fetch(row + stride);  // into the place just read
    sum = TEAM_WARP ? warp_sum(sum) : block_sum(sum, part[flip]);
    flip ^= 1;
    finish<T, V>(a, row, c0, step, h, [&](int v) { return EARLY ? gamma[v] : load_gamma(v); },
                 inv_rms(sum, a));
  }
}

// Rows too long for registers: x and r are read a second time (from L2 mostly).
template <typename T, typename TG>
__global__ void __launch_bounds__(1024, 2) add_rmsnorm_wide_kernel(const __grid_constant__ NormArgs a) {
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
  const float rs = inv_rms(block_sum(sum, part), a);
  for (int t = 0; t < steps; ++t) {
    const long long cl = ((long long)t * 1024 + threadIdx.x) * 8;
    const int c = (int)min(cl, (long long)a.k), valid = min(8, a.k - c);
    float h[1][8];
    load_h<T>(a, row, c, valid, h[0]);
    finish<T, 1>(a, row, c, 0, h, [&](int) {
      return gptq::load8(reinterpret_cast<const TG*>(a.gamma) + c, valid, a.vec_g);
    }, rs);
  }
}

inline bool rows_aligned(const void* p, long long ld, int elem, int to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && ld * elem % to == 0;
}

template <typename T>
int launch_rows(const void* x, long long ldx, int m, int k, uint8_t* q, long long ldq, float* s,
                long long lds, cudaStream_t stream) {
  constexpr int kWarp = 2 * kRowsUnroll, kWarps = kRowsThreads / 32;
  const int groups = (k + 127) / 128;
  const bool in_row = groups >= kWarp;
  const long long items = in_row ? (long long)m * ((groups + kWarp - 1) / kWarp)
                                 : (long long)m * groups;
  const int per_cta = in_row ? kWarps : kWarps * kWarp;
  auto run = [&](auto kernel) {
    return gptq_host::fp8_launch(kernel, (items + per_cta - 1) / per_cta, kRowsThreads, 0, 1, stream,
                                 static_cast<const T*>(x), ldx, items, groups, k, q, ldq, s, lds,
                                 rows_aligned(x, ldx, sizeof(T), 16), rows_aligned(q, ldq, 1, 8));
  };
  return in_row ? run(quantize_rows_kernel<T, true>) : run(quantize_rows_kernel<T, false>);
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
  using gptq_host::fp8_launch;
  const int vecs = (a.k + 7) / 8;
  // A warp per row while a row fits in two vectors a lane; then a CTA, of up to 512 threads. As many
  // CTAs as the SMs hold, which is 1024 threads with 64 registers, all rows dealt out to them (8192 x
  // 3584 of bf16 38.8 us, 8192 x 5120 53.2, 8192 x 7168 75; 1536 threads: 42.1, 56.1, 84; 2048: 41.3,
  // 52.8, 79; 640 threads a row instead of 320 took 69 at 8192 x 5120). Rows of fp32, which nothing
  // fetches ahead, get a CTA each (55 us at 4096 x 5120, dealt out 68).
  auto run = [&](auto kernel, int v, bool team_warp) {
    const int threads = team_warp ? 256 : ((vecs + v - 1) / v + 31) / 32 * 32;
    const int teams = team_warp ? threads / 32 : 1;
    const long long ctas = ((long long)a.m + teams - 1) / teams;
    const long long most = (long long)gptq_host::num_sms() * (1024 / threads);
    return fp8_launch(kernel, sizeof(T) == 4 || ctas < most ? ctas : most, threads,
                      sizeof(T) == 2 ? 2 * v * threads * 16 : 0, 1, stream, a);
  };
  if (vecs <= 32) return run(add_rmsnorm_kernel<T, TG, 1, true>, 1, true);
  if (vecs <= 64) return run(add_rmsnorm_kernel<T, TG, 2, true>, 2, true);
  if (vecs <= 256) return run(add_rmsnorm_kernel<T, TG, 1, false>, 1, false);
  if (vecs <= 768) return run(add_rmsnorm_kernel<T, TG, 2, false>, 2, false);
  if (vecs <= 2048) return run(add_rmsnorm_kernel<T, TG, 4, false>, 4, false);
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
