// fp8.cuh — what the 8-bit floating point kernels share: the e4m3 conversions, the scale of a
// block, and loads and stores of 16- and 32-bit elements as fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/fp8.h"
#include "common.cuh"
#include "fp8_scale.cuh"

namespace gptq {

constexpr int kFp8Block = 128;           // columns (and weight rows) that share one scale
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: 1 / s stays finite

// The kernels here are launched so that one may start while the kernel before it in the stream still
// runs (fp8_launch): they set up what is their own, then wait for that kernel and its writes. Every
// thread calls this before it reads or writes memory that a caller owns. That memory may change while the
// kernel is resident, so pointers to it are not __restrict__, and no load takes the read-only path.
GPTQ_DEV void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel in the stream start (it waits as above), once every CTA has a thread that came here. A
// kernel that needs tensor memory has it by then: otherwise the next one could take an SM's and wait.
GPTQ_DEV void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Two fp32 values -> two e4m3 bytes (a in the low byte), round to nearest even, +-448 beyond.
GPTQ_DEV uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
GPTQ_DEV uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two e4m3 bytes (low 16 bits of v) -> fp16 pair; exact.
GPTQ_DEV __half2 e4m3x2_to_half2(uint32_t v) {
  uint32_t r;
  const uint16_t h = (uint16_t)v;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return *reinterpret_cast<__half2*>(&r);
}

// Magnitude as an unsigned number whose order is that of |v|, infinities and NaNs on top: the
// maximum of these finds both the block's largest value and whether anything is not finite.
GPTQ_DEV uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The scale of a block from the largest mag_bits of its values, and the factor 1 / s.
GPTQ_DEV void block_scale(uint32_t amax_bits, float& s, float& inv) {
  if (amax_bits >= 0x7F800000u) {
    s = inv = __uint_as_float(0x7FC00000u);
  } else if (amax_bits == 0u) {
    s = inv = 1.f;
  } else {
    s = fmaxf(div_e4m3_max(__uint_as_float(amax_bits)), kMinScale);
    inv = __frcp_rn(s);
  }
}

template <typename T>
GPTQ_DEV float to_f32(T v);
template <>
GPTQ_DEV float to_f32<float>(float v) { return v; }
template <>
GPTQ_DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
GPTQ_DEV float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
GPTQ_DEV T from_f32(float v);
template <>
GPTQ_DEV float from_f32<float>(float v) { return v; }
template <>
GPTQ_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
GPTQ_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight consecutive elements, as loaded.
template <typename T>
struct Vec8 {
  static constexpr int kWords = (int)sizeof(T) * 2;  // 32-bit words
  uint32_t w[kWords];
  GPTQ_DEV float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint16_t h = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
      return to_f32<T>(*reinterpret_cast<const T*>(&h));
    }
  }
  GPTQ_DEV void set(int i, float v) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(v);
    } else {
      const T t = from_f32<T>(v);
      const uint32_t h = *reinterpret_cast<const uint16_t*>(&t);
      w[i >> 1] = (i & 1) ? (w[i >> 1] | (h << 16)) : h;
    }
  }
};

template <typename T>
GPTQ_DEV Vec8<T> pack8(const float (&f)[8]) {
  Vec8<T> v;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2 && __is_same(T, __nv_bfloat16)) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        v.w[i] = *reinterpret_cast<const uint32_t*>(&p);
      } else {
        const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        v.w[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
  }
  return v;
}

// The larger magnitude, NaN if either is NaN; the sign means nothing.
GPTQ_DEV float max_abs(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest magnitude of the eight, as mag_bits of it. 16-bit types are compared as they are: without
// the sign their bits are ordered like the values, infinities and NaNs on top.
template <typename T>
GPTQ_DEV uint32_t max_mag(const Vec8<T>& v) {
  if constexpr (sizeof(T) == 4) {
    float m = v.get(0);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_abs(m, v.get(i));
    return mag_bits(m);
  } else {
    uint32_t m = v.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, v.w[i] & 0x7FFF7FFFu);
    const uint16_t h = (uint16_t)max(m >> 16, m & 0xFFFFu);
    return __float_as_uint(to_f32<T>(*reinterpret_cast<const T*>(&h)));
  }
}

// Eight fp32 values in one access of 32 bytes: with two of 16 every access of a warp touches all of the
// sectors and takes half of each (norm of 6000 x 8192: 131 us, so 118).
GPTQ_DEV bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }
GPTQ_DEV void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                 "=r"(w[7])
               : "l"(p)
               : "memory");
}
GPTQ_DEV void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
               : "memory");
}

// `valid` (0..8) elements at p, zeros behind them. vec: p is 16-byte aligned.
template <typename T>
GPTQ_DEV Vec8<T> load8(const T* p, int valid, bool vec) {
  Vec8<T> v;
#pragma unroll
  for (int i = 0; i < Vec8<T>::kWords; ++i) v.w[i] = 0u;
  if constexpr (sizeof(T) == 4) {
    if (vec && valid == 8 && aligned32(p)) {
      load32(p, v.w);
      return v;
    }
  }
  if (vec && valid == 8) {
#pragma unroll
    for (int i = 0; i < Vec8<T>::kWords; i += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
      v.w[i] = q.x; v.w[i + 1] = q.y; v.w[i + 2] = q.z; v.w[i + 3] = q.w;
    }
  } else if (sizeof(T) == 2 && valid == 8) {
    // Whole words (norm of 8192 x 4097: 97 us, with 2-byte loads and stores 143), and an element at
    // either end where p is between two.
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
    if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
      uint32_t last = e[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t next = i < 3 ? *reinterpret_cast<const uint32_t*>(e + 1 + 2 * i) : e[7];
        v.w[i] = last | (next << 16);
        last = next >> 16;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) v.set(i, to_f32<T>(p[i]));
  }
  return v;
}
template <typename T>
GPTQ_DEV void store8(T* p, const Vec8<T>& v, int valid, bool vec) {
  if constexpr (sizeof(T) == 4) {
    if (vec && valid == 8 && aligned32(p)) return store32(p, v.w);
  }
  if (vec && valid == 8) {
#pragma unroll
    for (int i = 0; i < Vec8<T>::kWords; i += 4)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) =
          make_uint4(v.w[i], v.w[i + 1], v.w[i + 2], v.w[i + 3]);
  } else if (sizeof(T) == 2 && valid == 8) {
    uint16_t* e = reinterpret_cast<uint16_t*>(p);
    if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = v.w[i];
    } else {
      e[0] = (uint16_t)v.w[0];
#pragma unroll
      for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint32_t*>(e + 1 + 2 * i) = (v.w[i] >> 16) | (v.w[i + 1] << 16);
      e[7] = (uint16_t)(v.w[3] >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = from_f32<T>(v.get(i));
  }
}
// Eight e4m3 bytes; vec: p is 8-byte aligned.
GPTQ_DEV void store_q8(uint8_t* p, uint2 q, int valid, bool vec) {
  if (vec && valid == 8) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> ((i & 3) * 8));
  }
}

// One output value of the products.
GPTQ_DEV void store_out(void* Y, long long at, float v, int dtype) {
  if (dtype == GPTQ_F32)
    reinterpret_cast<float*>(Y)[at] = v;
  else if (dtype == GPTQ_BF16)
    reinterpret_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half*>(Y)[at] = __float2half_rn(v);
}

// The gated activation in fp32, g sigmoid(g) u, the sigmoid as e / (1 + e) with e = exp(g), and g up to 64,
// where it is 1: the divisor stays below 2^93. As g / (1 + exp(-g)) the approximate quotient, which is 0 for
// divisors beyond 2^126, made h zero from g = -87.3 down. Here the sigmoid is an fp32 number throughout,
// subnormal from -87.3 and zero from -104 on: 2^-147 of exp and quotient, beside 11 * 2^-24 of itself (exp
// 2 ulp, of 2^-23 at most: 4; the sum 1, the quotient of 2 ulp 4, two products 2). The minimum and one more
// product cost 0.7 % (gated pair of 2000 x 13824 x 5120: 260 us, so 262; with exp(g / 2) twice, which
// reaches -176, 265; with a branch for g far below zero 278).
GPTQ_DEV float silu_mul(float g, float u) {
  const float e = expf(fminf(g, 64.f));
  return g * __fdividef(e, 1.f + e) * u;
}

}  // namespace gptq

namespace gptq_host {

// Launch in clusters of `cluster` CTAs (1: none), with `smem` bytes of dynamic shared memory, allowed
// to start before the previous kernel of the stream has ended. Back to back the kernels of a decoding
// step are 2 to 3 us apart otherwise: the launch, and the set-up of barriers and tensor memory.
template <typename... P, typename... A>
int fp8_launch(void (*kernel)(P...), long long grid, int threads, int smem, int cluster,
               cudaStream_t stream, const A&... args) {
  if (grid < 1 || grid > 0x7FFFFFFFll) return GPTQ_ERR_CUDA;
  // 48 KB are open to every kernel, its static shared memory included. 64 KB at least are asked for, so that
  // a kernel whose need grows with its rows (the norm: up to that) is asked for once.
  const int most = smem < 64 * 1024 ? 64 * 1024 : smem;
  auto failed = [] {
    (void)cudaGetLastError();  // the library's next call would take this one's error for its own
    return GPTQ_ERR_CUDA;
  };
  if (smem > 47 * 1024 && ensure_smem_attr(reinterpret_cast<const void*>(kernel), most) != 0)
    return failed();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? 0 : failed();
}

// Clusters of `size` CTAs (2 to 8) of so many threads and bytes of shared memory that the current device
// holds at once; worked out once for each.
int resident_clusters(int threads, int smem, int size);

struct Fp8Gemm {  // arguments of one product, or of the gated pair (w1 != nullptr)
  const uint8_t* x;
  long long ldx;
  const float* sx;
  long long ldsx;
  const uint8_t* w[2];
  long long ldw[2];
  const float* sw[2];
  long long ldsw[2];
  int m, n, k;
  void* y;        // Y, or Q of the gated pair
  int y_dtype;    // of Y
  long long ldy;
  float* sy;      // the gated pair's scales
  long long ldsy;
  int32_t* status;
};

// The alignment in bytes (16, 8, 4, 2 or 1) that every row of a matrix has.
inline int row_align(const void* p, long long pitch_bytes) {
  const unsigned long long bits = reinterpret_cast<uintptr_t>(p) | (unsigned long long)pitch_bytes | 16;
  return (int)(bits & (0 - bits));
}

int fp8_quantize_rows(const void* x, int dtype, long long ldx, int m, int k, uint8_t* q,
                      long long ldq, float* s, long long lds, cudaStream_t stream);
int fp8_quantize_blocks(const void* x, int dtype, long long ldx, int m, int k, uint8_t* q,
                        long long ldq, float* s, long long lds, cudaStream_t stream);
int fp8_add_rmsnorm(const void* x, long long ldx, const void* r, long long ldr, int dtype,
                    const void* gamma, int gamma_dtype, float eps, int m, int k, void* h,
                    long long ldh, uint8_t* q, long long ldq, float* s, long long lds,
                    cudaStream_t stream);
int fp8_gemm_simt(const Fp8Gemm& a, cudaStream_t stream);
// Whether TMA can address the operands, as the kernels below want them.
bool fp8_tma_takes(const Fp8Gemm& a);
// The tensor-core kernels: bound by the arithmetic, and for few rows of activations, bound by the
// weight's bytes; with the time each needs for a block of 128 columns of K, in units of 1.7 ns.
int fp8_gemm_wide(const Fp8Gemm& a, cudaStream_t stream);
long long fp8_wide_cost(const Fp8Gemm& a);
int fp8_thin(const Fp8Gemm& a, cudaStream_t stream);
long long fp8_thin_cost(const Fp8Gemm& a);
bool fp8_skinny_takes(const Fp8Gemm& a);  // where it is the fastest
int fp8_skinny(const Fp8Gemm& a, cudaStream_t stream);  // up to 32 rows, gated 64
// A tensor map of whole blocks of 128 columns: boxes of 128 bytes x box_rows x box_blocks.
int make_tmap_blocks(CUtensorMap* map, const uint8_t* base, uint64_t rows, uint64_t ld,
                     uint64_t blocks, uint32_t box_rows, uint32_t box_blocks);

}  // namespace gptq_host
