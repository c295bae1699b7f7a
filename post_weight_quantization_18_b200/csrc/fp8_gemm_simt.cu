// fp8_gemm_simt.cu — the products of the e4m3 format on the CUDA cores, for operands whose base
// or pitch TMA cannot address (not multiples of 16 bytes).
//
// Y = sum_g sx sw (sum over 128 columns): a CTA owns 16 rows x 128 columns of the output (one
// block of the gated pair's output, so its scale is found in the CTA). Per block of 128 columns
// of K, X goes to shared memory as fp32 and W as bytes; a thread sums eight outputs of one row in
// fp32, then scales and adds.
#include "fp8.cuh"

namespace {

constexpr int TM = 16, TN = 128, TK = 128;
constexpr int W_PITCH = 132;  // 33 words: the sixteen rows a half warp reads lie in different banks

struct SimtArgs {
  gptq_host::Fp8Gemm g;
  int tiles_n;
};

template <bool GATED>
__global__ void __launch_bounds__(256) fp8_gemm_simt_kernel(SimtArgs a) {
  constexpr int NW = GATED ? 2 : 1;
  __shared__ float xs[TM][TK + 4];
  __shared__ __align__(16) uint8_t ws[NW][TN * W_PITCH];
  gptq::let_next_kernel_start();
  gptq::wait_for_previous_kernel();
  if (gptq::status_bad(a.g.status)) return;
  const int tm = blockIdx.x / a.tiles_n, tn = blockIdx.x % a.tiles_n;
  const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int row = tm * TM + r;
  float acc[NW][8];
#pragma unroll
  for (int w = 0; w < NW; ++w)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[w][j] = 0.f;
  const int groups = (a.g.k + TK - 1) / TK;
  for (int g = 0; g < groups; ++g) {
    for (int i = threadIdx.x; i < TM * TK; i += 256) {
      const int ri = tm * TM + i / TK, ki = g * TK + i % TK;
      float v = 0.f;
      if (ri < a.g.m && ki < a.g.k)
        v = __low2float(gptq::e4m3x2_to_half2(a.g.x[(long long)ri * a.g.ldx + ki]));
      xs[i / TK][i % TK] = v;
    }
    for (int w = 0; w < NW; ++w)
      for (int i = threadIdx.x; i < TN * TK; i += 256) {
        const int ni = tn * TN + i / TK, ki = g * TK + i % TK;
        ws[w][(i / TK) * W_PITCH + i % TK] =
            ni < a.g.n && ki < a.g.k ? a.g.w[w][(long long)ni * a.g.ldw[w] + ki] : (uint8_t)0;
      }
    __syncthreads();
    const float sx = row < a.g.m ? a.g.sx[(long long)row * a.g.ldsx + g] : 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = sx * a.g.sw[w][(long long)tn * a.g.ldsw[w] + g];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t* wr = reinterpret_cast<const uint32_t*>(ws[w] + (c + 16 * j) * W_PITCH);
        float d = 0.f;
        for (int k4 = 0; k4 < TK / 4; ++k4) {
          const uint32_t q = wr[k4];
          const float2 lo = __half22float2(gptq::e4m3x2_to_half2(q));
          const float2 hi = __half22float2(gptq::e4m3x2_to_half2(q >> 16));
          const float4 x = *reinterpret_cast<const float4*>(&xs[r][4 * k4]);
          d = fmaf(x.x, lo.x, d);
          d = fmaf(x.y, lo.y, d);
          d = fmaf(x.z, hi.x, d);
          d = fmaf(x.w, hi.y, d);
        }
        acc[w][j] = fmaf(f, d, acc[w][j]);
      }
    }
    __syncthreads();
  }
  if constexpr (GATED) {
    float h[8];
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = gptq::silu_mul(acc[0][j], acc[NW - 1][j]);
      if (tn * TN + c + 16 * j < a.g.n) mx = max(mx, gptq::mag_bits(h[j]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    float s, inv;
    gptq::block_scale(mx, s, inv);
    if (row >= a.g.m) return;
    uint8_t* q = reinterpret_cast<uint8_t*>(a.g.y) + (long long)row * a.g.ldy;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = tn * TN + c + 16 * j;
      if (col < a.g.n) q[col] = (uint8_t)gptq::e4m3x2(h[j] * inv, 0.f);
    }
    if (c == 0) a.g.sy[(long long)row * a.g.ldsy + tn] = s;
  } else {
    if (row >= a.g.m) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = tn * TN + c + 16 * j;
      if (col < a.g.n)
        gptq::store_out(a.g.y, (long long)row * a.g.ldy + col, acc[0][j], a.g.y_dtype);
    }
  }
}

}  // namespace

namespace gptq_host {

int fp8_gemm_simt(const Fp8Gemm& g, cudaStream_t stream) {
  SimtArgs a;
  a.g = g;
  a.tiles_n = (g.n + TN - 1) / TN;
  const long long ctas = (long long)((g.m + TM - 1) / TM) * a.tiles_n;
  return g.w[1] != nullptr ? fp8_launch(fp8_gemm_simt_kernel<true>, ctas, 256, 0, 1, stream, a)
                           : fp8_launch(fp8_gemm_simt_kernel<false>, ctas, 256, 0, 1, stream, a);
}

}  // namespace gptq_host
