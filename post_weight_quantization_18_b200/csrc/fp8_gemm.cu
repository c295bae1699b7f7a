// fp8_gemm.cu — the products of the e4m3 format on the tcgen05 tensor cores:
//   Y[i, j] = sum_g sx[i, g] sw[j / 128, g] (sum over the 128 columns of block g of X W),
// and the gated pair h = silu(X Wg^T) (X Wu^T), quantized again with one scale per row and 128
// columns.
//
// The scales differ from block to block of K, so a tensor-memory accumulator covers one block of
// 128 columns (four kind::f8f6f4 MMAs) and the scaled sum over the blocks is kept in fp32
// registers: while the MMAs fill one accumulator, the epilogue warps read the last one, multiply
// by sx sw (one number per row and weight block) and add.
//
// Warps: 0 TMA producer, 1 TMEM owner and MMA issuer, 4-11 epilogue (two per quarter of the TMEM
// lanes; a thread owns one row and 64 columns of each of the tile's NB weight blocks).
//   wide   (SPLIT = false): persistent, one CTA per SM, tiles of 128 x 256 (two blocks of W rows;
//          for the gated pair one of Wg and the same of Wu), stored through shared memory in
//          whole 128-byte lines.
//   split  (SPLIT = true): one tile of 128 x 128 (gated: 128 + 128) per cluster, the blocks of K
//          shared out among the cluster's CTAs; every CTA leaves its sums in shared memory and
//          the rows are then added up over the cluster, always in the same order.
// Every mbarrier wait is bounded (GPTQ_ERR_TIMEOUT on expiry); a CTA that gives up waits
// (bounded) for the loads and MMAs it already issued before it frees TMEM and exits.
#include "fp8.cuh"

namespace {

constexpr int BM = 128, BB = 128, BK = 128;  // rows of X, of one weight block, columns of K
constexpr int TILE_BYTES = 128 * BK;         // 16 KB: a 128 x 128 operand tile
constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4, N_EPI = 8;
// Registers a thread: 168 at launch (65536 / 384); the first warpgroup gives up all but 56 and the
// two epilogue warpgroups take 224: 128 * 56 + 256 * 224 = 64512 of the 384 * 168 = 64512.
constexpr int REGS_LOAD = 56, REGS_EPI = 224;
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUP = 8;                     // tile rows per band of the tile order
constexpr int STAGE_OUT = 4096;              // staging of one epilogue warp's stores
constexpr int PART_PITCH = 132;              // floats: rows of 33 * 16 bytes, conflict-free

template <int NB>
struct Cfg {
  static constexpr int STAGE_BYTES = (1 + NB) * TILE_BYTES;
  static constexpr int STAGES = NB == 2 ? 4 : 6;  // 192 KB either way
  static constexpr int NBUF = 4 / NB;             // accumulators of NB * 128 TMEM columns
  static constexpr int DATA = STAGES * STAGE_BYTES + N_EPI * STAGE_OUT;
  static constexpr int SMEM = DATA + 512 + 1024;    // barriers, alignment
};

struct TcArgs {
  int M, N, nkb;
  const float* sx;
  long long ldsx;
  const float* sw[2];
  long long ldsw[2];
  void* y;
  long long ldy;
  float* sy;
  long long ldsy;
  int y_dtype;
  bool y_vec;   // rows of y are 16-byte aligned
  int x_rows;   // rows of the X box
  int tiles_m, tiles_n, n_tiles;
  int split;    // CTAs per cluster
  int32_t* status;
};

// D[tmem] (+)= A[smem] B[smem], kind::f8f6f4 (e4m3 operands, fp32 accumulate), 32 columns of K.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// tcgen05.wait::ld naming the registers, so that no use of them is scheduled before it.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// Two fp32 fused multiply-adds in one instruction: acc += d * f.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t f2) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(f2));
}
__device__ __forceinline__ uint64_t pair2(float f) {
  uint64_t r;
  const uint32_t b = __float_as_uint(f);
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(b));
  return r;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Tile t -> (tm, tn): bands of GROUP tile rows; inside a band, down each tile column in turn, so
// that the CTAs running together share a few panels of each operand in L2.
__device__ __forceinline__ void tile_of(int t, const TcArgs& a, int& tm, int& tn) {
  const int band = GROUP * a.tiles_n;
  const int gm = t / band, r = t % band;
  const int h = min(GROUP, a.tiles_m - gm * GROUP);
  tm = gm * GROUP + r % h;
  tn = r / h;
}

// Eight 16-byte pieces a row of a warp's staging area, 32 rows: written by the lane that owns the
// row, read back as whole lines. The piece's place is swizzled by the row, so neither conflicts.
__device__ __forceinline__ uint4* staged(uint8_t* st, int row, int piece) {
  return reinterpret_cast<uint4*>(st + row * 128 + ((piece ^ (row & 7)) << 4));
}

// The same with four pieces a row.
__device__ __forceinline__ uint4* staged64(uint8_t* st, int row, int piece) {
  return reinterpret_cast<uint4*>(st + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}

// 128 bytes of each of the warp's 32 rows, from staging to Y at column col0 (of element size ES).
template <int ES>
__device__ __forceinline__ void flush_rows(const TcArgs& a, uint8_t* st, int row0, int col0,
                                           int lane) {
  constexpr int PER = 16 / ES;  // elements of a piece
  const int piece = lane & 7;
  const int col = col0 + piece * PER;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    const uint4 v = *staged(st, r, piece);
    if (row0 + r < a.M && col < a.N) {
      uint8_t* p = reinterpret_cast<uint8_t*>(a.y) + ((long long)(row0 + r) * a.ldy + col) * ES;
      if (a.y_vec && col + PER <= a.N) {
        *reinterpret_cast<uint4*>(p) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if (col + e < a.N) {
            if constexpr (ES == 4)
              reinterpret_cast<uint32_t*>(p)[e] = w[e];
            else if constexpr (ES == 2)
              reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
            else
              p[e] = (uint8_t)(w[e >> 2] >> ((e & 3) * 8));
          }
      }
    }
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == GPTQ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int NB, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW0,
                const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ TcArgs args) {
  using C = Cfg<NB>;
  static_assert(!GATED || NB == 2, "the gated pair holds a block of each weight");
  static_assert(C::SMEM <= 232448 && REGS_LOAD * 128 + REGS_EPI * 256 <= 168 * THREADS, "limits");
  static_assert(!SPLIT || NB * BM * PART_PITCH * 4 <= C::STAGES * C::STAGE_BYTES, "partial sums");
  constexpr uint32_t IDESC = gptq::instr_desc(/*e4m3*/ 0, 0, 0, BM, NB * BB);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* out_stage = smem + C::STAGES * C::STAGE_BYTES;
  // the gated pair stages 64 bytes a row; behind them the rows' maxima, [2 tiles][2 halves][BM]
  uint32_t* amax = reinterpret_cast<uint32_t*>(out_stage + N_EPI * STAGE_OUT / 2);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::DATA);  // [STAGES]
  uint64_t* empty = full + C::STAGES;                            // [STAGES]
  uint64_t* acc_full = empty + C::STAGES;                        // [NBUF]
  uint64_t* acc_empty = acc_full + C::NBUF;                      // [NBUF]
  uint64_t* halves = acc_empty + C::NBUF;                        // [4] row maxima exchanged
  uint64_t* mma_drain = halves + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* skip_flag = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *skip_flag = gptq::status_bad(args.status) ? 1 : 0;
    *abort_flag = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      gptq::mbar_init(&full[s], 1);
      gptq::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::NBUF; ++b) {
      gptq::mbar_init(&acc_full[b], 1);
      gptq::mbar_init(&acc_empty[b], N_EPI);
    }
    for (int q = 0; q < 4; ++q) gptq::mbar_init(&halves[q], 2);
    gptq::mbar_init(mma_drain, 1);
    gptq::fence_barrier_init();
    gptq::tma_prefetch_desc(&tmX);
    gptq::tma_prefetch_desc(&tmW0);
    if (GATED) gptq::tma_prefetch_desc(&tmW1);
  }
  if (warp == 1) {
    gptq::tmem_alloc(tmem_slot, TMEM_COLS);
    gptq::tmem_relinquish();
  }
  gptq::tc_fence_before();
  __syncthreads();
  gptq::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // The CTA's share: tiles t, t + step, ..., blocks [kb0, kb1) of K.
  int t0 = blockIdx.x, step = gridDim.x, kb0 = 0, kb1 = args.nkb;
  uint32_t rank = 0;
  if constexpr (SPLIT) {
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    t0 = blockIdx.x / args.split;
    step = args.n_tiles;
    kb0 = (int)((long long)args.nkb * rank / args.split);
    kb1 = (int)((long long)args.nkb * (rank + 1) / args.split);
  }

  if (warp < EPI_WARP0) {
    regs_dec<REGS_LOAD>();
    if (*skip_flag) {
    } else if (warp == 0) {
      if (lane == 0) {  // ---------------- TMA producer ----------------
        const uint32_t bytes = (uint32_t)(args.x_rows * BK + NB * TILE_BYTES);
        int stage = 0;
        uint32_t phase = 0, filled = 0, fill_parity = 0;
        for (int t = t0; t < args.n_tiles && !*abort_flag; t += step) {
          int tm, tn;
          tile_of(t, args, tm, tn);
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!gptq::mbar_wait(&empty[stage], phase ^ 1, abort_flag)) break;
            uint8_t* sx = smem + stage * C::STAGE_BYTES;
            gptq::mbar_arrive_expect_tx(&full[stage], bytes);
            gptq::tma_load_2d(sx, &tmX, &full[stage], kb * BK, tm * BM);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              gptq::tma_load_2d(sx + (1 + b) * TILE_BYTES, GATED && b ? &tmW1 : &tmW0,
                                &full[stage], kb * BK, (GATED ? tn : tn * NB + b) * BB);
            filled |= 1u << stage;
            fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
          }
        }
        if (*abort_flag)
          for (int s = 0; s < C::STAGES; ++s)
            if (filled & (1u << s)) gptq::mbar_drain(&full[s], (fill_parity >> s) & 1u);
      }
    } else if (warp == 1) {
      if (lane == 0) {  // ---------------- MMA issuer ----------------
        int stage = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int t = t0; t < args.n_tiles && ok; t += step) {
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!gptq::mbar_wait(&acc_empty[buf], acc_phase ^ 1, abort_flag) ||
                !gptq::mbar_wait(&full[stage], phase, abort_flag)) {
              ok = false;
              break;
            }
            gptq::tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(buf * NB * BB);
            const uint32_t sx = gptq::smem_u32(smem + stage * C::STAGE_BYTES);
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)  // 32 columns: 32 bytes along the swizzled rows
              mma_f8(d, gptq::smem_desc_sw128(sx + kk * 32, 16, 1024),
                     gptq::smem_desc_sw128(sx + TILE_BYTES + kk * 32, 16, 1024), IDESC, kk > 0);
            gptq::mma_commit(&empty[stage]);
            gptq::mma_commit(&acc_full[buf]);
            if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
            if (++buf == C::NBUF) { buf = 0; acc_phase ^= 1; }
          }
        }
        if (*abort_flag) {
          gptq::mma_commit(mma_drain);
          gptq::mbar_drain(mma_drain, 0);
        }
      }
    }
    if constexpr (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    regs_inc<REGS_EPI>();
    if (!*skip_flag) {
      // ---------------- epilogue ----------------
      const int quarter = warp & 3, half = (warp - EPI_WARP0) >> 2;
      const uint32_t lane_field = (uint32_t)(quarter * 32) << 16;
      uint8_t* st = out_stage + (warp - EPI_WARP0) * (GATED ? STAGE_OUT / 2 : STAGE_OUT);
      int buf = 0;
      uint32_t acc_phase = 0, tile_parity = 0;
      bool ok = true;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        int tm, tn;
        tile_of(t, args, tm, tn);
        const int row0 = tm * BM + quarter * 32, row = row0 + lane;
        // The thread's NB chunks of 64 columns: chunk c starts at TMEM column tcol[c], sw[c] are
        // the scales of its weight block (of some block, for columns behind the last).
        int tcol[NB];
        const float* sw[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) {
          const int blk = GATED ? tn : tn * NB + (NB == 2 ? half : 0);
          tcol[c] = GATED ? c * BB + half * 64 : half * (NB * 64) + c * 64;
          const bool in = blk * BB < args.N;
          sw[c] = GATED && c ? args.sw[1] + (in ? blk * args.ldsw[1] : 0)
                             : args.sw[0] + (in ? blk * args.ldsw[0] : 0);
        }
        const float* sxr = args.sx + (long long)min(row, args.M - 1) * args.ldsx;
        const bool rows_here = row0 < args.M;  // of the warp
        uint64_t acc[NB][32];
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[c][e] = 0ull;
        float nsx = 0.f, nsw[NB];
        if (kb0 < kb1) {
          nsx = __ldg(sxr + kb0);
#pragma unroll
          for (int c = 0; c < NB; ++c) nsw[c] = __ldg(sw[c] + kb0);
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          uint64_t f[NB];
#pragma unroll
          for (int c = 0; c < NB; ++c) f[c] = pair2(nsx * nsw[c]);
          if (kb + 1 < kb1) {  // the next block's scales, on their way while this one is summed
            nsx = __ldg(sxr + kb + 1);
#pragma unroll
            for (int c = 0; c < NB; ++c) nsw[c] = __ldg(sw[c] + kb + 1);
          }
          if (!gptq::mbar_wait(&acc_full[buf], acc_phase, abort_flag)) {
            ok = false;
            break;
          }
          gptq::tc_fence_after();
          if (rows_here) {
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t r[32];
                __syncwarp();
                gptq::tmem_ld_32x32b_x32(
                    tmem_base + lane_field + (uint32_t)(buf * NB * BB + tcol[c] + 32 * q), r);
                tmem_wait32(r);
#pragma unroll
                for (int e = 0; e < 16; ++e) fma2(acc[c][16 * q + e], r[2 * e], r[2 * e + 1], f[c]);
              }
          }
          gptq::tc_fence_before();
          __syncwarp();
          if (lane == 0) gptq::mbar_arrive(&acc_empty[buf]);
          if (++buf == C::NBUF) { buf = 0; acc_phase ^= 1; }
        }
        if (!ok) break;
        if constexpr (SPLIT) {
          // All MMAs of the CTA are done, so the operand ring is free: rows of sums, one array of
          // 128 columns per weight block.
          if (row < args.M) {
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              float* p = reinterpret_cast<float*>(smem) + (c * BM + quarter * 32 + lane) * PART_PITCH +
                         half * 64;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                *reinterpret_cast<float4*>(p + 4 * e) =
                    make_float4(lo2(acc[c][2 * e]), hi2(acc[c][2 * e]), lo2(acc[c][2 * e + 1]),
                                hi2(acc[c][2 * e + 1]));
            }
          }
        } else if constexpr (GATED) {
          // h over the thread's 64 columns; the row's maximum with the warp of the other half.
          const int col0 = tn * BB + half * 64;
          uint32_t mx = 0;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float h0 = gptq::silu_mul(lo2(acc[0][e]), lo2(acc[1][e]));
            const float h1 = gptq::silu_mul(hi2(acc[0][e]), hi2(acc[1][e]));
            if (col0 + 2 * e < args.N) mx = max(mx, gptq::mag_bits(h0));
            if (col0 + 2 * e + 1 < args.N) mx = max(mx, gptq::mag_bits(h1));
            asm("mov.b64 %0, {%1, %2};"
                : "=l"(acc[0][e])
                : "r"(__float_as_uint(h0)), "r"(__float_as_uint(h1)));
          }
          uint32_t* slot = amax + tile_parity * 2 * BM + quarter * 32 + lane;
          slot[half * BM] = mx;
          __syncwarp();
          if (lane == 0) gptq::mbar_arrive(&halves[quarter]);
          if (!gptq::mbar_wait(&halves[quarter], tile_parity, abort_flag)) {
            ok = false;
            break;
          }
          mx = max(mx, slot[(half ^ 1) * BM]);
          tile_parity ^= 1;
          float s, inv;
          gptq::block_scale(mx, s, inv);
          if (half == 0 && row < args.M) args.sy[(long long)row * args.ldsy + tn] = s;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t a = acc[0][8 * p + 2 * e], b = acc[0][8 * p + 2 * e + 1];
              w[e] = gptq::e4m3x4(lo2(a) * inv, hi2(a) * inv, lo2(b) * inv, hi2(b) * inv);
            }
            *staged64(st, lane, p) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), piece = lane & 3, col = col0 + piece * 16;
            const uint4 v = *staged64(st, r, piece);
            if (row0 + r < args.M && col < args.N) {
              uint8_t* p = reinterpret_cast<uint8_t*>(args.y) + (long long)(row0 + r) * args.ldy + col;
              if (args.y_vec && col + 16 <= args.N) {
                *reinterpret_cast<uint4*>(p) = v;
              } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (col + e < args.N) p[e] = (uint8_t)(w[e >> 2] >> ((e & 3) * 8));
              }
            }
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            const int col0 = tn * NB * BB + tcol[c];
            if (args.y_dtype == GPTQ_F32) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                  const uint64_t a = acc[c][16 * q + 2 * p], b = acc[c][16 * q + 2 * p + 1];
                  *staged(st, lane, p) = make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b,
                                                    (uint32_t)(b >> 32));
                }
                flush_rows<4>(args, st, row0, col0 + 32 * q, lane);
              }
            } else {
#pragma unroll
              for (int p = 0; p < 8; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack2(lo2(acc[c][4 * p + e]), hi2(acc[c][4 * p + e]), args.y_dtype);
                *staged(st, lane, p) = make_uint4(w[0], w[1], w[2], w[3]);
              }
              flush_rows<2>(args, st, row0, col0, lane);
            }
          }
        }
      }
    }
    if constexpr (SPLIT) {
      // Every thread of every CTA of the cluster passes both barriers, whatever happened above.
      cluster_sync();
      if (!*skip_flag) {
        int tm, tn;
        tile_of(t0, args, tm, tn);
        const int rows = min(BM, args.M - tm * BM);
        // Row rank + split * i of the tile belongs to this CTA; a warp takes a whole row.
        for (int r = (int)rank + args.split * (warp - EPI_WARP0); r < rows; r += args.split * N_EPI) {
          float4 v[NB];
  #pragma unroll
          for (int c = 0; c < NB; ++c) {
            const uint32_t at = gptq::smem_u32(reinterpret_cast<float*>(smem) +
                                               (c * BM + r) * PART_PITCH + lane * 4);
            float4 p[8];
  #pragma unroll
            for (int s = 0; s < 8; ++s)
              if (s < args.split) p[s] = ld_cluster(at, s);
            v[c] = p[0];
  #pragma unroll
            for (int s = 1; s < 8; ++s)
              if (s < args.split) {
                v[c].x += p[s].x;
                v[c].y += p[s].y;
                v[c].z += p[s].z;
                v[c].w += p[s].w;
              }
          }
          const long long row = tm * BM + r;
          const int col = tn * BB + lane * 4;
          float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
          if constexpr (GATED) {
            const float u[4] = {v[NB - 1].x, v[NB - 1].y, v[NB - 1].z, v[NB - 1].w};
            uint32_t mx = 0;
  #pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[e] = gptq::silu_mul(o[e], u[e]);
              if (col + e < args.N) mx = max(mx, gptq::mag_bits(o[e]));
            }
            float s, inv;
            gptq::block_scale(__reduce_max_sync(0xFFFFFFFFu, mx), s, inv);
            if (lane == 0) args.sy[row * args.ldsy + tn] = s;
            const uint32_t w = gptq::e4m3x4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
            uint8_t* p = reinterpret_cast<uint8_t*>(args.y) + row * args.ldy + col;
            if (args.y_vec && col + 4 <= args.N) {
              *reinterpret_cast<uint32_t*>(p) = w;
            } else {
  #pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < args.N) p[e] = (uint8_t)(w >> (e * 8));
            }
          } else {
            const long long at = row * args.ldy + col;
            if (args.y_vec && col + 4 <= args.N) {
              if (args.y_dtype == GPTQ_F32)
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(args.y) + at) = v[0];
              else
                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(args.y) + at) =
                    make_uint2(pack2(o[0], o[1], args.y_dtype), pack2(o[2], o[3], args.y_dtype));
            } else {
  #pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < args.N) gptq::store_out(args.y, at + e, o[e], args.y_dtype);
            }
          }
        }
      }
      cluster_sync();  // no CTA leaves while its sums may still be read
    }
  }

  gptq::tc_fence_before();
  __syncthreads();
  if (warp == 1) gptq::tmem_dealloc(tmem_base, TMEM_COLS);
  if (threadIdx.x == 0 && *abort_flag) gptq::set_status(args.status, GPTQ_ERR_TIMEOUT, 5);
}

template <int NB, bool GATED, bool SPLIT>
int launch(const CUtensorMap& tx, const CUtensorMap& tw0, const CUtensorMap& tw1, const TcArgs& a,
           int grid, cudaStream_t stream) {
  auto kernel = fp8_gemm_kernel<NB, GATED, SPLIT>;
  if (gptq_host::ensure_smem_attr(reinterpret_cast<const void*>(kernel), Cfg<NB>::SMEM) != 0)
    return GPTQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Cfg<NB>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = SPLIT ? (unsigned)a.split : 1u;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = SPLIT ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, tx, tw0, tw1, a) == cudaSuccess ? 0 : GPTQ_ERR_CUDA;
}

}  // namespace

namespace gptq_host {

bool fp8_gemm_tc_takes(const Fp8Gemm& g) {
  auto ok = [](const uint8_t* p, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0;
  };
  return ok(g.x, g.ldx) && ok(g.w[0], g.ldw[0]) && (g.w[1] == nullptr || ok(g.w[1], g.ldw[1]));
}

int fp8_gemm_tc(const Fp8Gemm& g, cudaStream_t stream) {
  const bool gated = g.w[1] != nullptr;
  const int sms = num_sms();
  TcArgs a{};
  a.M = g.m; a.N = g.n;
  a.nkb = (g.k + BK - 1) / BK;
  a.sx = g.sx; a.ldsx = g.ldsx;
  for (int i = 0; i < 2; ++i) {
    a.sw[i] = g.sw[i];
    a.ldsw[i] = g.ldsw[i];
  }
  a.y = g.y; a.ldy = g.ldy; a.y_dtype = g.y_dtype;
  a.sy = g.sy; a.ldsy = g.ldsy;
  a.status = g.status;
  const int es = gated ? 1 : g.y_dtype == GPTQ_F32 ? 4 : 2;
  a.y_vec = reinterpret_cast<uintptr_t>(g.y) % 16 == 0 && g.ldy * es % 16 == 0;
  a.tiles_m = (g.m + BM - 1) / BM;
  const int blocks_n = (g.n + BB - 1) / BB;
  // Rows of X that a tile can hold: a call of few rows brings only those (whole groups of the
  // swizzle's eight rows); what the MMA reads behind them feeds accumulator rows nobody reads.
  a.x_rows = g.m >= BM ? BM : (g.m + 7) / 8 * 8;

  // Few tiles: share the blocks of K out among a cluster, as long as every CTA keeps two of them.
  const long long narrow = (long long)a.tiles_m * blocks_n;
  const bool split = narrow <= sms;
  a.tiles_n = split || gated ? blocks_n : (blocks_n + 1) / 2;
  if ((long long)a.tiles_m * a.tiles_n > 0x3FFFFFFF) return GPTQ_ERR_CUDA;
  a.n_tiles = a.tiles_m * a.tiles_n;
  a.split = 1;
  if (split)
    while (a.split < 8 && narrow * a.split * 2 <= sms && a.nkb >= 4 * a.split) a.split *= 2;

  CUtensorMap tx, tw0, tw1;
  if (make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.x, (uint64_t)g.k, (uint64_t)g.m,
                   (uint64_t)g.ldx, BK, (uint32_t)a.x_rows, CU_TENSOR_MAP_SWIZZLE_128B) != 0 ||
      make_tmap_2d(&tw0, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.w[0], (uint64_t)g.k, (uint64_t)g.n,
                   (uint64_t)g.ldw[0], BK, BB, CU_TENSOR_MAP_SWIZZLE_128B) != 0)
    return GPTQ_ERR_CUDA;
  tw1 = tw0;
  if (gated &&
      make_tmap_2d(&tw1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.w[1], (uint64_t)g.k, (uint64_t)g.n,
                   (uint64_t)g.ldw[1], BK, BB, CU_TENSOR_MAP_SWIZZLE_128B) != 0)
    return GPTQ_ERR_CUDA;
  if (split) {
    const int grid = a.n_tiles * a.split;
    return gated ? launch<2, true, true>(tx, tw0, tw1, a, grid, stream)
                 : launch<1, false, true>(tx, tw0, tw1, a, grid, stream);
  }
  const int grid = a.n_tiles < sms ? a.n_tiles : sms;
  return gated ? launch<2, true, false>(tx, tw0, tw1, a, grid, stream)
               : launch<2, false, false>(tx, tw0, tw1, a, grid, stream);
}

}  // namespace gptq_host
