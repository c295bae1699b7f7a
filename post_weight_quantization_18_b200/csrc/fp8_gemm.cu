// fp8_gemm.cu — the products of the e4m3 format where the arithmetic outweighs the bytes:
//   Y[i, j] = sum_g sx[i, g] sw[j / 128, g] (sum over the 128 columns of block g of X W),
// and the gated pair h = silu(X Wg^T) (X Wu^T), quantized again with one scale per row and 128
// columns. (fp8_thin.cu has the calls of few rows.)
//
// The scales differ from block to block of K, so a tensor-memory accumulator covers one block of
// 128 columns (four kind::f8f6f4 MMAs) and the scaled sum over the blocks is kept in fp32
// registers: while the MMAs fill one accumulator, the epilogue warps read the last one, multiply
// by sx sw (one number per row and weight block) and add.
//
// Persistent pairs of CTAs (cta_group::2) own tiles of 256 x 256: each CTA brings its 128 rows of
// X and one of the tile's two blocks of 128 weight rows (gated pair: the first CTA the block of
// Wg, the second the same block of Wu), and the MMAs, issued by the first CTA, read both CTAs'
// shared memory. Each SM so loads 32 KB for a block of K instead of the 48 KB of a 128 x 256 tile
// of its own, which L2 does not deliver in the 512 cycles the MMAs take.
// Warps: 0 TMA producer, 1 TMEM owner and (first CTA) MMA issuer, 2 scales, 4-11 epilogue (two per
// quarter of the TMEM lanes; a thread owns one row and 64 columns of each of two chunks).
// Every mbarrier wait is bounded (GPTQ_ERR_TIMEOUT on expiry); a pair that gives up waits
// (bounded) for the loads and MMAs it already issued before it frees TMEM and exits.
//
// Measured (B200): 8192 x 8192 x 28672 in 1.86 to 1.93 ms, 2.0 PFLOP/s, at 1335 MHz under the 1 kW
// power limit. Two things bound it. The clock is the power's; and of the cycles at that clock the tensor
// pipe is busy 50 to 60 % (2048 x 4096 x 4096, 34 us: 52 %; gated 2000 x 6912 x 5120: 57 %), because a block
// of K takes the pair about 800 cycles, of which the MMAs are 512: they wait until the epilogue has read
// an accumulator, all eight loads of it. Without reading and scaling the accumulators the same pipeline
// takes 1.47 ms, the reads add 0.12, the multiply-adds 0.26. A 128 x 256 tile per CTA with the same
// loops: 2.3 ms.
#include "fp8_mma.cuh"

namespace {

using gptq::fma2;
using gptq::hi2;
using gptq::lo2;
using gptq::pack2;
using Scales = gptq::ScaleRing<128>;
using gptq::bar_wait;
using gptq::bar_wait_rest;

constexpr int BM = 128, BB = 128, BK = 128;  // rows of X of a CTA, of one weight block, columns of K
constexpr int TILE_BYTES = 128 * BK;         // 16 KB: a 128 x 128 operand tile
constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // of one CTA
constexpr int STAGES = 5;                    // 160 KB
constexpr int NBUF = 2;                      // accumulators of 256 TMEM columns
constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4, N_EPI = 8;
// Registers a thread: 168 at launch (65536 / 384); the first warpgroup gives up all but 56 and the
// two epilogue warpgroups take 224: 128 * 56 + 256 * 224 = 64512 = 384 * 168.
constexpr int REGS_LOAD = 56, REGS_EPI = 224;
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUP = 8;                     // tile rows per band of the tile order
constexpr int STAGE_OUT = 4096;              // staging of one epilogue warp's stores
constexpr int DATA = STAGES * STAGE_BYTES + N_EPI * STAGE_OUT + Scales::BYTES;
constexpr int SMEM = DATA + 512 + 1024;      // barriers, alignment
static_assert(SMEM <= 232448 && REGS_LOAD * 128 + REGS_EPI * 256 <= 168 * THREADS, "limits");
constexpr uint32_t IDESC = gptq::instr_desc(/*e4m3*/ 0, 0, 0, 2 * BM, 2 * BB);

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
  int y_align;  // of the rows of y, in bytes
  int tiles_m, tiles_n, n_tiles;
  int32_t* status;
};

// ---- the cta_group::2 forms: one pair of CTAs, barriers in the first ----
__device__ __forceinline__ uint32_t in_first_cta(uint32_t at) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(at));
  return a;
}
// A tile into this CTA's shared memory, counted on the first CTA's barrier.
__device__ __forceinline__ void load_tile_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                               int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// D (both CTAs' TMEM) (+)= A (both CTAs' rows) B (both CTAs' rows), 32 columns of K.
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(IDESC), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at the same place in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// Relaxed: what the arrival orders are reads of tensor memory, which the tcgen05 fence before it
// covers. A release at cluster scope would wait for every access to memory of the thread, 1000
// cycles in each block of K.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tile t -> (tm, tn): bands of GROUP tile rows; inside a band, down each tile column in turn, so
// that the pairs running together share a few panels of each operand in L2.
__device__ __forceinline__ void tile_of(int t, const TcArgs& a, int& tm, int& tn) {
  const int band = GROUP * a.tiles_n;
  const int gm = t / band, r = t % band;
  const int h = min(GROUP, a.tiles_m - gm * GROUP);
  tm = gm * GROUP + r % h;
  tn = r / h;
}

// Eight 16-byte pieces a row of a warp's staging area, 32 rows: written by the lane that owns the
// row, read back as whole lines. The piece's place is swizzled by the row, so neither conflicts.
__device__ __forceinline__ uint32_t staged(uint32_t st, int row, int piece) {
  return st + (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}

// The same with four pieces a row.
__device__ __forceinline__ uint32_t staged64(uint32_t st, int row, int piece) {
  return st + (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// 128 bytes of each of the warp's 32 rows, from staging to Y at column col0 (of element size ES).
template <int ES>
__device__ __forceinline__ void flush_rows(const TcArgs& a, uint32_t st, int row0, int col0,
                                           int lane) {
  constexpr int PER = 16 / ES;  // elements of a piece
  __syncwarp();
  if (a.y_align == 16) {
    const int piece = lane & 7, col = col0 + piece * PER;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      const uint4 v = lds16(staged(st, r, piece));
      if (row0 + r < a.M && col < a.N) {
        uint8_t* p = reinterpret_cast<uint8_t*>(a.y) + ((long long)(row0 + r) * a.ldy + col) * ES;
        if (col + PER <= a.N) {
          *reinterpret_cast<uint4*>(p) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < PER; ++e)
            if (col + e < a.N) {
              if constexpr (ES == 4)
                reinterpret_cast<uint32_t*>(p)[e] = w[e];
              else
                reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
            }
        }
      }
    }
  } else {  // a row at a time, one word a lane, so that the warp's stores are neighbours all the same
    uint8_t* p = reinterpret_cast<uint8_t*>(a.y) + ((long long)row0 * a.ldy + col0) * ES;
    const long long pitch = a.ldy * ES;
    const int rows = a.M - row0;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 4) {
      uint32_t w[4], next[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = gptq::flag_read(staged(st, r0 + i, lane >> 2) + (lane & 3) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) next[i] = ES == 4 ? 0u : __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
#pragma unroll
      for (int i = 0; i < 4; ++i, p += pitch)
        gptq::store_word<ES, 32>(p, lane, w[i], next[i], r0 + i < rows ? a.N - col0 : 0);
    }
  }
  __syncwarp();
}

template <bool GATED>
__global__ void __launch_bounds__(THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW0,
                const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ TcArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = (gptq::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t out_stage = smem + STAGES * STAGE_BYTES;
  // the gated pair stages 64 bytes a row; behind them the rows' maxima, [2 tiles][2 halves][BM]
  const uint32_t amax = out_stage + N_EPI * STAGE_OUT / 2;
  Scales scales;
  scales.buf = out_stage + N_EPI * STAGE_OUT;
  const uint32_t bars = smem + DATA;
  auto full = [&](int s) { return bars + (uint32_t)s * 8; };          // used in the first CTA
  auto empty = [&](int s) { return bars + (uint32_t)(STAGES + s) * 8; };
  auto acc_full = [&](int b) { return bars + (uint32_t)(2 * STAGES + b) * 8; };
  auto acc_empty = [&](int b) { return bars + (uint32_t)(2 * STAGES + NBUF + b) * 8; };  // first CTA
  auto halves = [&](int q) { return bars + (uint32_t)(2 * STAGES + 2 * NBUF + q) * 8; };
  const uint32_t mma_drain = bars + (2 * STAGES + 2 * NBUF + 4) * 8;
  scales.bars = mma_drain + 8;
  const uint32_t tmem_slot = scales.bars + Scales::BAR_BYTES;
  const uint32_t abort_flag = tmem_slot + 4, skip_flag = tmem_slot + 8;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));

  if (threadIdx.x == 0) {
    gptq::flag_write(abort_flag, 0);
    for (int s = 0; s < STAGES; ++s) {
      gptq::bar_init(full(s), 1);
      gptq::bar_init(empty(s), 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      gptq::bar_init(acc_full(b), 1);
      gptq::bar_init(acc_empty(b), 2 * N_EPI);
    }
    for (int q = 0; q < 4; ++q) gptq::bar_init(halves(q), 2);
    scales.init(N_EPI);
    gptq::bar_init(mma_drain, 1);
    gptq::fence_barrier_init();
    gptq::tma_prefetch_desc(&tmX);
    gptq::tma_prefetch_desc(&tmW0);
    if (GATED) gptq::tma_prefetch_desc(&tmW1);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    // Only now: the next kernel's CTAs wait for this kernel with their tensor memory in hand.
    gptq::let_next_kernel_start();
  }
  gptq::wait_for_previous_kernel();
  if (threadIdx.x == 0)
    gptq::flag_write(skip_flag, rank == 0 && gptq::status_bad(args.status) ? 1 : 0);
  gptq::tc_fence_before();
  gptq::cluster_sync();  // both CTAs' barriers are set up before either is signalled
  gptq::tc_fence_after();
  const uint32_t tmem_base = gptq::flag_read(tmem_slot);
  // Both CTAs take the same decision on the status: the first one's reading.
  uint32_t skip;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(skip)
               : "r"(in_first_cta(skip_flag))
               : "memory");
  const int t0 = blockIdx.x >> 1, step = gridDim.x >> 1, nkb = args.nkb;

  if (warp < EPI_WARP0) {
    gptq::regs_dec<REGS_LOAD>();
    if (skip) {
    } else if (warp == 0) {  // ---------------- TMA producer, of both CTAs ----------------
      const CUtensorMap* tmW = GATED && rank ? &tmW1 : &tmW0;
      const bool leader = gptq::elect_one();
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_parity = 0;
      bool ready = gptq::bar_poll(empty(0), 1), ok = true;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        int tm, tn;
        tile_of(t, args, tm, tn);
        const int xrow = (tm * 2 + (int)rank) * BM;
        const int wrow = (GATED ? tn : tn * 2 + (int)rank) * BB;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!bar_wait_rest(ready, empty(stage), phase ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sx = smem + (uint32_t)(stage * STAGE_BYTES), here = full(stage);
          filled |= 1u << stage;
          fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
          ready = gptq::bar_poll(empty(stage), phase ^ 1);
          if (leader) {
            const uint32_t bar = in_first_cta(here);
            // the first CTA expects both CTAs' bytes
            if (rank == 0) gptq::bar_expect(here, 2 * STAGE_BYTES);
            load_tile_pair(sx, &tmX, bar, kb * BK, xrow);
            load_tile_pair(sx + TILE_BYTES, tmW, bar, kb * BK, wrow);
          }
          __syncwarp();
        }
      }
      if (gptq::flag_read(abort_flag) && rank == 0)
        for (int s = 0; s < STAGES; ++s)
          if (filled & (1u << s)) gptq::bar_drain(full(s), (fill_parity >> s) & 1u);
    } else if (warp == 1 && rank == 0) {  // ---------------- MMA issuer, of the pair ----------------
      const bool leader = gptq::elect_one();
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, acc_ready = true, full_ready = gptq::bar_poll(full(0), 0);
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        for (int kb = 0; kb < nkb; ++kb) {
          if (!bar_wait_rest(acc_ready, acc_empty(buf), acc_phase ^ 1, abort_flag) ||
              !bar_wait_rest(full_ready, full(stage), phase, abort_flag)) {
            ok = false;
            break;
          }
          gptq::tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(buf * 2 * BB);
          const uint32_t sx = smem + (uint32_t)(stage * STAGE_BYTES);
          const uint32_t freed = empty(stage), filled = acc_full(buf);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
          if (++buf == NBUF) { buf = 0; acc_phase ^= 1; }
          full_ready = gptq::bar_poll(full(stage), phase);
          acc_ready = gptq::bar_poll(acc_empty(buf), acc_phase ^ 1);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)  // 32 columns: 32 bytes along the swizzled rows
              mma_f8_pair(d, gptq::smem_desc_sw128(sx + kk * 32, 16, 1024),
                          gptq::smem_desc_sw128(sx + TILE_BYTES + kk * 32, 16, 1024), kk > 0);
            commit_pair(freed);
            commit_pair(filled);
          }
          __syncwarp();
        }
      }
      if (gptq::flag_read(abort_flag)) {
        if (leader) commit_pair(mma_drain);
        __syncwarp();
        gptq::bar_drain(mma_drain, 0);
      }
    } else if (warp == 2) {  // ---------------- scales ----------------
      int chunk = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        int tm, tn;
        tile_of(t, args, tm, tn);
        // of some block, for columns behind the last
        const int last = (args.N - 1) / BB, b0 = GATED ? tn : tn * 2, b1 = min(b0 + 1, last);
        ok = scales.produce(args.sx, args.ldsx, (tm * 2 + (int)rank) * BM, BM, args.M,
                            args.sw[0] + b0 * args.ldsw[0],
                            GATED ? args.sw[1] + b0 * args.ldsw[1] : args.sw[0] + b1 * args.ldsw[0],
                            0, nkb, chunk, phase, abort_flag);
      }
      Scales::drain();
    }
  } else {
    gptq::regs_inc<REGS_EPI>();
    if (!skip) {
      // ---------------- epilogue ----------------
      const int quarter = warp & 3, half = (warp - EPI_WARP0) >> 2;
      const uint32_t lane_field = (uint32_t)(quarter * 32) << 16;
      const uint32_t st = out_stage + (warp - EPI_WARP0) * (GATED ? STAGE_OUT / 2 : STAGE_OUT);
      int buf = 0, chunk = 0;
      uint32_t acc_phase = 0, tile_parity = 0, chunk_phase = 0;
      bool ok = true, acc_ready = false;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        int tm, tn;
        tile_of(t, args, tm, tn);
        const int row0 = (tm * 2 + (int)rank) * BM + quarter * 32, row = row0 + lane;
        // The thread's two chunks of 64 columns: chunk c starts at TMEM column tcol[c].
        int tcol[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) tcol[c] = GATED ? c * BB + half * 64 : half * BB + c * 64;
        uint64_t acc[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[c][e] = 0ull;
        for (int kb = 0; kb < nkb; ++kb) {
          const int j = kb % Scales::KC;
          if (j == 0 && !bar_wait(scales.full(chunk), chunk_phase, abort_flag)) {
            ok = false;
            break;
          }
          const float sx = scales.row(chunk, j, quarter * 32 + lane);
          const float2 sw = scales.blocks(chunk, j);
          uint64_t f[2];
          f[0] = gptq::pair2(sx * (GATED ? sw.x : half ? sw.y : sw.x));
          f[1] = GATED ? gptq::pair2(sx * sw.y) : f[0];
          if (j == Scales::KC - 1 || kb == nkb - 1) {
            __syncwarp();
            if (lane == 0) gptq::bar_arrive(scales.empty(chunk));
            if (++chunk == Scales::CHUNKS) { chunk = 0; chunk_phase ^= 1; }
          }
          if (!bar_wait_rest(acc_ready, acc_full(buf), acc_phase, abort_flag)) {
            ok = false;
            break;
          }
          gptq::tc_fence_after();
          const uint32_t acc_col = tmem_base + lane_field + (uint32_t)(buf * 2 * BB);
          const uint32_t freed = acc_empty(buf);
          if (++buf == NBUF) { buf = 0; acc_phase ^= 1; }
          // Sixteen columns at a time: while the MMAs write tensor memory, larger loads are slower
          // (32: 750 cycles for the block instead of 660, alone with the MMAs).
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = q >> 2, e0 = (q & 3) * 8;
            uint32_t r[16];
            gptq::tmem_ld_32x32b_x16(acc_col + (uint32_t)(tcol[c] + 16 * (q & 3)), r);
            gptq::tmem_ld_wait();
            if (q == 7) {  // all of it is in registers: the accumulator is free
              gptq::tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_first(in_first_cta(freed));
              acc_ready = gptq::bar_poll(acc_full(buf), acc_phase);
            }
            gptq::settled(r);
#pragma unroll
            for (int e = 0; e < 8; ++e) fma2(acc[c][e0 + e], r[2 * e], r[2 * e + 1], f[c]);
          }
        }
        if (!ok) break;
        if constexpr (GATED) {
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
          const uint32_t slot = amax + (uint32_t)(tile_parity * 2 * BM + quarter * 32 + lane) * 4;
          gptq::flag_write(slot + half * BM * 4, mx);
          __syncwarp();
          if (lane == 0) gptq::bar_arrive(halves(quarter));
          if (!bar_wait(halves(quarter), tile_parity, abort_flag)) {
            ok = false;
            break;
          }
          mx = max(mx, gptq::flag_read(slot + (half ^ 1) * BM * 4));
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
            sts16(staged64(st, lane, p), make_uint4(w[0], w[1], w[2], w[3]));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), piece = lane & 3, col = col0 + piece * 16;
            const uint4 v = lds16(staged64(st, r, piece));
            if (row0 + r < args.M && col < args.N) {
              uint8_t* p = reinterpret_cast<uint8_t*>(args.y) + (long long)(row0 + r) * args.ldy + col;
              if (args.y_align == 16 && col + 16 <= args.N) {
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
          for (int c = 0; c < 2; ++c) {
            const int col0 = tn * 2 * BB + tcol[c];
            if (args.y_dtype == GPTQ_F32) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                  const uint64_t a = acc[c][16 * q + 2 * p], b = acc[c][16 * q + 2 * p + 1];
                  sts16(staged(st, lane, p), make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b,
                                                    (uint32_t)(b >> 32)));
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
                sts16(staged(st, lane, p), make_uint4(w[0], w[1], w[2], w[3]));
              }
              flush_rows<2>(args, st, row0, col0, lane);
            }
          }
        }
      }
    }
  }

  // The pair leaves together: the MMAs read both CTAs' shared memory and the barriers are the first
  // CTA's. A CTA that gave up may have loads in flight that the other one's barrier never counted;
  // they have long landed a millisecond later.
  if (gptq::flag_read(abort_flag) && threadIdx.x == 0) {
    const uint64_t now = gptq::globaltimer_ns();
    while (gptq::globaltimer_ns() - now < 1000000ull) {
    }
  }
  gptq::tc_fence_before();
  __syncthreads();
  gptq::cluster_sync();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  if (threadIdx.x == 0 && gptq::flag_read(abort_flag)) gptq::set_status(args.status, GPTQ_ERR_TIMEOUT, 5);
}

}  // namespace

namespace gptq_host {

bool fp8_tma_takes(const Fp8Gemm& g) {
  auto ok = [](const uint8_t* p, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0;
  };
  return ok(g.x, g.ldx) && ok(g.w[0], g.ldw[0]) && (g.w[1] == nullptr || ok(g.w[1], g.ldw[1]));
}

// Rounds of pairs, 0.48 us for a block of K (512 x 4096 x 4096: 19 us, one round of 32 blocks).
long long fp8_wide_cost(const Fp8Gemm& g) {
  const long long cols = g.w[1] != nullptr ? BB : 2 * BB;
  const long long tiles = ((g.m + 2 * BM - 1) / (2 * BM)) * ((g.n + cols - 1) / cols);
  const int pairs = num_sms() / 2;
  return (tiles + pairs - 1) / pairs * 285;
}

int fp8_gemm_wide(const Fp8Gemm& g, cudaStream_t stream) {
  const bool gated = g.w[1] != nullptr;
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
  a.y_align = row_align(g.y, g.ldy * es);
  a.tiles_m = (g.m + 2 * BM - 1) / (2 * BM);
  const int cols = gated ? BB : 2 * BB;
  a.tiles_n = (g.n + cols - 1) / cols;
  if ((long long)a.tiles_m * a.tiles_n > 0x3FFFFFFF) return GPTQ_ERR_CUDA;
  a.n_tiles = a.tiles_m * a.tiles_n;
  CUtensorMap tx, tw0, tw1;
  if (make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.x, (uint64_t)g.k, (uint64_t)g.m,
                   (uint64_t)g.ldx, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B) != 0 ||
      make_tmap_2d(&tw0, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.w[0], (uint64_t)g.k, (uint64_t)g.n,
                   (uint64_t)g.ldw[0], BK, BB, CU_TENSOR_MAP_SWIZZLE_128B) != 0)
    return GPTQ_ERR_CUDA;
  tw1 = tw0;
  if (gated &&
      make_tmap_2d(&tw1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.w[1], (uint64_t)g.k, (uint64_t)g.n,
                   (uint64_t)g.ldw[1], BK, BB, CU_TENSOR_MAP_SWIZZLE_128B) != 0)
    return GPTQ_ERR_CUDA;
  const int pairs = num_sms() / 2;
  const int grid = 2 * (a.n_tiles < pairs ? a.n_tiles : pairs);
  return gated ? fp8_launch(fp8_gemm_kernel<true>, grid, THREADS, SMEM, 2, stream, tx, tw0, tw1, a)
               : fp8_launch(fp8_gemm_kernel<false>, grid, THREADS, SMEM, 2, stream, tx, tw0, tw1, a);
}

}  // namespace gptq_host
