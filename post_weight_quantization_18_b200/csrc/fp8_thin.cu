// fp8_thin.cu — the products of the e4m3 format where the weight's bytes outweigh the arithmetic: a
// few hundred rows of activations at most.
//
// The time is that of streaming W once, so the output is cut into columns only: tiles of 128
// activation rows by BN = 32 CH weight rows, BN chosen so that one round of CTAs covers the
// weight, each CTA running over all of K. A pipeline stage is KPS blocks of 128 columns, brought by one
// TMA load per operand (a three-dimensional box: 128 bytes of each row, KPS blocks along K),
// because the streaming rate of a CTA is set by its loads and barrier steps, not by its bytes. As
// in fp8_gemm.cu a tensor-memory accumulator covers one block of K, and the scaled sums live in
// fp32 registers of the epilogue warps.
//   CLUSTERED = false  persistent; results go out from registers (gated pair: BN = 128, the row's
//                      scale found by the two warps that hold the row)
//   CLUSTERED = true   one output tile per cluster, when there are too few tiles for the SMs: its
//                      CTAs share out the blocks of K (plain) or the 128 columns of the gated
//                      pair's scale and then K. Plain: the sums of a row are sent to one of them
//                      and added up there, always in the same order. Gated:
//                      h is made where its sums are, a row's maximum goes round the cluster.
// Measured (B200): 64 x 8192 x 28672 in 45 us (5.3 TB/s), 64 x 11008 x 4096 in 12.0 us (a loop that
// only streams this weight: 10.3), 512 x 4096 x 4096 in 13.0 us, gated 100 x 11008 x 4096 in 24.5 us.
// Warps: 0 TMA producer, 1 TMEM owner and MMA issuer, 2 scales, 4-11 epilogue (two per quarter of the TMEM
// lanes, half the tile's columns each). Every wait is bounded as in fp8_gemm.cu.
#include <cudaTypedefs.h>

#include "fp8_mma.cuh"

namespace {

using gptq::fma2;
using gptq::hi2;
using gptq::lo2;
using Scales = gptq::ScaleRing<128>;
using gptq::bar_wait;
using gptq::bar_wait_rest;

constexpr int BM = 128, BK = 128;
constexpr int THREADS = 384, EPI_WARP0 = 4, N_EPI = 8;
constexpr int RING_BYTES = 196 * 1024;   // operand ring
constexpr int MAX_STAGES = 8;
constexpr int STAGE_OUT = 1024;          // staging of one epilogue warp's stores
constexpr int SMEM_BYTES = RING_BYTES + Scales::BYTES + 4 * BM * 4 + N_EPI * STAGE_OUT + 512 + 1024;
constexpr uint32_t TMEM_COLS = 512;

struct ThinArgs {
  int M, N, nkb;      // nkb: blocks of K, the last possibly short
  int nfull;          // whole ones, which the three-dimensional maps cover
  const float* sx;
  long long ldsx;
  const float* sw[2];
  long long ldsw[2];
  void* y;
  long long ldy;
  float* sy;
  long long ldsy;
  int y_dtype;
  int y_align;        // of the rows of y, in bytes
  int x_rows;         // rows of the X box
  int tiles_n, n_tiles;
  int ksplit;         // CTAs of a cluster along K, which have kq stages each, the first kr one more
  int kq, kr;
  int stages, stage_bytes;
  int32_t* status;
};

// Rows that 16-byte stores cannot address: 32 bytes of each of the warp's 32 rows, the lane's own being
// the words get(0) .. get(7), through shared memory, so that a store of the warp covers four rows and not
// 32 (2000 x 300 x 4096: 19 us with one row a lane, 10.2 so; 300 x 14001 x 512: 13.2).
template <int ES, typename Get>
__device__ __forceinline__ void store_rows(const ThinArgs& a, uint32_t st, int row0, int col0, int lane,
                                           Get get) {
  auto place = [&](int row, int piece) {  // neither the writes nor the reads conflict
    return st + (uint32_t)(row * 32 + ((piece ^ ((row >> 2) & 1)) << 4));
  };
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 2; ++p)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(place(lane, p)), "r"(get(4 * p)),
                 "r"(get(4 * p + 1)), "r"(get(4 * p + 2)), "r"(get(4 * p + 3))
                 : "memory");
  __syncwarp();
  const int i = lane & 7;
  uint32_t w[8];
#pragma unroll
  for (int r = 0; r < 8; ++r)
    w[r] = gptq::flag_read(place(4 * r + (lane >> 3), i >> 2) + (i & 3) * 4);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w[r], 1, 8);
    const int row = row0 + 4 * r + (lane >> 3);
    if (row < a.M)
      gptq::store_word<ES, 8>(reinterpret_cast<uint8_t*>(a.y) + ((long long)row * a.ldy + col0) * ES, i,
                              w[r], next, a.N - col0);
  }
}

struct Maps {  // [0]: whole blocks of K, three-dimensional; [1]: any block, two-dimensional
  CUtensorMap x[2], w0[2], w1[2];
};

template <int NW, int CH, bool CLUSTERED>
__global__ void __launch_bounds__(THREADS, 1)
fp8_thin_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ThinArgs args) {
  constexpr int BN = 32 * CH;
  constexpr int COLS = NW * BN;                                 // TMEM columns of a block of K
  constexpr int KPS = COLS <= 64 ? 4 : COLS <= 128 ? 2 : 1;     // two groups fit in 512 columns
  constexpr int CN = NW == 2 ? 128 / BN : 1;                    // CTAs along the columns of a scale
  constexpr bool GROUPED = CLUSTERED && NW == 2;                // a cluster holds groups of a scale
  constexpr bool TWO_BLOCKS = 128 % BN != 0;                    // a tile may span two weight blocks
  constexpr int PITCH = BN + 4;                                 // floats; an odd number of 16 bytes
  // 128 sums a thread: the first warpgroup's registers go to the epilogue's, 128 * 56 + 256 * 224 =
  // 384 * 168 as in fp8_gemm.cu
  constexpr bool SPLIT_REGS = NW * CH == 8;
  static_assert(NW == 1 || CN * BN == 128, "the gated pair's tiles divide a scale's columns");
  static_assert(!CLUSTERED || GROUPED || CH == 1, "sixteen columns a thread");
  static_assert((BM + 7) * PITCH * 4 <= RING_BYTES, "partial sums");
  constexpr uint32_t IDESC = gptq::instr_desc(/*e4m3*/ 0, 0, 0, BM, BN);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = (gptq::smem_u32(smem_raw) + 1023u) & ~1023u;
  Scales scales;
  scales.buf = smem + RING_BYTES;
  // [2 tiles][2 halves][BM], or clustered [BM]
  const uint32_t amax = scales.buf + Scales::BYTES;
  const uint32_t out_stage = amax + 4 * BM * 4;
  const uint32_t bars = out_stage + N_EPI * STAGE_OUT;
  auto full = [&](int s) { return bars + (uint32_t)s * 8; };
  auto empty = [&](int s) { return bars + (uint32_t)(MAX_STAGES + s) * 8; };
  auto acc_full = [&](int b) { return bars + (uint32_t)(2 * MAX_STAGES + b) * 8; };
  auto acc_empty = [&](int b) { return bars + (uint32_t)(2 * MAX_STAGES + 2 + b) * 8; };
  auto halves = [&](int q) { return bars + (uint32_t)(2 * MAX_STAGES + 4 + q) * 8; };
  const uint32_t mma_drain = bars + (2 * MAX_STAGES + 8) * 8;
  scales.bars = mma_drain + 8;
  const uint32_t tmem_slot = scales.bars + Scales::BAR_BYTES;
  const uint32_t abort_flag = tmem_slot + 4, skip_flag = tmem_slot + 8;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if constexpr (GROUPED) {
    if (threadIdx.x < BM) gptq::flag_write(amax + threadIdx.x * 4, 0);
    gptq::cluster_arrive();  // the CTA has started, its maxima are zero
  }
  if (threadIdx.x == 0) {
    gptq::flag_write(abort_flag, 0);
    for (int s = 0; s < MAX_STAGES; ++s) {
      gptq::bar_init(full(s), 1);
      gptq::bar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      gptq::bar_init(acc_full(b), 1);
      gptq::bar_init(acc_empty(b), N_EPI);
    }
    for (int q = 0; q < 4; ++q) gptq::bar_init(halves(q), 2);
    scales.init(N_EPI);
    gptq::bar_init(mma_drain, 1);
    gptq::fence_barrier_init();
  } else if (threadIdx.x == 32 * 3) {
    gptq::tma_prefetch_desc(&maps.x[0]);
    gptq::tma_prefetch_desc(&maps.w0[0]);
    if (NW == 2) gptq::tma_prefetch_desc(&maps.w1[0]);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot),
                 "r"(TMEM_COLS)
                 : "memory");
    gptq::tmem_relinquish();
    // Only now: the next kernel's CTAs wait for this kernel with their tensor memory in hand.
    gptq::let_next_kernel_start();
  }
  gptq::wait_for_previous_kernel();
  if (threadIdx.x == 0) gptq::flag_write(skip_flag, gptq::status_bad(args.status) ? 1 : 0);
  gptq::tc_fence_before();
  __syncthreads();
  gptq::tc_fence_after();
  const uint32_t tmem_base = gptq::flag_read(tmem_slot);

  // The CTA's tiles t0, t0 + step, ... (of whole clusters), its part of the scale's columns, and
  // its blocks [kb0, kb1) of K: whole stages, the last one possibly short.
  int t0 = blockIdx.x, step = gridDim.x, kb0 = 0, kb1 = args.nkb, npart = 0;
  uint32_t rank = 0;
  int csize = 1;
  if constexpr (CLUSTERED) {
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    csize = CN * args.ksplit;
    asm("mov.u32 %0, %clusterid.x;" : "=r"(t0));
    step = args.n_tiles;
    npart = rank % CN;
    const int ks = rank / CN;
    kb0 = (ks * args.kq + min(ks, args.kr)) * KPS;
    kb1 = min(args.nkb, kb0 + (args.kq + (ks < args.kr ? 1 : 0)) * KPS);
  }
  auto row_tile = [&](int t) { return t / args.tiles_n; };
  auto col_of = [&](int t) { return (t % args.tiles_n) * (CN * BN) + npart * BN; };

  // In clusters: the barriers that every thread passes, whatever happens to it.
  auto pass_barriers = [&] {
    if constexpr (GROUPED) gptq::cluster_wait();
    if (!GROUPED || args.ksplit == 2) gptq::cluster_sync();
    gptq::cluster_sync();
  };

  if (warp < EPI_WARP0) {
    if constexpr (SPLIT_REGS) gptq::regs_dec<56>();
    if (gptq::flag_read(skip_flag)) {
    } else if (warp == 0) {  // ---------------- TMA producer ----------------
      const bool leader = gptq::elect_one();
      const int xb = args.x_rows * BK, wb = BN * BK;  // bytes of one block
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_parity = 0;
      bool ok = true, ready = true;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        const int xr = row_tile(t) * BM, wr = col_of(t);
        for (int kb = kb0; kb < kb1; kb += KPS) {
          if (!bar_wait_rest(ready, empty(stage), phase ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sx = smem + (uint32_t)(stage * args.stage_bytes);
          const uint32_t sw = sx + (uint32_t)(KPS * xb), here = full(stage);
          filled |= 1u << stage;
          fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == args.stages) { stage = 0; phase ^= 1; }
          ready = gptq::bar_poll(empty(stage), phase ^ 1);
          if (leader) {
            const int nb = min(KPS, kb1 - kb);
            if (kb + nb <= args.nfull) {
              // blocks behind the last whole one come as zeros and are not multiplied
              gptq::bar_expect(here, (uint32_t)(KPS * (xb + NW * wb)));
              gptq::load_tile_3d(sw, &maps.w0[0], here, 0, wr, kb);
              if (NW == 2) gptq::load_tile_3d(sw + KPS * wb, &maps.w1[0], here, 0, wr, kb);
              gptq::load_tile_3d(sx, &maps.x[0], here, 0, xr, kb);
            } else {
              gptq::bar_expect(here, (uint32_t)(nb * (xb + NW * wb)));
              for (int b = 0; b < nb; ++b) {
                gptq::load_tile_2d(sw + b * wb, &maps.w0[1], here, (kb + b) * BK, wr);
                if (NW == 2)
                  gptq::load_tile_2d(sw + (KPS + b) * wb, &maps.w1[1], here, (kb + b) * BK, wr);
                gptq::load_tile_2d(sx + b * xb, &maps.x[1], here, (kb + b) * BK, xr);
              }
            }
          }
          __syncwarp();
        }
      }
      if (gptq::flag_read(abort_flag))
        for (int s = 0; s < MAX_STAGES; ++s)
          if (filled & (1u << s)) gptq::bar_drain(full(s), (fill_parity >> s) & 1u);
    } else if (warp == 1) {  // ---------------- MMA issuer ----------------
      const bool leader = gptq::elect_one();
      const uint32_t xb = (uint32_t)(args.x_rows * BK);
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, acc_ready = true, full_ready = false;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1; kb += KPS) {
          if (!bar_wait_rest(acc_ready, acc_empty(buf), acc_phase ^ 1, abort_flag) ||
              !bar_wait_rest(full_ready, full(stage), phase, abort_flag)) {
            ok = false;
            break;
          }
          gptq::tc_fence_after();
          const int nb = min(KPS, kb1 - kb);
          const uint32_t d0 = tmem_base + (uint32_t)(buf * KPS * COLS);
          const uint32_t sx = smem + (uint32_t)(stage * args.stage_bytes), sw = sx + KPS * xb;
          const uint32_t freed = empty(stage), filled = acc_full(buf);
          if (++stage == args.stages) { stage = 0; phase ^= 1; }
          if (++buf == 2) { buf = 0; acc_phase ^= 1; }
          full_ready = gptq::bar_poll(full(stage), phase);
          acc_ready = gptq::bar_poll(acc_empty(buf), acc_phase ^ 1);
          if (leader) {
#pragma unroll
            for (int b = 0; b < KPS; ++b) {
              if (b >= nb) break;
#pragma unroll
              for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)  // 32 columns: 32 bytes along swizzled rows
                  gptq::mma_f8(d0 + (uint32_t)(b * COLS + w * BN),
                               gptq::smem_desc_sw128(sx + b * xb + kk * 32, 16, 1024),
                               gptq::smem_desc_sw128(sw + (w * KPS + b) * BN * BK + kk * 32, 16,
                                                     1024),
                               IDESC, kk > 0);
            }
            gptq::commit_to(freed);
            gptq::commit_to(filled);
          }
          __syncwarp();
        }
      }
      if (gptq::flag_read(abort_flag)) {
        if (leader) gptq::commit_to(mma_drain);
        __syncwarp();
        gptq::bar_drain(mma_drain, 0);
      }
    } else if (warp == 2) {  // ---------------- scales ----------------
      int chunk = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = t0; t < args.n_tiles && ok; t += step) {
        // The weight blocks of the tile: where it spans two, the second one too (of some block,
        // for columns behind the last).
        const int last = (args.N - 1) / 128, b0 = min(col_of(t) / 128, last), b1 = min(b0 + 1, last);
        ok = scales.produce(args.sx, args.ldsx, row_tile(t) * BM, args.x_rows, args.M,
                            args.sw[0] + b0 * args.ldsw[0],
                            NW == 2 ? args.sw[NW - 1] + b0 * args.ldsw[NW - 1]
                                    : args.sw[0] + b1 * args.ldsw[0],
                            kb0, kb1, chunk, phase, abort_flag);
      }
      Scales::drain();
    }
    if constexpr (CLUSTERED) pass_barriers();
  } else {
    // ---------------- epilogue ----------------
    if constexpr (SPLIT_REGS) gptq::regs_inc<224>();
    const int quarter = warp & 3, half = (warp - EPI_WARP0) >> 2;
    const uint32_t lane_field = (uint32_t)(quarter * 32) << 16;
    constexpr int HC = BN / 2;  // columns of a thread, per weight: CH chunks of 16
    int buf = 0, chunk = 0;
    uint32_t acc_phase = 0, tile_parity = 0, chunk_phase = 0;
    bool ok = !gptq::flag_read(skip_flag), acc_ready = false, passed = false;
    for (int t = t0; t < args.n_tiles && ok; t += step) {
      const int row0 = row_tile(t) * BM + quarter * 32, row = row0 + lane;
      const int col0 = col_of(t) + half * HC;
      const bool rows_here = row0 < args.M;  // of the warp
      // The chunks from `cut` on belong to the tile's second weight block.
      const int tile_col = col_of(t);
      const int cut = TWO_BLOCKS ? ((tile_col / 128 + 1) * 128 - col0) / 16 : CH;
      uint64_t acc[NW][CH][8];
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[w][c][e] = 0ull;
      for (int kb = kb0; kb < kb1; kb += KPS) {
        const int nb = min(KPS, kb1 - kb), j = (kb - kb0) % Scales::KC;
        if (j == 0 && !bar_wait(scales.full(chunk), chunk_phase, abort_flag)) {
          ok = false;
          break;
        }
        uint64_t f[KPS][2];  // per block of K: of the tile's two weight blocks (or weights)
        if (rows_here) {
#pragma unroll
          for (int b = 0; b < KPS; ++b) {
            const float sx = scales.row(chunk, j + b, quarter * 32 + lane);
            const float2 sw = scales.blocks(chunk, j + b);
            f[b][0] = gptq::pair2(sx * sw.x);
            if (NW == 2 || TWO_BLOCKS) f[b][1] = gptq::pair2(sx * sw.y);
          }
        }
        if (j + KPS == Scales::KC || kb + KPS >= kb1) {
          __syncwarp();
          if (lane == 0) gptq::bar_arrive(scales.empty(chunk));
          if (++chunk == Scales::CHUNKS) { chunk = 0; chunk_phase ^= 1; }
        }
        if (!bar_wait_rest(acc_ready, acc_full(buf), acc_phase, abort_flag)) {
          ok = false;
          break;
        }
        gptq::tc_fence_after();
        const uint32_t acc_col =
            tmem_base + lane_field + (uint32_t)(buf * KPS * COLS + half * HC);
        const uint32_t freed = acc_empty(buf);
        if (++buf == 2) { buf = 0; acc_phase ^= 1; }
        // The group's chunks of 16 columns, four loads at a time; chunk i is of block i / (NW CH).
        constexpr int CHUNKS = KPS * NW * CH;
        auto column = [&](int i) {
          return acc_col + (uint32_t)(i / (NW * CH) * COLS + i / CH % NW * BN + i % CH * 16);
        };
        auto add = [&](int i, uint32_t(&r)[16]) {
          const int b = i / (NW * CH), w = i / CH % NW, c = i % CH;
          uint64_t fc = f[b][w];
          if constexpr (TWO_BLOCKS) fc = c < cut ? f[b][0] : f[b][1];
          gptq::settled(r);
#pragma unroll
          for (int e = 0; e < 8; ++e) fma2(acc[w][c][e], r[2 * e], r[2 * e + 1], fc);
        };
        auto release = [&] {  // all of it is in registers: the accumulators are free
          gptq::tc_fence_before();
          __syncwarp();
          if (lane == 0) gptq::bar_arrive(freed);
          acc_ready = gptq::bar_poll(acc_full(buf), acc_phase);
        };
        if (!rows_here) {
          release();
        } else if (nb == KPS) {
#pragma unroll
          for (int i = 0; i < CHUNKS; i += 4) {
            uint32_t r[4][16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (i + j < CHUNKS) gptq::tmem_ld_32x32b_x16(column(i + j), r[j]);
            gptq::tmem_ld_wait();
            if (i + 4 >= CHUNKS) release();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (i + j < CHUNKS) add(i + j, r[j]);
          }
        } else {  // the last blocks of K: accumulators behind them hold something else
#pragma unroll
          for (int i = 0; i < CHUNKS; ++i)
            if (i / (NW * CH) < nb) {
              uint32_t r[16];
              gptq::tmem_ld_32x32b_x16(column(i), r);
              gptq::tmem_ld_wait();
              add(i, r);
            }
          release();
        }
      }
      if constexpr (CLUSTERED) ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if constexpr (GROUPED) {
        // Each thread makes h of its own columns; what crosses the cluster is a maximum per row. (The
        // sums themselves through shared memory, a row at a time: 4400 cycles instead of 1500.)
        passed = true;
        const int ks = (int)rank / CN, tid = threadIdx.x - EPI_WARP0 * 32;
        int first = col0;
        gptq::cluster_wait();
        if (args.ksplit == 2) {
          // Two CTAs hold halves of K: the sums of eight columns each for the other's, by way of the
          // operand ring, which is free (all MMAs of the CTA are done).
          const uint32_t slot = smem + (uint32_t)tid * 16;
#pragma unroll
          for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(slot + (w * 2 + e / 2) * 4096),
                           "l"(ks ? acc[w][0][e] : acc[w][0][e + 4]),
                           "l"(ks ? acc[w][0][e + 1] : acc[w][0][e + 5])
                           : "memory");
          gptq::cluster_sync();
#pragma unroll
          for (int w = 0; w < NW; ++w) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float4 p = gptq::ld_cluster(slot + (w * 2 + e / 2) * 4096, rank ^ CN);
              acc[w][0][e] = gptq::add2(ks ? acc[w][0][e + 4] : acc[w][0][e], p.x, p.y);
              acc[w][0][e + 1] = gptq::add2(ks ? acc[w][0][e + 5] : acc[w][0][e + 1], p.z, p.w);
            }
#pragma unroll
            for (int e = 4; e < 8; ++e) acc[w][0][e] = 0ull;
          }
          first += 8 * ks;
        }
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float h0 = gptq::silu_mul(lo2(acc[0][c][e]), lo2(acc[NW - 1][c][e]));
            const float h1 = gptq::silu_mul(hi2(acc[0][c][e]), hi2(acc[NW - 1][c][e]));
            const int col = first + 16 * c + 2 * e;
            if (col < args.N) mx = max(mx, gptq::mag_bits(h0));
            if (col + 1 < args.N) mx = max(mx, gptq::mag_bits(h1));
            asm("mov.b64 %0, {%1, %2};"
                : "=l"(acc[0][c][e])
                : "r"(__float_as_uint(h0)), "r"(__float_as_uint(h1)));
          }
        const uint32_t slot = amax + (uint32_t)(quarter * 32 + lane) * 4;
        for (int r = 0; r < csize; ++r) gptq::max_cluster(slot, (uint32_t)r, mx);
        gptq::cluster_sync();  // behind it a CTA touches its own memory only
        if (row < args.M) {
          float s, inv;
          gptq::block_scale(gptq::flag_read(slot), s, inv);
          if (rank == 0 && half == 0) args.sy[(long long)row * args.ldsy + col_of(t) / 128] = s;
          uint8_t* q = reinterpret_cast<uint8_t*>(args.y) + (long long)row * args.ldy + first;
          const int cols = args.ksplit == 2 ? 8 : 16;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t a = acc[0][c][2 * e], b = acc[0][c][2 * e + 1];
              o[e] = gptq::e4m3x4(lo2(a) * inv, hi2(a) * inv, lo2(b) * inv, hi2(b) * inv);
            }
            const bool whole = first + 16 * c + cols <= args.N && args.y_align >= cols;
            if (whole && cols == 16) {
              *reinterpret_cast<uint4*>(q + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
            } else if (whole) {
              *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (e < cols && first + 16 * c + e < args.N)
                  q[16 * c + e] = (uint8_t)(o[e >> 2] >> ((e & 3) * 8));
            }
          }
        }
      } else if constexpr (CLUSTERED) {
        // Rows are dealt out to the CTAs, each of which gets the parts of its rows side by side in its
        // operand ring. They are sent, not fetched: a load from another CTA takes 900 cycles, and so does
        // the barrier that keeps a CTA until the others have loaded.
        passed = true;
        gptq::cluster_sync();  // all MMAs of all CTAs are done
        const int r = quarter * 32 + lane, ks = args.ksplit;
        if (row < args.M) {
          const uint32_t to = smem + (uint32_t)((r / ks * ks + (int)rank) * PITCH + half * HC) * 4;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            gptq::st_cluster(to + 16 * e, (uint32_t)(r % ks), acc[0][0][2 * e], acc[0][0][2 * e + 1]);
        }
        gptq::cluster_sync();  // behind it a CTA touches its own memory only
        // Eight lanes a row, four columns each; the parts are added up in their order.
        const int rows = min(BM, args.M - row_tile(t) * BM), c4 = (lane & 7) * 4;
        for (int i = (warp - EPI_WARP0) * 4 + (lane >> 3); (int)rank + i * ks < rows; i += 4 * N_EPI) {
          const uint32_t from = smem + (uint32_t)(i * ks * PITCH + c4) * 4;
          float4 p[8], v[NW];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < ks) p[j] = gptq::lds_f32x4(from + j * PITCH * 4);
          v[0] = p[0];
#pragma unroll
          for (int j = 1; j < 8; ++j)
            if (j < ks) {
              v[0].x += p[j].x;
              v[0].y += p[j].y;
              v[0].z += p[j].z;
              v[0].w += p[j].w;
            }
          gptq::store_row4<NW>(v, args.y, (row_tile(t) * BM + (long long)rank + i * ks) * args.ldy,
                               tile_col + c4, args.N, args.y_dtype, args.y_align, nullptr);
        }
      } else if constexpr (NW == 2) {
        // h over the thread's 64 columns; the row's maximum with the warp of the other half.
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float h0 = gptq::silu_mul(lo2(acc[0][c][e]), lo2(acc[NW - 1][c][e]));
            const float h1 = gptq::silu_mul(hi2(acc[0][c][e]), hi2(acc[NW - 1][c][e]));
            const int col = col0 + 16 * c + 2 * e;
            if (col < args.N) mx = max(mx, gptq::mag_bits(h0));
            if (col + 1 < args.N) mx = max(mx, gptq::mag_bits(h1));
            asm("mov.b64 %0, {%1, %2};"
                : "=l"(acc[0][c][e])
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
        if (row < args.M) {
          float s, inv;
          gptq::block_scale(mx, s, inv);
          if (half == 0) args.sy[(long long)row * args.ldsy + col0 / 128] = s;
          uint8_t* q = reinterpret_cast<uint8_t*>(args.y) + (long long)row * args.ldy + col0;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t a = acc[0][c][2 * e], b = acc[0][c][2 * e + 1];
              o[e] = gptq::e4m3x4(lo2(a) * inv, hi2(a) * inv, lo2(b) * inv, hi2(b) * inv);
            }
            if (args.y_align == 16 && col0 + 16 * c + 16 <= args.N) {
              *reinterpret_cast<uint4*>(q + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (col0 + 16 * c + e < args.N) q[16 * c + e] = (uint8_t)(o[e >> 2] >> ((e & 3) * 8));
            }
          }
        }
      } else if (args.y_align < 16) {
        if (rows_here) {
          const uint32_t st = out_stage + (uint32_t)(warp - EPI_WARP0) * STAGE_OUT;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (args.y_dtype == GPTQ_F32) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                store_rows<4>(args, st, row0, col0 + 16 * c + 8 * h, lane,
                              [&](int i) { return (uint32_t)(acc[0][c][4 * h + i / 2] >> (i % 2 * 32)); });
            } else {
              store_rows<2>(args, st, row0, col0 + 16 * c, lane, [&](int i) {
                return gptq::pack2(lo2(acc[0][c][i]), hi2(acc[0][c][i]), args.y_dtype);
              });
            }
          }
        }
      } else if (row < args.M) {
        // 32 or 64 bytes of the row per chunk: whole sectors
        const long long at = (long long)row * args.ldy + col0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const bool vec = col0 + 16 * c + 16 <= args.N;
          if (vec && args.y_dtype == GPTQ_F32) {
            float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(args.y) + at + 16 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = make_float4(lo2(acc[0][c][2 * e]), hi2(acc[0][c][2 * e]),
                                 lo2(acc[0][c][2 * e + 1]), hi2(acc[0][c][2 * e + 1]));
          } else if (vec) {
            uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(args.y) + at + 16 * c);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[i] = gptq::pack2(lo2(acc[0][c][4 * e + i]), hi2(acc[0][c][4 * e + i]),
                                   args.y_dtype);
              p[e] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (col0 + 16 * c + e < args.N)
                gptq::store_out(args.y, at + 16 * c + e,
                                e & 1 ? hi2(acc[0][c][e >> 1]) : lo2(acc[0][c][e >> 1]),
                                args.y_dtype);
          }
        }
      }
    }
    if constexpr (CLUSTERED)
      if (!passed) pass_barriers();
  }

  gptq::tc_fence_before();
  __syncthreads();
  if (warp == 1) gptq::tmem_dealloc(tmem_base, TMEM_COLS);
  if (threadIdx.x == 0 && gptq::flag_read(abort_flag)) gptq::set_status(args.status, GPTQ_ERR_TIMEOUT, 6);
}

// Both maps of one operand: boxes of `rows` rows by 128 bytes, and by kps whole blocks of 128.
int operand_maps(CUtensorMap (&map)[2], const uint8_t* p, int rows_total, int k, long long ld,
                 int rows, int kps) {
  const int nfull = k / BK;
  if (k % BK != 0) {
    if (gptq_host::make_tmap_2d(&map[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p, (uint64_t)k,
                                (uint64_t)rows_total, (uint64_t)ld, BK, (uint32_t)rows,
                                CU_TENSOR_MAP_SWIZZLE_128B) != 0)
      return -1;
  }
  if (nfull > 0) {
    if (gptq_host::make_tmap_blocks(&map[0], p, (uint64_t)rows_total, (uint64_t)ld,
                                    (uint64_t)nfull, (uint32_t)rows, (uint32_t)kps) != 0)
      return -1;
  } else {
    map[0] = map[1];
  }
  if (k % BK == 0) map[1] = map[0];
  return 0;
}

template <int NW, int CH, bool CLUSTERED>
int launch(const gptq_host::Fp8Gemm& g, ThinArgs a, int sms, cudaStream_t stream) {
  constexpr int BN = 32 * CH, COLS = NW * BN;
  constexpr int KPS = COLS <= 64 ? 4 : COLS <= 128 ? 2 : 1;
  constexpr int CN = NW == 2 ? 128 / BN : 1;
  const int tiles_m = (g.m + BM - 1) / BM;
  a.tiles_n = (g.n + CN * BN - 1) / (CN * BN);
  a.kq = (a.nkb + KPS - 1) / KPS / a.ksplit;
  a.kr = (a.nkb + KPS - 1) / KPS % a.ksplit;
  if ((long long)tiles_m * a.tiles_n > 0x3FFFFFFF) return GPTQ_ERR_CUDA;
  a.n_tiles = tiles_m * a.tiles_n;
  a.stage_bytes = KPS * (a.x_rows + NW * BN) * BK;
  a.stages = RING_BYTES / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  Maps maps;
  if (operand_maps(maps.x, g.x, g.m, g.k, g.ldx, a.x_rows, KPS) != 0 ||
      operand_maps(maps.w0, g.w[0], g.n, g.k, g.ldw[0], BN, KPS) != 0)
    return GPTQ_ERR_CUDA;
  if (NW == 2) {
    if (operand_maps(maps.w1, g.w[1], g.n, g.k, g.ldw[1], BN, KPS) != 0) return GPTQ_ERR_CUDA;
  } else {
    maps.w1[0] = maps.w1[1] = maps.w0[0];
  }
  const int csize = CLUSTERED ? CN * a.ksplit : 1;
  const int grid = CLUSTERED ? a.n_tiles * csize : a.n_tiles < sms ? a.n_tiles : sms;
  return gptq_host::fp8_launch(fp8_thin_kernel<NW, CH, CLUSTERED>, grid, THREADS, SMEM_BYTES, csize,
                               stream, maps, a);
}

}  // namespace

namespace gptq_host {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode_fn();  // host_util.cu

int make_tmap_blocks(CUtensorMap* map, const uint8_t* base, uint64_t rows, uint64_t ld,
                     uint64_t blocks, uint32_t box_rows, uint32_t box_blocks) {
  auto fn = tensor_map_encode_fn();
  if (fn == nullptr) return -1;
  cuuint64_t dims[3] = {128, rows, blocks};
  cuuint64_t strides[2] = {ld, 128};
  cuuint32_t box[3] = {128, box_rows, box_blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? 0
             : -1;
}

// Time of a block of K with CTAs of 32 ch weight rows, all rounds, in units of 1.7 ns: a round has a
// fixed part (4096 x 4096 with 32 rows: 0.18 us) and one for its rows (512 x 4096 x 4096 with
// 128: 0.34 us).
static long long tile_cost(const Fp8Gemm& g, int ch, int sms) {
  const long long tiles = (long long)((g.m + BM - 1) / BM) * ((g.n + 32 * ch - 1) / (32 * ch));
  return (tiles + sms - 1) / sms * (75 + 32 * ch);
}
// The tile of the plain product that needs the least time.
static int plain_tile(const Fp8Gemm& g, int sms) {
  int best = 1;
  for (int ch = 2; ch <= 4; ++ch)
    if (tile_cost(g, ch, sms) < tile_cost(g, best, sms)) best = ch;
  return best;
}

// Clusters of `size` CTAs, one CTA an SM, that the device holds at once.
static int resident(int size) {
  return resident_clusters(THREADS, SMEM_BYTES, size);
}

long long fp8_thin_cost(const Fp8Gemm& g) {
  const int sms = num_sms();
  if (g.w[1] == nullptr) return tile_cost(g, plain_tile(g, sms), sms);
  // Gated pair: 32 or 64 rows of each weight where clusters hold all groups (100 x 4096 x 4096: 13.1 us, a
  // block 0.33), else 128 (100 x 11008 x 4096: 24.5 us, a block 0.6).
  const long long groups = (long long)((g.m + BM - 1) / BM) * ((g.n + 127) / 128);
  if (groups <= resident(4)) return 195;
  if (groups <= resident(2)) return 300;
  return (groups + sms - 1) / sms * 355;
}

int fp8_thin(const Fp8Gemm& g, cudaStream_t stream) {
  const bool gated = g.w[1] != nullptr;
  const int sms = num_sms();
  ThinArgs a{};
  a.M = g.m; a.N = g.n;
  a.nkb = (g.k + BK - 1) / BK;
  a.nfull = g.k / BK;
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
  // Rows of X that a tile can hold: a call of few rows brings only those (whole groups of the
  // swizzle's eight rows); what the MMA reads behind them feeds accumulator rows nobody reads.
  a.x_rows = g.m >= BM ? BM : (g.m + 7) / 8 * 8;
  a.ksplit = 1;
  const long long tiles_m = (g.m + BM - 1) / BM;
  auto tiles = [&](int cols) { return tiles_m * ((g.n + cols - 1) / cols); };
  // Clusters are used where they are all resident at once: of one CTA an SM, that is fewer than the
  // SMs divided by their size (15 of eight, not 18).
  if (gated) {
    const long long groups = tiles(128);
    if (groups <= resident(4)) {
      if (groups <= resident(8) && a.nkb >= 16) a.ksplit = 2;  // two stages of four blocks each
      return launch<2, 1, true>(g, a, sms, stream);
    }
    if (groups <= resident(2)) return launch<2, 2, true>(g, a, sms, stream);
    return launch<2, 4, false>(g, a, sms, stream);
  }
  for (int s = 8; s >= 2; --s)
    if (a.nkb >= 8 * s && tiles(32) <= resident(s)) {
      a.ksplit = s;
      return launch<1, 1, true>(g, a, sms, stream);
    }
  switch (plain_tile(g, sms)) {
    case 1: return launch<1, 1, false>(g, a, sms, stream);
    case 2: return launch<1, 2, false>(g, a, sms, stream);
    case 3: return launch<1, 3, false>(g, a, sms, stream);
    default: return launch<1, 4, false>(g, a, sms, stream);
  }
}

}  // namespace gptq_host
