// fp8_skinny.cu — the products of the e4m3 format for few rows of activations (decoding), where the time
// is that of streaming the weight: up to 32 rows, in the gated pair up to 64.
//
// The operands change places: the 128 rows of a weight block are the M of the MMAs (lanes of tensor
// memory), the activation rows their N. A thread of the epilogue then owns one weight row and reads
// one column per activation row, so all lanes work however few rows there are: with the
// activations as M, one warp in four did, and a gated pair's block of 128 columns took it 2000
// cycles.
//
// A cluster owns the 128 weight rows of a scale block (gated pair: of both weights); its CTAs share
// out the blocks of K. The sums of a block are scaled by sx sw in fp32 registers as in fp8_gemm.cu.
// At the end the CTAs send one another their sums, each row of the output tile to one of them, where a
// warp adds them up, always in the same order; for the gated pair it also has the whole 128
// columns of the row's scale.
// Two CTAs share an SM, so that one's start and end pass behind the other's stream.
// Measured (B200, weights larger than L2 in a graph of calls): 1 x 8192 x 28672 in 38.7 us (6.1 TB/s, 0.94
// of the measured copy rate), 8 x 11008 x 4096 gated in 18.0 us (5.0 TB/s), 16 x 11008 x 4096 in 10.4 us
// (what a loop that only streams this weight takes), 1 x 4096 x 4096 in 6.0 us, of which more than 3 are
// the kernel's start, the latency of its first load and the cluster's exchange (weights in L2: 5.4).
// Further from their floors: 32 x 11008 x 4096 in 11.1 us (floor 7.1; four stages, with 16 rows five), gated 64 x
// 11008 x 4096 in 21.5 us and 32 x 11008 x 4096 in 21.0 (floor 14.1). The last, Cfg<2, 32>, is the poorest
// variant: two stages, a third 1280 bytes short of the shared memory, and 16 bytes of registers spilled.
// Warps: 0 TMA producer, 1 TMEM owner and MMA issuer, 2 scales, 4-7 epilogue (gated pair: 8-11 the
// second weight's). Every wait is bounded as in fp8_gemm.cu.
#include "fp8_exchange.cuh"
#include "fp8_mma.cuh"

namespace {

using gptq::bar_wait;
using gptq::bar_wait_rest;

constexpr int BM = 128, BK = 128;
constexpr int W_TILE = BM * BK;  // 16 KB
constexpr int EPI_WARP0 = 4;

template <int NW, int MT>
struct Cfg {
  using Scales = gptq::ScaleRing<(MT > 32 ? MT : 32)>;
  static constexpr int THREADS = 128 + 128 * NW;
  // Two, but for the gated pair of 64 rows, whose 64 sums a thread of 384 take the registers of one.
  static constexpr int CTAS_PER_SM = NW * MT > 64 ? 1 : 2;
  static constexpr int NBUF = 4;  // accumulators
  static constexpr int STAGE_BYTES = NW * W_TILE + MT * BK;
  // Where the cluster's sums arrive: the CTA's share of the rows times the CTAs. The plain product has room
  // for it beside the ring, the gated pair uses the ring again.
  static constexpr bool APART = NW == 1;
  static constexpr int SUMS = gptq::exchange_rows(MT) * NW * BM * 4, RECV = APART ? SUMS : 0;
  static constexpr int STAGES = 
      (228 * 1024 / CTAS_PER_SM - 1024 - 1024 - 512 - RECV - Scales::BYTES) / STAGE_BYTES;
  static constexpr int RING = STAGES * STAGE_BYTES;
  static constexpr int SMEM = RING + RECV + Scales::BYTES + 512 + 1024;
  static constexpr uint32_t TMEM_COLS = NBUF * NW * MT;  // 64 to 512
  static_assert(CTAS_PER_SM * (SMEM + 1024) <= 228 * 1024 && STAGES >= 2, "shared memory");
  static_assert(CTAS_PER_SM * TMEM_COLS <= 512, "tensor memory");
  static_assert(APART || SUMS <= RING, "sums");
};

struct SkinnyArgs {
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
  int ksplit;   // CTAs of a cluster, which have kq blocks of K each, the first kr one more
  int kq, kr;
  int32_t* status;
};

template <int NW, int MT>
__global__ void __launch_bounds__(Cfg<NW, MT>::THREADS, Cfg<NW, MT>::CTAS_PER_SM)
fp8_skinny_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW0,
                  const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ SkinnyArgs args) {
  using C = Cfg<NW, MT>;
  using Scales = typename C::Scales;
  constexpr int NBUF = C::NBUF;
  constexpr uint32_t IDESC = gptq::instr_desc(/*e4m3*/ 0, 0, 0, BM, MT);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = (gptq::smem_u32(smem_raw) + 1023u) & ~1023u;
  Scales scales;
  const uint32_t recv = C::APART ? smem + C::RING : smem;
  scales.buf = smem + C::RING + C::RECV;
  const uint32_t bars = scales.buf + Scales::BYTES;
  auto full = [&](int s) { return bars + (uint32_t)s * 8; };
  auto empty = [&](int s) { return bars + (uint32_t)(C::STAGES + s) * 8; };
  auto acc_full = [&](int b) { return bars + (uint32_t)(2 * C::STAGES + b) * 8; };
  auto acc_empty = [&](int b) { return bars + (uint32_t)(2 * C::STAGES + NBUF + b) * 8; };
  const uint32_t mma_drain = bars + (2 * C::STAGES + 2 * NBUF) * 8;
  scales.bars = mma_drain + 8;
  const uint32_t tmem_slot = scales.bars + Scales::BAR_BYTES;
  const uint32_t abort_flag = tmem_slot + 4, skip_flag = tmem_slot + 8;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t rank, cluster_id;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %clusterid.x;" : "=r"(cluster_id));

  if constexpr (C::APART) gptq::cluster_arrive();  // the CTA has started
  if (threadIdx.x == 0) {
    gptq::flag_write(abort_flag, 0);
    for (int s = 0; s < C::STAGES; ++s) {
      gptq::bar_init(full(s), 1);
      gptq::bar_init(empty(s), 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      gptq::bar_init(acc_full(b), 1);
      gptq::bar_init(acc_empty(b), 4 * NW);
    }
    scales.init(4 * NW);
    gptq::bar_init(mma_drain, 1);
    gptq::fence_barrier_init();
  } else if (threadIdx.x == 32 * 3) {
    gptq::tma_prefetch_desc(&tmX);
    gptq::tma_prefetch_desc(&tmW0);
    if (NW == 2) gptq::tma_prefetch_desc(&tmW1);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot),
                 "r"(C::TMEM_COLS)
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
  const bool skip = gptq::flag_read(skip_flag) != 0;
  // The cluster's block of 128 weight rows (no division: it would stand between the CTA and its first load).
  const int block = (int)cluster_id;
  const int kb0 = (int)rank * args.kq + min((int)rank, args.kr);
  const int kb1 = kb0 + args.kq + ((int)rank < args.kr ? 1 : 0);

  // Every thread of every CTA of the cluster passes this barrier and the next, whatever happens to it.
  auto ready_to_receive = [&] {
    if constexpr (C::APART)
      gptq::cluster_wait();  // all CTAs have started
    else
      gptq::cluster_sync();  // all MMAs of all CTAs are done
  };

  if (warp < EPI_WARP0) {
    if (skip) {
    } else if (warp == 0) {  // ---------------- TMA producer ----------------
      const bool leader = gptq::elect_one();
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_parity = 0;
      bool ready = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!bar_wait_rest(ready, empty(stage), phase ^ 1, abort_flag)) break;
        const uint32_t sw = smem + (uint32_t)(stage * C::STAGE_BYTES), here = full(stage);
        filled |= 1u << stage;
        fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        ready = gptq::bar_poll(empty(stage), phase ^ 1);
        if (leader) {
          gptq::bar_expect(here, C::STAGE_BYTES);
          gptq::load_tile_2d(sw, &tmW0, here, kb * BK, block * BM);
          if (NW == 2) gptq::load_tile_2d(sw + W_TILE, &tmW1, here, kb * BK, block * BM);
          gptq::load_tile_2d(sw + NW * W_TILE, &tmX, here, kb * BK, 0);
        }
        __syncwarp();
      }
      if (gptq::flag_read(abort_flag))
        for (int s = 0; s < C::STAGES; ++s)
          if (filled & (1u << s)) gptq::bar_drain(full(s), (fill_parity >> s) & 1u);
    } else if (warp == 1) {  // ---------------- MMA issuer ----------------
      const bool leader = gptq::elect_one();
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool acc_ready = true, full_ready = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!bar_wait_rest(acc_ready, acc_empty(buf), acc_phase ^ 1, abort_flag) ||
            !bar_wait_rest(full_ready, full(stage), phase, abort_flag))
          break;
        gptq::tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(buf * NW * MT);
        const uint32_t sw = smem + (uint32_t)(stage * C::STAGE_BYTES), sx = sw + NW * W_TILE;
        const uint32_t freed = empty(stage), filled = acc_full(buf);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        if (++buf == NBUF) { buf = 0; acc_phase ^= 1; }
        full_ready = gptq::bar_poll(full(stage), phase);
        acc_ready = gptq::bar_poll(acc_empty(buf), acc_phase ^ 1);
        if (leader) {
#pragma unroll
          for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)  // 32 columns: 32 bytes along the swizzled rows
              gptq::mma_f8(d + (uint32_t)(w * MT),
                           gptq::smem_desc_sw128(sw + w * W_TILE + kk * 32, 16, 1024),
                           gptq::smem_desc_sw128(sx + kk * 32, 16, 1024), IDESC, kk > 0);
          gptq::commit_to(freed);
          gptq::commit_to(filled);
        }
        __syncwarp();
      }
      if (gptq::flag_read(abort_flag)) {
        if (leader) gptq::commit_to(mma_drain);
        __syncwarp();
        gptq::bar_drain(mma_drain, 0);
      }
    } else if (warp == 2) {  // ---------------- scales ----------------
      int chunk = 0;
      uint32_t phase = 0;
      scales.produce(args.sx, args.ldsx, 0, MT, args.M, args.sw[0] + block * args.ldsw[0],
                     args.sw[NW - 1] + block * args.ldsw[NW - 1], kb0, kb1, chunk, phase,
                     abort_flag);
      Scales::drain();
    }
    ready_to_receive();
    gptq::cluster_sync();
  } else {
    // ---------------- epilogue: one weight row a thread ----------------
    const int quarter = warp & 3, w = (warp - EPI_WARP0) >> 2;
    const uint32_t acc_col = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(w * MT);
    int buf = 0, chunk = 0;
    uint32_t acc_phase = 0, chunk_phase = 0;
    bool ok = !skip, acc_ready = false;
    uint64_t acc[MT / 2];
#pragma unroll
    for (int c = 0; c < MT / 2; ++c) acc[c] = 0ull;
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      const int j = (kb - kb0) % Scales::KC;
      if ((j == 0 && !bar_wait(scales.full(chunk), chunk_phase, abort_flag)) ||
          !bar_wait_rest(acc_ready, acc_full(buf), acc_phase, abort_flag)) {
        ok = false;
        break;
      }
      gptq::tc_fence_after();
      const float2 sw2 = scales.blocks(chunk, j);
      const uint64_t sw = gptq::pair2(NW == 2 && w ? sw2.y : sw2.x);
      // Sixteen columns (activation rows) a load, two loads at a time.
      const uint32_t col = acc_col + (uint32_t)(buf * NW * MT), freed = acc_empty(buf);
      if (++buf == NBUF) { buf = 0; acc_phase ^= 1; }
#pragma unroll
      for (int c0 = 0; c0 < MT / 16; c0 += 2) {
        uint32_t r[2][16];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (c0 + i < MT / 16) gptq::tmem_ld_32x32b_x16(col + (uint32_t)(16 * (c0 + i)), r[i]);
        gptq::tmem_ld_wait();
        if (c0 + 2 >= MT / 16) {  // all of it is in registers: the accumulator is free
          gptq::tc_fence_before();
          __syncwarp();
          if (lane == 0) gptq::bar_arrive(freed);
          acc_ready = gptq::bar_poll(acc_full(buf), acc_phase);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = c0 + i;
          if (c >= MT / 16) break;
          gptq::settled(r[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 sx = scales.rows4(chunk, j, 16 * c + 4 * e);
            uint64_t* a = acc + 8 * c + 2 * e;
            gptq::fma2(a[0], r[i][4 * e], r[i][4 * e + 1], gptq::mul2(sx.x, sx.y, sw));
            gptq::fma2(a[1], r[i][4 * e + 2], r[i][4 * e + 3], gptq::mul2(sx.z, sx.w, sw));
          }
        }
      }
      if (j == Scales::KC - 1) {
        __syncwarp();
        if (lane == 0) gptq::bar_arrive(scales.empty(chunk));
        if (++chunk == Scales::CHUNKS) { chunk = 0; chunk_phase ^= 1; }
      }
    }
    // Rows are dealt out to the CTAs, each of which gets ksplit sums of its rows, side by side. They are
    // sent and not fetched: a load from another CTA takes 900 cycles, and so does the barrier that
    // keeps a CTA until the others have loaded (1 x 2048 x 4096: 5.55 us so, 4.5 sent).
    ready_to_receive();
    const uint32_t mine = recv + (rank * NW + w) * (BM * 4) + (uint32_t)(quarter * 32 + lane) * 4;
    auto sum = [&](int c) { return c & 1 ? gptq::hi2(acc[c / 2]) : gptq::lo2(acc[c / 2]); };
    if (ok && args.ksplit == 1) {
#pragma unroll
      for (int c = 0; c < MT; ++c)
        if (c < args.M)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + c * (NW * BM * 4)), "f"(sum(c)) : "memory");
    } else if (ok) {
      uint32_t at = mine;
      int to = 0;
#pragma unroll
      for (int c = 0; c < MT; ++c)
        if (c < args.M) {
          gptq::st_cluster(at, (uint32_t)to, sum(c));
          if (++to == args.ksplit) {
            to = 0;
            at += (uint32_t)(NW * BM * 4) * args.ksplit;
          }
        }
    }
    gptq::cluster_sync();  // behind it a CTA touches its own memory only
    // A warp a row, four columns a lane; the parts of K are added up in their order.
    for (int i = warp - EPI_WARP0; !skip; i += 4 * NW) {
      const int r = (int)rank + i * args.ksplit;
      if (r >= args.M) break;
      const uint32_t from = recv + (uint32_t)(i * args.ksplit * NW * BM + lane * 4) * 4;
      float4 p[gptq::kMaxSplit][NW];
#pragma unroll
      for (int s = 0; s < gptq::kMaxSplit; ++s)
        if (s < args.ksplit) {
#pragma unroll
          for (int j = 0; j < NW; ++j) p[s][j] = gptq::lds_f32x4(from + (s * NW + j) * (BM * 4));
        }
#pragma unroll
      for (int s = 1; s < gptq::kMaxSplit; ++s)
        if (s < args.ksplit) {
#pragma unroll
          for (int j = 0; j < NW; ++j) {
            p[0][j].x += p[s][j].x;
            p[0][j].y += p[s][j].y;
            p[0][j].z += p[s][j].z;
            p[0][j].w += p[s][j].w;
          }
        }
      gptq::store_row4<NW>(p[0], args.y, (long long)r * args.ldy, block * 128 + lane * 4, args.N,
                           args.y_dtype, args.y_align,
                           args.sy + (NW == 2 ? (long long)r * args.ldsy + block : 0));
    }
  }

  gptq::tc_fence_before();
  __syncthreads();
  if (warp == 1) gptq::tmem_dealloc(tmem_base, C::TMEM_COLS);
  if (threadIdx.x == 0 && gptq::flag_read(abort_flag))
    gptq::set_status(args.status, GPTQ_ERR_TIMEOUT, 7);
}

template <int NW, int MT>
int launch(const gptq_host::Fp8Gemm& g, const SkinnyArgs& a, int blocks, cudaStream_t stream) {
  using C = Cfg<NW, MT>;
  using gptq_host::make_tmap_2d;
  CUtensorMap tx, tw[2];
  if (make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.x, (uint64_t)g.k, (uint64_t)g.m,
                   (uint64_t)g.ldx, BK, MT, CU_TENSOR_MAP_SWIZZLE_128B) != 0)
    return GPTQ_ERR_CUDA;
  for (int i = 0; i < NW; ++i)
    if (make_tmap_2d(&tw[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.w[i], (uint64_t)g.k, (uint64_t)g.n,
                     (uint64_t)g.ldw[i], BK, BM, CU_TENSOR_MAP_SWIZZLE_128B) != 0)
      return GPTQ_ERR_CUDA;
  return gptq_host::fp8_launch(fp8_skinny_kernel<NW, MT>, (long long)blocks * a.ksplit, C::THREADS,
                               C::SMEM, a.ksplit, stream, tx, tw[0], tw[NW - 1], a);
}

}  // namespace

namespace gptq_host {

// Measured on both sides (us, this kernel / fp8_thin): plain 32 x 11008 x 4096 12.0 / 12.3, 64 x 11008 x
// 4096 13.3 / 12.0, 64 x 4096 x 4096 10.1 / 7.8; gated 64 x 11008 x 4096 21.4 / 23.4, 64 x 4096 x 4096
// 12.0 / 13.2, 34 x 8576 x 1024 8.7 / 10.5, 64 x 256 x 4096 7.1 / 8.4, but 64 x 1024 x 1024 6.8 / 5.7,
// where K is short and fp8_thin's clusters are all resident.
bool fp8_skinny_takes(const Fp8Gemm& g) {
  if (g.m <= 32 || g.w[1] == nullptr) return g.m <= 32;
  const long long groups = (g.n + BM - 1) / BM;
  return g.m <= 64 && (g.k > 8 * BK || 4 * groups > num_sms());
}

int fp8_skinny(const Fp8Gemm& g, cudaStream_t stream) {
  const bool gated = g.w[1] != nullptr;
  SkinnyArgs a{};
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
  const int blocks = (g.n + BM - 1) / BM;
  // As many CTAs along K as clusters of them are resident at once, each with four blocks of K at least;
  // large clusters with room to spare, since the last ones start late (1 x 4096 x 4096 in 32 clusters
  // of 8 of the 33 there are: 6.8 us, of 7: 6.3, of 6: 6.0; 1 x 8192 x 8192 in 64 of 4 of 71: 14.2, of 3:
  // 13.4; but 16 x 11008 x 4096 in 86 of 3: 10.3, of 2: 11.6; gated 1 x 4096 x 4096 of 7: 9.5, of 6: 9.8).
  auto run = [&](auto launch, int threads, int smem) {
    a.ksplit = a.nkb >= 4 * gptq::kMaxSplit ? gptq::kMaxSplit : a.nkb >= 8 ? a.nkb / 4 : 1;
    auto fits = [&](int s) {
      return blocks + (s > 3 ? blocks / (gated ? 8 : 4) : 0) <= resident_clusters(threads, smem, s);
    };
    while (a.ksplit > 1 && !fits(a.ksplit)) --a.ksplit;
    a.kq = a.nkb / a.ksplit;
    a.kr = a.nkb % a.ksplit;
    return launch(g, a, blocks, stream);
  };
#define FP8_SKINNY(NW, MT) run(launch<NW, MT>, Cfg<NW, MT>::THREADS, Cfg<NW, MT>::SMEM)
  if (gated) return g.m <= 16 ? FP8_SKINNY(2, 16) : g.m <= 32 ? FP8_SKINNY(2, 32) : FP8_SKINNY(2, 64);
  return g.m <= 16 ? FP8_SKINNY(1, 16) : FP8_SKINNY(1, 32);
#undef FP8_SKINNY
}

}  // namespace gptq_host
