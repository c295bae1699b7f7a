// fp8_mma.cuh — what the tensor-core kernels of the e4m3 format share.
#pragma once

#include "fp8.cuh"

namespace gptq {

// D[tmem] (+)= A[smem] B[smem], kind::f8f6f4 (e4m3 operands, fp32 accumulate), 32 columns of K.
GPTQ_DEV void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Waits for the loads from tensor memory issued so far; `settled` names their registers, so that no
// use of them is scheduled before the wait.
template <int N>
GPTQ_DEV void settled(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Barriers, flags and tiles in shared memory by their 32-bit addresses: the epilogue threads hold
// 128 sums and have no registers for 64-bit pointers (as generic pointers they cost four reloads
// from local memory in every block of K).
GPTQ_DEV void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
GPTQ_DEV void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
GPTQ_DEV void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
GPTQ_DEV bool bar_try(uint32_t bar, uint32_t parity) {  // may sleep for a while
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
GPTQ_DEV bool bar_poll(uint32_t bar, uint32_t parity) {  // returns at once
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
GPTQ_DEV uint32_t flag_read(uint32_t flag) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(flag) : "memory");
  return v;
}
GPTQ_DEV void flag_write(uint32_t flag, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(flag), "r"(v) : "memory");
}
// Wait for the phase of the given parity, with the limit of mbar_wait: false (and the abort flag
// raised) if it ran out or another thread gave up. The barrier alone is polled at first: reading
// the timer and the flag after every poll, as mbar_wait does, made a pipeline step of a streaming
// kernel 250 cycles longer.
GPTQ_DEV bool bar_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (bar_try(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!bar_try(bar, parity)) {
    if (flag_read(abort)) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      flag_write(abort, 1);
      return false;
    }
  }
  return true;
}
// bar_wait whose first poll was made earlier (`ready`), so that its latency passed behind other work.
GPTQ_DEV bool bar_wait_rest(bool ready, uint32_t bar, uint32_t parity, uint32_t abort) {
  return ready || bar_wait(bar, parity, abort);
}
// mbar_drain by address: on the way out after an abort, wait for what was already issued.
GPTQ_DEV bool bar_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!bar_try(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}
GPTQ_DEV void load_tile_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
GPTQ_DEV void load_tile_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
GPTQ_DEV void commit_to(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
GPTQ_DEV float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
GPTQ_DEV float2 lds_f32x2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

GPTQ_DEV float4 lds_f32x4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// One lane of the warp, the same one each time. The loops that issue MMAs and loads are run by
// whole warps, with only the instructions themselves under this predicate: in a branch of one lane
// the compiler cannot keep descriptors and addresses in uniform registers, and a block of K
// then cost the issuing thread 940 cycles instead of 590 (four MMAs, two waits, two commits;
// 520 with the next waits polled ahead; the MMAs themselves take 512).
GPTQ_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The scales of a tile's 128 rows and of its (up to) two weight blocks, on their way to the epilogue
// through shared memory, in chunks of eight blocks of K. Loads by the epilogue itself arrive
// too late, however early within a step they are issued: they queue behind the operand tiles that the ring
// has in flight (192 KB, 2500 cycles at 8192 x 8192 x 28672). One warp copies the
// chunks with cp.async, several of them ahead.
// ROWS (a multiple of 32) is the number of rows a chunk has room for.
template <int ROWS>
struct ScaleRing {
  static constexpr int CHUNKS = 4, KC = 8;
  static constexpr int PITCH = ROWS + 4;  // floats between blocks of K: 8 x 4 copies hit 32 banks
  static constexpr int FLOATS = KC * PITCH + KC * 2;
  static constexpr int BYTES = CHUNKS * FLOATS * 4;
  static constexpr int BAR_BYTES = 2 * CHUNKS * 8;
  uint32_t buf, bars;  // shared-memory addresses: the chunks; CHUNKS full barriers, then CHUNKS empty

  GPTQ_DEV uint32_t full(int c) const { return bars + c * 8; }
  GPTQ_DEV uint32_t empty(int c) const { return bars + (CHUNKS + c) * 8; }
  GPTQ_DEV void init(int consumers) const {  // one thread
    for (int c = 0; c < CHUNKS; ++c) {
      bar_init(full(c), 32);
      bar_init(empty(c), consumers);
    }
  }
  // Producer, a whole warp: blocks [kb0, kb1) of K for the `rows` rows from row0 on (rows past m - 1
  // repeat it) and the weight blocks whose scales start at sw0 and sw1. False if a wait gave up.
  GPTQ_DEV bool produce(const float* sx, long long ldsx, int row0, int rows, int m,
                        const float* sw0, const float* sw1, int kb0, int kb1, int& chunk,
                        uint32_t& phase, uint32_t abort) const {
    const int lane = threadIdx.x & 31, j = lane & 7;
    for (int kb = kb0; kb < kb1; kb += KC) {
      if (!bar_wait(empty(chunk), phase ^ 1, abort)) return false;
      const int k = min(kb + j, kb1 - 1);
      const uint32_t dst = buf + chunk * (FLOATS * 4);
      for (int r = lane >> 3; r < rows; r += 4)
        copy(dst + (uint32_t)(j * PITCH + r) * 4, sx + (long long)min(row0 + r, m - 1) * ldsx + k);
      if (lane < 16)
        copy(dst + (uint32_t)(KC * PITCH + j * 2 + (lane >> 3)) * 4, (lane < 8 ? sw0 : sw1) + k);
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full(chunk))
                   : "memory");
      if (++chunk == CHUNKS) { chunk = 0; phase ^= 1; }
    }
    return true;
  }
  GPTQ_DEV static void drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
  GPTQ_DEV static void copy(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
  }
  // Consumer: scale of a row of the tile, and of the two weight blocks, at block j of the chunk.
  GPTQ_DEV float row(int chunk, int j, int r) const {
    return lds_f32(buf + (uint32_t)(chunk * FLOATS + j * PITCH + r) * 4);
  }
  GPTQ_DEV float4 rows4(int chunk, int j, int r) const {  // of rows r .. r + 3, r a multiple of 4
    return lds_f32x4(buf + (uint32_t)(chunk * FLOATS + j * PITCH + r) * 4);
  }
  GPTQ_DEV float2 blocks(int chunk, int j) const {
    return lds_f32x2(buf + (uint32_t)(chunk * FLOATS + KC * PITCH + j * 2) * 4);
  }
};

// Two fp32 fused multiply-adds in one instruction: acc += d * f.
GPTQ_DEV void fma2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t f2) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(f2));
}
GPTQ_DEV uint64_t pair2(float f) {
  uint64_t r;
  const uint32_t b = __float_as_uint(f);
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(b));
  return r;
}
GPTQ_DEV uint64_t mul2(float a, float b, uint64_t f2) {  // (a, b) * f
  uint64_t v, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(v), "l"(f2));
  return r;
}
GPTQ_DEV uint64_t add2(uint64_t v, float a, float b) {  // v + (a, b)
  uint64_t p, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(v), "l"(p));
  return r;
}
GPTQ_DEV float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
GPTQ_DEV float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

template <int N>
GPTQ_DEV void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
GPTQ_DEV void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

GPTQ_DEV void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
GPTQ_DEV void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
GPTQ_DEV void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// The maximum with a word in the shared memory of a CTA of the cluster.
GPTQ_DEV void max_cluster(uint32_t saddr, uint32_t rank, uint32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
GPTQ_DEV void st_cluster(uint32_t saddr, uint32_t rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
GPTQ_DEV void st_cluster(uint32_t saddr, uint32_t rank, uint64_t v0, uint64_t v1) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(a), "l"(v0), "l"(v1) : "memory");
}
GPTQ_DEV float4 ld_cluster(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

GPTQ_DEV uint32_t pack2(float a, float b, int dtype) {
  if (dtype == GPTQ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four consecutive columns of an output row from their sums: v[0] as it is in the type of Y (NW = 1),
// or h = silu(v[0]) v[1] in the format (NW = 2), where the whole warp holds the row's 128 columns
// of one scale, which goes to sy. align: of Y's rows, in bytes. row_at: element offset of the row;
// columns from n on do not exist.
template <int NW>
GPTQ_DEV void store_row4(const float4 (&v)[NW], void* y, long long row_at, int col, int n,
                         int y_dtype, int align, float* sy) {
  float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
  const bool vec = col + 4 <= n && align >= (NW == 2 ? 4 : y_dtype == GPTQ_F32 ? 16 : 8);
  if constexpr (NW == 2) {
    const float u[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t mx = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = silu_mul(o[e], u[e]);
      if (col + e < n) mx = max(mx, mag_bits(o[e]));
    }
    float s, inv;
    block_scale(__reduce_max_sync(0xFFFFFFFFu, mx), s, inv);
    if ((threadIdx.x & 31) == 0) *sy = s;
    const uint32_t q = e4m3x4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    uint8_t* p = reinterpret_cast<uint8_t*>(y) + row_at + col;
    if (vec) {
      *reinterpret_cast<uint32_t*>(p) = q;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < n) p[e] = (uint8_t)(q >> (e * 8));
    }
  } else if (vec) {
    if (y_dtype == GPTQ_F32)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + row_at + col) = v[0];
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(y) + row_at + col) =
          make_uint2(pack2(o[0], o[1], y_dtype), pack2(o[2], o[3], y_dtype));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < n) store_out(y, row_at + col + e, o[e], y_dtype);
  }
}

GPTQ_DEV void store_if(bool on, void* p, uint32_t v) {  // a branch would cost more than the store
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q st.global.u32 [%0], %1;\n\t}" ::"l"(p),
               "r"(v), "r"((uint32_t)on)
               : "memory");
}
GPTQ_DEV void store_if(bool on, void* p, uint16_t v) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q st.global.u16 [%0], %1;\n\t}" ::"l"(p),
               "h"(v), "r"((uint32_t)on)
               : "memory");
}
// One 4-byte word a lane of WORDS neighbours, which begin a row's piece at p, `left` elements of ES bytes
// before the row's end: this lane's word i and its neighbour's. Where 2-byte elements start between
// words, every lane takes one element from its neighbour, so that whole words are stored all the
// same, and the first and the last lane store one element each (8000 x 8191 x 512 with two 2-byte
// stores a lane: 108 us, with branches around these: 125, so: 92).
template <int ES, int WORDS>
GPTQ_DEV void store_word(uint8_t* p, int i, uint32_t w, uint32_t next, int left) {
  if constexpr (ES == 4) {
    store_if(i < left, p + 4 * i, w);
  } else {
    const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
    const int at = 2 * i + odd, end = min(2 * WORDS, left);
    const uint32_t v = __funnelshift_r(w, next, odd * 16);
    uint8_t* q = p + 2 * at;
    store_if(at + 1 < end, q, v);
    const bool first = odd && i == 0;
    store_if(first ? end > 0 : at + 1 == end, first ? p : q, (uint16_t)(first ? w : v));
    if (end == 2 && first) store_if(true, q, (uint16_t)v);  // both ends are this lane's
  }
}

}  // namespace gptq
