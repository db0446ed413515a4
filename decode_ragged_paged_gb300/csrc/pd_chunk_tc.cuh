// pd_chunk_tc.cuh -- what the tensor-core kernels of the chunk attention share: the tiles'
// sizes, tensor memory's columns, waits that a warp agrees on, masks and remainders of
// weights.
#pragma once

#include "pd_chunk.cuh"
#include "pd_launch.cuh"
#include "pd_tc.cuh"

namespace pd {

namespace {

constexpr int kM = 128;  // query rows of a tile
constexpr int kN = kChunkKeys;
constexpr float kSumLimit = 256.0f;   // 2^8: largest row sum of weights taken with a stale maximum
constexpr float kRaise = 8.0f;        // log2 of it: a maximum is raised when it grew by more

// Rows of a box: the largest power of two, up to a tile, that a page is a multiple of,
// so that every box lies in one page (and is at least a swizzle's 8 rows high).
__host__ __device__ __forceinline__ int page_box(int page_size) {
  const int b = page_size & -page_size;
  return b < kN ? b : kN;
}

// TMEM: two S / P buffers of 64 columns a group, then the groups' O accumulators.
__device__ __forceinline__ uint32_t col_s(int g, uint32_t buf) { return (uint32_t)(2 * g + buf) * kN; }
__device__ __forceinline__ uint32_t col_o(int g) { return 256u + (uint32_t)g * 128; }

// Whether the item has a second query tile (else its groups share the first).
__device__ __forceinline__ bool two_tiles(const ChunkParams& p, const ChunkItem& I) {
  return I.tokens > p.tile_tokens;
}

// The whole warp looks at a barrier and agrees: one uniform branch if the phase is
// there. (mbar_wait's lanes look one by one and meet again afterwards, which took a
// warp 100 to 200 cycles at a barrier that was ready: a fifth of a tile's time.)
__device__ __forceinline__ bool try_all(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred q, p, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// warp_mbar_wait by try_all. The waiting itself is a function of its own: the roles'
// loops together are more than an instruction cache holds, and 16 copies of it in
// line cost every case 2 to 4 %.
__device__ __noinline__ bool warp_wait_long(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (try_all(bar, parity)) return true;
    const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
    if (late) {
      report(status, PD_DEV_TIMEOUT);
      *abort = 1;
    }
    if (__any_sync(0xffffffffu, late || *abort != 0)) return false;
  }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  return try_all(bar, parity) || warp_wait_long(bar, parity, abort, status);
}

// Makes the scores of a row outside columns [lo, hi) of the tile -inf, in tensor
// memory, before a tile of a mask's edge is weighed: in line with the weights, where
// most tiles jump over it, it made those slower (D 64: 1450 cycles a tile for 1380).
__device__ __noinline__ void hide_scores(uint32_t t_s, int lo, int hi) {
#pragma unroll 1
  for (int c = 0; c < kN; c += 32) {
    const int from = lo - c, to = hi - c;
    if (__all_sync(0xffffffffu, from <= 0 && to >= 32)) continue;  // no row of the warp has any to hide
    // bits [from, to) of 32
    const uint32_t keep = (to <= 0 ? 0u : 0xffffffffu >> (32 - min(to, 32))) & (from >= 32 ? 0u : 0xffffffffu << max(from, 0));
    uint32_t v[32];
    tmem_ld32(t_s + c, v);
    tmem_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = (keep >> e) & 1u ? v[e] : 0xff800000u;
    tmem_st32(t_s + c, v);
  }
  tmem_wait_st();
}

// Whether some row of the item sees fewer keys than average the weights' rounding
// out. What a row sees grows with its position under the causal mask, and shrinks
// without it (a window's lower end alone moves), so the first or the last row sees the fewest.
constexpr int kFewKeys = 128;
__device__ __forceinline__ bool few_keys(const ChunkParams& p, const ChunkItem& I) {
  const int last = I.first_tok + I.tokens - 1;
  const KeyRange a = chunk_keys(p, I.qo, I.kv, I.first_tok, I.first_tok + 1), b = chunk_keys(p, I.qo, I.kv, last, last + 1);
  return min(a.hi - a.lo, b.hi - b.lo) < kFewKeys;
}

// What bf16 leaves of a row's weights 2^(s scale - m), nm = -m, as bf16 pairs in columns
// 32 .. 63 of its scores' buffer, before the weights themselves overwrite columns
// 0 .. 31; the upper scores first, so that none is overwritten unread. A function
// of its own, as hide_scores.
__device__ __noinline__ void write_remainders(uint32_t t_s, float scale, float nm) {
  const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(nm, nm);
#pragma unroll 1
  for (int c = kN / 32 - 1; c >= 0; --c) {
    uint32_t v[32], w[16];
    tmem_ld32(t_s + 32 * c, v);
    tmem_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 x = ffma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, nm2);
      const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      const uint32_t hi = pack_bf16x2(pe.x, pe.y);
      w[e / 2] = pack_bf16x2(pe.x - bf16_lo(hi), pe.y - bf16_hi(hi));  // (the differences are exact)
    }
    tmem_st16(t_s + kN / 2 + 16 * c, w);
  }
}

// 32 bytes, a whole sector where the buffers are aligned to it: rows are a thread
// each, so narrower stores write sectors in pieces.
__device__ __forceinline__ void store_sector(void* to, const uint32_t* v, bool aligned32) {
  if (!aligned32) {
    static_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

}  // namespace

}  // namespace pd
