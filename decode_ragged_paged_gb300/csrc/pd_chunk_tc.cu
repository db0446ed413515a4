// pd_chunk_tc.cu -- the tensor-core kernel of the chunk attention (bf16, pages
// of a multiple of 8 slots): tcgen05 products with S, P and O in
// tensor memory, tiles fetched by TMA.
//
// One persistent CTA per SM walks its part of the work line (pd_chunk.cuh). Two
// groups of four softmax warps, each with its own S / P buffer and O accumulator
// in TMEM, keep the tensor cores and the exponential units busy in turn: while
// one group turns its scores into weights, the other group's products run. What
// the two groups share depends on the item:
//   more tokens than a tile holds: group g takes query tile g, both against the
//     same K and V tiles, so a K/V tile fetched once serves 256 query rows;
//   one query tile: the groups take alternate key tiles of it, each with its own
//     running maximum, sum and output, and are merged at the end.
// A query tile packs the query heads of a KV head: row m is token m /
// tile_heads, head m % tile_heads.
// Warps: 0 loads K, 2 V and 4 Q; 1 and 5 issue the products with K of group 0
// and 1, 3 and 7 those with V (each issuer waits only for its own group: with one
// for both, a group that is late held up the other); 8-11 and 12-15 are the
// groups, one query row a thread.
//
// Softmax. Weights are 2^(s scale log2 e - m) with a running maximum m that may
// be stale: a tile's weights are computed with the m of the tiles before, in one
// pass over its scores, and kept if every row's weights sum to at most 2^8;
// otherwise the tile is done again with its own maximum, and O is rescaled.
// Sums are fp32. The weights enter the product with V as bf16, as the tensor
// cores want V's own type there; the sum that divides takes them unrounded, so
// a result is off by the average of its weights' rounding errors, each at most
// half a bf16 step. Over many keys that averages out; where a row of the item sees
// fewer than 128 the weights' remainders are multiplied with V too, which leaves
// 2^-16 of a weight (two keys, values 3.5 to 4 and 0 to 1, bf16 output: 1.1e-2
// off with bf16 weights, 7.8e-3 with the remainders, half a step of the output).
//
// Bound and measured: 4 x 2048 tokens over 14000 to 16384 keys, 32 / 8 heads, D 128:
// the tensor cores (81 % of their cycles), 1025 us for one launch after a pause (1775
// TFLOP/s); calls one after another take 1140 to 1177 (1546 to 1597 TFLOP/s), as the
// power limit takes the clock down. 500 tokens over 32700: 163 us, and 186 a call one
// after another (1430 TFLOP/s, with the merge). 32 verifications of 2 to 8 tokens over
// 512 to 4096 keys: 55 us for 273 MB, HBM behind 17 us of start and merge. Prompts of
// 128 tokens, all with remainders: 64 of them 64.7 us, 58.6 without; a window of 64
// keys: 8 x 2000 tokens 112 us, 97 without. Windowed prefill, D 64: 47 us; there
// a tile takes 1380 cycles, two softmax warps a sub-partition with 350 instructions
// each and their latencies (issue 39 to 50 %; the exponentials 23 to 38 %), and an
// item 7000 more, from its last tile's product over the output to its next first.
//
// Every wait is bounded; on a timeout the CTA records PD_DEV_TIMEOUT, drains
// and frees its TMEM.
#include <math.h>
#include <stddef.h>
#include <string.h>

#include "pd_chunk_tc.cuh"

namespace pd {

namespace {

constexpr int kCtThreads = 512;

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;                // 64-column halves of a row (128 bytes each)
  static constexpr uint32_t kQHalf = kM * 128, kQTile = kHalves * kQHalf;  // query tiles
  static constexpr uint32_t kHalf = kN * 128, kTile = kHalves * kHalf;     // K and V tiles
  static constexpr int kRing = D == 128 ? 5 : 8;        // slots of the K ring and of the V ring
  static constexpr int kQ = D == 128 ? 2 : 4;           // slots of the Q ring
  static constexpr uint32_t kOffK = kQ * kQTile, kOffV = kOffK + kRing * kTile, kOffBar = kOffV + kRing * kTile;
  static constexpr uint32_t kOffML = kOffBar + 1024;    // group 1's maxima and sums
  static constexpr size_t kSmem = kOffML + 128 * 2 * sizeof(float) + 1024;
};
static_assert(kSelfBytes <= Shape<64>::kOffBar && kSelfBytes <= Shape<128>::kOffBar, "the rings hold the line first");
static_assert(Shape<128>::kSmem <= 232448 && Shape<64>::kSmem <= 232448, "shared memory of a CTA");

// Slots of the Q, K and V rings are freed by one arrival of each group. A group
// waits for every slot's every fill, its own or not, and then frees it, at once
// if the tile is the other group's: were it to pass over a fill without waiting,
// it could look at a barrier two phases early, where a parity wait lets it by.
constexpr int kItems = 4;  // items that the scheduler is ahead
struct Bars {
  ChunkItem items[kItems];  // no tokens: the end
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t q_full[4], q_empty[4];
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [group][S buffer]
  uint64_t ml_ready, merged;  // group 1's maxima and sums are in shared memory; its output has been read
  uint64_t drain;
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// V rows of keys that no row of the item sees become zeros, so that nothing of
// what they hold reaches O through a zero weight.
template <int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int to, int lane) {
  constexpr int kVec = Shape<D>::kHalves * 8;
  for (int i = lane; i < (to - from) * kVec; i += 32) {
    const int r = from + i / kVec, c = i % kVec;
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (c / 8) * Shape<D>::kHalf + r * 128 +
                                                                (c % 8) * 16),
                 "r"(0)
                 : "memory");
  }
}

}  // namespace

// POW2: pages of a power of two (others cost the loads of every tile a little more:
// 8 % of a large chunked prefill, so they have a kernel of their own).
template <int D, bool POW2>
__global__ void __launch_bounds__(kCtThreads, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
  using S = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = base, *sK = base + S::kOffK, *sV = base + S::kOffV;
  Bars* bars = reinterpret_cast<Bars*>(base + S::kOffBar);
  float2* sML = reinterpret_cast<float2*>(base + S::kOffML);  // group 1's (m, l) of every row
  volatile int* abort = &bars->abort;
  const uint32_t bars32 = smem_u32(bars);
  auto bar = [&](size_t member, uint32_t i = 0) { return bars32 + (uint32_t)member + 8 * i; };
  auto wait = [&](uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, abort, p.status); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kQ; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 2);  // the tile's last scores are there
    }
    for (int i = 0; i < S::kRing; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->s_full[i >> 1][i & 1], 1);
      mbar_init(&bars->p_full[i >> 1][i & 1], 4);
      mbar_init(&bars->pv_done[i >> 1][i & 1], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], kCtThreads / 32 - 1);  // every warp but the scheduler
    }
    mbar_init(&bars->ml_ready, 4);
    mbar_init(&bars->merged, 4);
    mbar_init(&bars->drain, 4);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  if (warp == 6) {
    tmem_alloc(&bars->tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  pdl_launch_dependents();
  pdl_wait_primary();  // the plan's work line
  ChunkItem I{};
  if (warp == 6) {
    // ------------------------------------------------------------ scheduler
    // Finds the CTA's work and walks through it ahead of the other warps. The
    // rings hold the line until the first item is out, as nothing else uses them
    // before that.
    ChunkWalk walk;
    const int4 cut = walk.begin(p, take_line(p, base), blockIdx.x);
    if (lane == 0) p.cuts[blockIdx.x] = cut;
    fence_proxy_async_smem();
    __syncwarp();
    uint32_t slot = 0, turn = 0;
    for (bool more = true; more;) {
      more = walk.next(p, I);
      if (!more) I.tokens = 0;
      if (!wait(bar(offsetof(Bars, item_empty), slot), (turn & 1u) ^ 1u)) break;
      if (lane == 0) {
        bars->items[slot] = I;
        mbar_arrive(&bars->item_full[slot]);
      }
      __syncwarp();
      if (++slot == kItems) slot = 0, ++turn;
    }
  }
  // The next item of the scheduler's, in every other warp.
  uint32_t item_slot = 0, item_turn = 0;
  auto next_item = [&]() -> bool {
    if (!wait(bar(offsetof(Bars, item_full), item_slot), item_turn & 1u)) return false;
    I = bars->items[item_slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[item_slot]);
    if (++item_slot == kItems) item_slot = 0, ++item_turn;
    return I.tokens > 0;
  };

  if (warp == 0 || warp == 2) {
    // ----------------------------------------------------------- K, V loads
    // One thread: a tile is a box per page and 64-column half, up to 16 of them,
    // and a box issued by a lane of its own takes 130 cycles (the lanes take turns
    // at an instruction that wants uniform operands) against 30 here. A tile's page
    // ids are read a tile ahead.
    const bool is_v = warp == 2, leader = elect_one();
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    uint8_t* ring = is_v ? sV : sK;
    uint64_t *full = is_v ? bars->v_full : bars->k_full, *empty = is_v ? bars->v_empty : bars->k_empty;
    const int pb = page_box(p.page_size), boxes = kN / pb;
    // to the next box: a page of a power of two has one (or the tile has)
    auto step_box = [&](int& idx, int& off) {
      if (POW2) {
        ++idx;
      } else {
        off += pb;
        if (off == p.page_size) off = 0, ++idx;
      }
    };
    uint32_t slot = 0, turn = 0;
    bool ok = true;
    while (ok && next_item()) {
      if (I.t1 <= I.t0) continue;
      if (leader) {
        const int kv_head = I.h / p.group;
        const int* list = p.page_indices + I.pbase;
        // Pages of the next tile's boxes, the first one's number in the request's list and its first row there.
        int next[8], next_idx = 0, next_off = 0;
        auto read = [&](int tile) {
          const int key = tile * kN;
          next_idx = POW2 ? key >> p.page_shift : key / p.page_size;
          next_off = POW2 ? key & (p.page_size - 1) & ~(kN - 1) : key - next_idx * p.page_size;
          int idx = next_idx, off = next_off;
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            next[b] = b < boxes && idx < I.need ? __ldg(list + idx) : 0;
            step_box(idx, off);
          }
        };
        const int nt = I.t1 - I.t0;
        read(I.tile(0));
        for (int i = 0; i < nt; ++i) {
          int idx = next_idx, off = next_off, page[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) page[b] = next[b];
          if (i + 1 < nt) read(I.tile(i + 1));
          ok = mbar_wait(&empty[slot], (turn & 1u) ^ 1u, abort, p.status);
          if (!ok) break;
          uint8_t* to = ring + slot * S::kTile;
          mbar_arrive_expect_tx(&full[slot], S::kTile);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            if (b == boxes) break;
            // pages past the request's end, and ids outside the pools: page num_pages, which TMA reads as zeros
            int id = page[b];
            if (idx >= I.need) {
              id = p.num_pages;
            } else if (id < 0 || id >= p.num_pages) {
              report(p.status, PD_DEV_BAD_PAGE_TABLE);
              id = p.num_pages;
            }
#pragma unroll
            for (int h = 0; h < S::kHalves; ++h)
              tma_load_4d(to + h * S::kHalf + b * pb * 128, map, 64 * h, p.nhd ? kv_head : off, p.nhd ? off : kv_head, id,
                          &full[slot]);
            step_box(idx, off);
          }
          if (++slot == S::kRing) slot = 0, ++turn;
        }
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp == 4) {
    // --------------------------------------------------------------- Q loads
    uint32_t q = 0, qturn = 0;
    bool ok = true;
    while (ok && next_item()) {
      if (I.t1 <= I.t0) continue;
      const int tiles = two_tiles(p, I) ? 2 : 1, tok = p.tile_tokens;
      for (int x = 0; ok && x < tiles; ++x) {
        ok = wait(bar(offsetof(Bars, q_empty), q), (qturn & 1u) ^ 1u);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[q], (uint32_t)(S::kHalves * tok * p.tile_heads * 128));
          for (int h = 0; h < S::kHalves; ++h)
            tma_load_3d(sQ + q * S::kQTile + h * S::kQHalf, &tm_q, 64 * h, I.h, I.q0 + x * tok, &bars->q_full[q]);
        }
        __syncwarp();
        if (++q == S::kQ) q = 0, ++qturn;
      }
    }
  } else if (warp == 1 || warp == 5) {
    // -------------------------------------------------------------- S = Q K^T
    // A group's scores run two tiles ahead of its weights, in two buffers: a
    // tile's are issued once the product with V of the tile two before has read
    // its weights out of the same columns.
    const int g = warp >> 2;
    constexpr uint32_t idesc_s = idesc_bf16_f32(kM, kN, 0);
    const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK);
    uint32_t q = 0, qturn = 0, ks = 0, kturn = 0;
    uint32_t own = 0;  // scores issued
    bool ok = true;
    while (ok && next_item()) {
      const int nt = I.t1 - I.t0;
      if (nt <= 0) continue;
      const bool two = two_tiles(p, I);
      const int step = two ? 1 : 2;
      uint32_t q_slot = q;  // of the group's query tile
      for (int x = 0; ok && x < (two ? 2 : 1); ++x) {
        ok = wait(bar(offsetof(Bars, q_full), q), qturn & 1u);
        if (x == g || !two) q_slot = q;
        else if (ok && lane == 0) mbar_arrive(&bars->q_empty[q]);  // the other group's
        if (++q == S::kQ) q = 0, ++qturn;
      }
      if (!ok) break;
      const uint64_t dq = sw128_desc(__shfl_sync(0xffffffffu, sQa + q_slot * S::kQTile, 0), 16, 1024);
      for (int i = 0; i < nt; ++i) {
        ok = wait(bar(offsetof(Bars, k_full), ks), kturn & 1u);
        if (!ok) break;
        if (two || (i & 1) == g) {
          const uint32_t buf = own & 1u;
          ok = own < 2 || wait(bar(offsetof(Bars, pv_done), 2 * g + buf), ((own - 2) >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dk = sw128_desc(__shfl_sync(0xffffffffu, sKa + ks * S::kTile, 0), 16, 1024);
          const uint32_t t_s = __shfl_sync(0xffffffffu, tmem + col_s(g, buf), 0);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_f16(t_s, desc_advance(dq, (kk / 4) * S::kQHalf + (kk % 4) * 32),
                         desc_advance(dk, (kk / 4) * S::kHalf + (kk % 4) * 32), idesc_s, kk > 0);
            tc_commit(&bars->s_full[g][buf]);
            // (by the softmax warps, who may still be two tiles behind, the K ring would be half held)
            tc_commit(&bars->k_empty[ks]);
            if (i + step >= nt) tc_commit(&bars->q_empty[q_slot]);  // the group's last of this item
          }
          __syncwarp();
          ++own;
        } else if (lane == 0) {
          mbar_arrive(&bars->k_empty[ks]);
        }
        if (++ks == S::kRing) ks = 0, ++kturn;
      }
      if (ok && !two && g >= nt && lane == 0) mbar_arrive(&bars->q_empty[q_slot]);  // no tile of the item is its own
    }
  } else if (warp == 3 || warp == 7) {
    // --------------------------------------------------------------- O += P V
    const int g = warp >> 2;
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kM, D, 1);
    const uint32_t sVa = smem_u32(sV);
    const uint32_t t_o = __shfl_sync(0xffffffffu, tmem + col_o(g), 0);
    uint32_t vs = 0, vturn = 0, own = 0;
    bool ok = true;
    while (ok && next_item()) {
      const int nt = I.t1 - I.t0;
      const bool two = two_tiles(p, I), few = few_keys(p, I);
      const int i0 = two ? 0 : g;
      for (int i = 0; i < nt; ++i) {
        ok = wait(bar(offsetof(Bars, v_full), vs), vturn & 1u);
        if (!ok) break;
        if (two || (i & 1) == g) {
          const uint32_t buf = own & 1u;
          const int k0 = I.tile(i) * kN;
          const int from = max(I.keys.lo - k0, 0), to = min(I.keys.hi - k0, kN);
          if (from > 0 || to < kN) {
            // with two tiles both groups' warps write the same zeros
            zero_rows<D>(sVa + vs * S::kTile, 0, from, lane);
            zero_rows<D>(sVa + vs * S::kTile, to, kN, lane);
            fence_proxy_async_smem();
            __syncwarp();
          }
          ok = wait(bar(offsetof(Bars, p_full), 2 * g + buf), (own >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = sw128_desc(__shfl_sync(0xffffffffu, sVa + vs * S::kTile, 0), S::kHalf, 1024);
          const uint32_t t_p = __shfl_sync(0xffffffffu, tmem + col_s(g, buf), 0);
          const uint32_t more = __shfl_sync(0xffffffffu, i > i0 ? 1u : 0u, 0);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              tc_mma_f16_tmem_a(t_o, t_p + 8 * kk, desc_advance(dv, kk * 2048), idesc_pv, kk > 0 ? 1u : more);
            if (few) {  // and their remainders
#pragma unroll
              for (int kk = 0; kk < kN / 16; ++kk)
                tc_mma_f16_tmem_a(t_o, t_p + kN / 2 + 8 * kk, desc_advance(dv, kk * 2048), idesc_pv, 1u);
            }
            tc_commit(&bars->pv_done[g][buf]);
          }
          __syncwarp();
          // the V slot is free once the product is done: a wait and a plain arrival here cost less than a second commit
          ok = wait(bar(offsetof(Bars, pv_done), 2 * g + buf), (own >> 1) & 1u);
          if (!ok) break;
          ++own;
        }
        if (lane == 0) mbar_arrive(&bars->v_empty[vs]);
        if (++vs == S::kRing) vs = 0, ++vturn;
      }
    }
  }
  if (warp < 8 && (warp & 1)) {
    // every product completes before TMEM is released; after an abort some may be under way
    if (elect_one()) {
      tc_commit(&bars->drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bars->drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  }
  if (warp >= 8) {
    // ----------------------------------------------------- softmax, epilogue
    const int g = (warp - 8) >> 2, wq = warp & 3, row = wq * 32 + lane;
    const int tok_row = row / p.tile_heads, head = row - tok_row * p.tile_heads;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    uint32_t own = 0, merges = 0;
    bool ok = true;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    while (ok && next_item()) {
      const int nt = max(I.t1 - I.t0, 0);
      const bool two = two_tiles(p, I), few = few_keys(p, I);
      const int half_tok = p.tile_tokens;
      const int tokens = two ? (g == 0 ? half_tok : I.tokens - half_tok) : I.tokens;  // of this group's tile
      const int tok0 = two && g == 1 ? half_tok : 0;
      const bool valid = tok_row < tokens;
      const bool warp_valid = wq * 32 < tokens * p.tile_heads;
      int lo = 0, hi = 0x7fffffff;  // rows that are not there are never masked and never stored
      if (valid) {
        const int tok = I.first_tok + tok0 + tok_row;
        const KeyRange k = chunk_keys(p, I.qo, I.kv, tok, tok + 1);
        lo = k.lo;
        hi = k.hi;
      }
      float m = valid ? -INFINITY : 0.f, l = 0.f;
      const int step = two ? 1 : 2, keys_end = (I.tile0 + I.t1) * kN;
      int k0 = (I.tile0 + I.t0 + I.rot + (two ? 0 : g) - step) * kN;  // first key of the tile before
      for (int i = two ? 0 : g; i < nt; i += step) {  // (with one query tile the others are the other group's)
        k0 += step * kN;
        if (k0 >= keys_end) k0 -= nt * kN;
        const uint32_t buf = own & 1u, t_s = tmem + lanes + col_s(g, buf);
        ok = wait(bar(offsetof(Bars, s_full), 2 * g + buf), (own >> 1) & 1u);
        if (!ok) break;
        ++own;
        if (warp_valid) {
          tc_fence_after();
          const int c_lo = lo - k0, c_hi = hi - k0;
          const bool full = __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kN);
          if (!full) hide_scores(t_s, c_lo, c_hi);
          uint32_t w[kN / 2];
          float2 sum[2];
          // weights of the tile with maximum m, as bf16 pairs, and their sum
          auto weights = [&](float nm) {
            const float2 nm2 = make_float2(nm, nm);
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            uint32_t v[2][32];
            tmem_ld32(t_s, v[0]);
            tmem_ld32(t_s + 32, v[1]);
            tmem_wait_ld(v[0]);
            tmem_wait_ld(v[1]);
#pragma unroll
            for (int c = 0; c < kN / 32; ++c) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 x =
                    ffma2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sc2, nm2);
                const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                w[16 * c + e / 2] = pack_bf16x2(pe.x, pe.y);
                sum[(e / 2) & 1] = fadd2(sum[(e / 2) & 1], pe);
              }
            }
          };
          bool stale = __all_sync(0xffffffffu, m > -INFINITY), over = false;
          if (stale) {
            weights(-m);
            const float s = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            over = __any_sync(0xffffffffu, valid && s > kSumLimit);
            stale = !over;
          }
          if (!stale) {
            // the tile's own maximum
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kN / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(t_s + 32 * c, v);
              tmem_wait_ld(v);
#pragma unroll
              for (int e = 0; e < 32; e += 2) mx = fmax3(mx, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            }
            const float ms = mx * p.scale_log2;
            float alpha = 1.f;
            if (valid && mx > -INFINITY) {
              if (m == -INFINITY) {
                m = ms;
              } else if (ms > (over ? m : m + kRaise)) {
                // (a maximum left below a row's weights' limit would do every tile twice)
                alpha = exp2f(m - ms);
                m = ms;
              }
            }
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
              // the product of the tile before (own counts this one already) is under way
              ok = wait(bar(offsetof(Bars, pv_done), 2 * g + ((own - 2) & 1u)), ((own - 2) >> 1) & 1u);
              if (!ok) break;
              tc_fence_after();
              l *= alpha;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tmem + lanes + col_o(g) + 32 * c, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(tmem + lanes + col_o(g) + 32 * c, o);
              }
              tmem_wait_st();
            }
            weights(m == -INFINITY ? 0.f : -m);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (few) write_remainders(t_s, p.scale_log2, m == -INFINITY ? 0.f : -m);
          tmem_st32(t_s, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
        }
        // warps without rows leave what is there: only rows that are not stored read it
        if (lane == 0) mbar_arrive(&bars->p_full[g][buf]);
      }
      if (!ok) break;
      const bool other = !two && nt > 1;  // group 1 has tiles of the same rows
      if (g == 1 && !two) {
        if (nt < 2) continue;
        ok = wait(bar(offsetof(Bars, pv_done), 2 + ((own - 1) & 1u)), ((own - 1) >> 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        sML[row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ml_ready);
        // group 0 has read this group's output: its accumulator may be written again
        ok = wait(bar(offsetof(Bars, merged)), merges & 1u);
        tc_fence_after();
        ++merges;
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      if (nt > 0) {
        ok = wait(bar(offsetof(Bars, pv_done), 2 * g + ((own - 1) & 1u)), ((own - 1) >> 1) & 1u);
        if (!ok) break;
      }
      if (other) {
        ok = wait(bar(offsetof(Bars, ml_ready)), merges & 1u);
        if (!ok) break;
        const float2 b = sML[row];
        const float top = fmaxf(m, b.x), at = top == -INFINITY ? 0.f : top;
        f0 = exp2f(m - at);
        f1 = exp2f(b.x - at);
        l = l * f0 + b.y * f1;
        m = top;
      }
      tc_fence_after();
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const float lse2 = l != 0.f ? m + log2f(l) : -INFINITY;
      const int64_t slot = part_slot(I, blockIdx.x);
      const int mrow = tok0 * p.tile_heads + row;
      const int64_t orow = (int64_t)(I.q0 + tok0 + tok_row) * p.hq + I.h + head;
      f0 *= inv;
      f1 *= inv;
      if (warp_valid) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (nt > 0) {
            tmem_ld32(tmem + lanes + col_o(g) + 32 * c, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f0);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          if (other) {
            uint32_t b[32];
            tmem_ld32(tmem + lanes + col_o(1) + 32 * c, b);
            tmem_wait_ld(b);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(b[e]) * f1);
          }
          if (valid) {
            if (slot < 0 && p.o_dtype == PD_BF16) {
              uint16_t* o = static_cast<uint16_t*>(p.o) + orow * D + 32 * c;
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                uint32_t u[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  u[x] = pack_bf16x2(__uint_as_float(v[e + 2 * x]), __uint_as_float(v[e + 2 * x + 1]));
                store_sector(o + e, u, p.aligned32);
              }
            } else {
              float* o = (slot < 0 ? static_cast<float*>(p.o) + orow * D : p.part_o + (slot * p.rows + mrow) * D) +
                         32 * c;
#pragma unroll
              for (int e = 0; e < 32; e += 8) store_sector(o + e, v + e, p.aligned32);
            }
          }
        }
      }
      if (valid) {
        if (slot >= 0) p.part_lse[slot * p.rows + mrow] = lse2;
        else if (p.lse != nullptr) p.lse[orow] = lse2 * kLn2;
      }
      tc_fence_before();
      __syncwarp();
      if (other) {
        if (lane == 0) mbar_arrive(&bars->merged);
        ++merges;
      }
    }
  }

  // Normally every copy has been consumed here. After an abort, copies may still
  // be in flight: give them a bounded 2 ms to land before shared memory is freed.
  if (*abort && warp == 0 && lane == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 6) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- host
namespace {

template <int D, bool POW2>
cudaError_t launch_d(const ChunkParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t stream) {
  const cudaError_t e = allow_smem<chunk_tc_kernel<D, POW2>>(Shape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_tc_kernel<D, POW2>, dim3((unsigned)p.grid), kCtThreads, Shape<D>::kSmem, stream, tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkParams& p, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const int pb = page_box(p.page_size);
  if (!make_rows_map(&tq, p.q, PD_BF16, p.total_qo, p.hq, p.head_dim, 64, p.tile_tokens, true, p.tile_heads,
                     p.q_stride) ||
      !make_pool_map(&tk, p.k_pool, PD_BF16, p.num_pages, p.hkv, p.page_size, p.head_dim, 64, pb, true, p.nhd != 0) ||
      !make_pool_map(&tv, p.v_pool, PD_BF16, p.num_pages, p.hkv, p.page_size, p.head_dim, 64, pb, true, p.nhd != 0))
    return cudaErrorInvalidValue;
  last_kernel() = "chunk_tc_kernel";
  profile_begin(stream);
  cudaError_t e;
  if (p.page_shift >= 0)
    e = p.head_dim == 64 ? launch_d<64, true>(p, tq, tk, tv, stream) : launch_d<128, true>(p, tq, tk, tv, stream);
  else
    e = p.head_dim == 64 ? launch_d<64, false>(p, tq, tk, tv, stream) : launch_d<128, false>(p, tq, tk, tv, stream);
  profile_end(stream);
  return e;
}

}  // namespace pd
