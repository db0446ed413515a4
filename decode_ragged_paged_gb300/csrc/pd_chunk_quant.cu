// pd_chunk_quant.cu -- the tensor-core kernel of the chunk attention over a cache held
// in 8 bits (bf16 queries; pages and blocks of a multiple of 8 tokens; more than 8 query rows a KV head).
//
// For a block of tokens with scales a of K and b of V, and e4m3 values k, v:
//   s_j = scale a_j <q, k_j>,  o = sum_j softmax(s)_j b_j v_j
// How the work is dealt and what the two groups of softmax warps share are those of pd_chunk_tc.cu.
// What the 8 bits change:
//   K enters the products as it is in memory (kind::f8f6f4), and so q has to be e4m3
//     too: x = h + l of the row's scaled values, h = rn(x), l = rn(x - h). With the row's
//     largest value in (224, 448], bf16's 8 bits are two times e4m3's 4, so h + l is x itself
//     from 1/4 up and off by at most 2^-10 below (2^-17 of the row's largest value). [h | l]
//     [k | k]^T takes as long as bf16's product and reads half the bytes; K is not converted.
//   V becomes fp16, exactly and without its scale, on its way from the ring of its 8-bit rows to
//     a short one of the products' operands, by four warps of their own.
//   Both scales belong to 8 tokens at least, and act on the scores: with m the row's running maximum
//     of s_j + log2 b_j (base 2) the weights are W_j = 2^(s_j + log2 b_j - m), o = sum W_j v_j / sum (W_j / b_j).
//     An exponent is one product and sum either way, so the scales cost a load and a sum for each 8.
//   W is fp16, as V is. A row's largest is 2^3 to 2^8 when m is set, and m stays until 32 weights of a tile
//     add up to more than fp16 holds: then m is raised out of that sum, the output so far scaled, and the tile done
//     again. At 2^3 the rounding of weights below 2^-14 is at most 2^-28 of the largest contribution. The sums are
//     fp32. (Of 64 weights and 2^15: 232 us where it takes 227; of 16 or 8 the registers did not do: 239.)
// Warps (20, of 96 registers: the softmax's tile of 64 scores and its weights want them): 0 finds the work; 6 loads K
// and makes a tile's factors out of its scales, 2 loads V and 4 Q; 1 and 5 issue the products with K of group 0 and
// 1, 3 and 7 those with V; 8-11 and 12-15 are the groups; 16-19 split q and convert V. A tile's factors are kept for
// 32 tiles, as the softmax reads them after K's slot is free.
//
// Bound (D 128, 152 SMs): the softmax warps. A pair of tiles (64 keys, two query tiles) is 1024 cycles of products, half of
// them e4m3's, and the tensor cores are busy in 55 % of the cycles (over bf16, pd_chunk_tc.cu: 77 %); shared memory's
// banks are read in 28 % of them and written in 7 (there 36 and 9). The scales and V's conversion make it 127
// million instructions for 90 (500 tokens over 32700 keys), and warps wait longest for loads, of tensor memory above all.
// That case takes 228 to 230 us (over bf16 184), without the softmax 172; 4 x 2048 tokens over 14000 to 16384 keys 1355 to 1385
// (1140 to 1177), 69 % of the dense bf16 rate, 8 % of it raised maxima where scales differ much. With
// one query tile (32 requests of 2 to 8 tokens: 51 us, bf16 55) a tile of keys takes 0.5 us, 5.0 TB/s, and an
// item's ends 4.5: the last product, both groups' outputs joined, and the first tile's own maximum, each
// after the other (152 x 4 tokens over 1024 keys 114 us, 38 over 4096, as many keys, 87).
//
// Every wait is bounded; on a timeout the CTA records PD_DEV_TIMEOUT, drains
// and frees its TMEM.
#include <math.h>
#include <stddef.h>

#include "pd_chunk_quant.cuh"
#include "pd_chunk_tc.cuh"
#include "pd_quant.cuh"

namespace pd {

namespace {

constexpr int kCqThreads = 640;
constexpr int kScaleTiles = 32;  // tiles whose factors are kept
constexpr int kGroups = kN / 8;  // 8-token groups of a tile
constexpr int kCqItems = 6;      // items that the scheduler is ahead
constexpr float kShift = 3.0f;            // log2 of the weight of a row's largest key
constexpr float kSumShift = kShift + 5;   // and of the sum of 32 alike
constexpr float kWeightLimit = 65504.0f;  // fp16's largest: sum of 32 weights taken with a stale maximum

// A tile's scales as the softmax takes them.
struct Factors {
  float4 k[kGroups / 4];        // K's
  float4 log_v[kGroups / 4];    // log2 of V's
  float4 inverse[kGroups / 4];  // 1 / V's
};

template <int D>
struct QuantShape {
  static constexpr uint32_t kQHalf = kM * 128, kQTile = D / 64 * kQHalf;  // query tiles: bf16, then [h | l]
  static constexpr uint32_t kCodes = kN * D;                              // a tile of 8-bit K or V
  static constexpr uint32_t kVHalf = kN * 128, kVTile = D / 64 * kVHalf;  // a tile of fp16 V
  static constexpr int kQ = D == 128 ? 2 : 4;       // slots of the Q ring
  static constexpr int kK = D == 128 ? 7 : 8;       // of K's
  static constexpr int kC = D == 128 ? 6 : 8;       // of V's 8-bit rows
  static constexpr int kV = D == 128 ? 3 : 4;       // of V's fp16 tiles
  static constexpr uint32_t kOffK = kQ * kQTile, kOffC = kOffK + kK * kCodes, kOffV = kOffC + kC * kCodes;
  static constexpr uint32_t kOffBar = kOffV + kV * kVTile;
  static constexpr uint32_t kOffML = kOffBar + 1024;                       // group 1's maxima and sums
  static constexpr uint32_t kOffFactors = kOffML + kM * 8;                 // of the last tiles
  static constexpr uint32_t kOffQS = kOffFactors + kScaleTiles * sizeof(Factors);  // the rows' scales of q [slot][row]
  static constexpr size_t kSmem = kOffQS + kQ * kM * 4 + 1024;
  static_assert(kSelfBytes <= kOffBar, "the rings hold the line first");
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

struct QuantBars {
  ChunkItem items[kCqItems];  // no tokens: the end
  int nan[kCqItems];          // V had a NaN where not all of the item's rows see it
  uint64_t item_full[kCqItems], item_empty[kCqItems];
  uint64_t q_full[4], q_ready[4], q_empty[4];
  uint64_t k_full[8], k_empty[8], c_full[8], c_empty[8], v_full[4], v_empty[4];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [group][S buffer]
  uint64_t ml_ready, merged, drain;
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(QuantBars) <= 1024, "barrier block");

__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Two bf16 values (times f) as two e4m3 terms each: h in the low 16 bits, l in the high ones.
__device__ __forceinline__ uint32_t split_pair(uint32_t pair, float f) {
  const float x = bf16_lo(pair) * f, y = bf16_hi(pair) * f;
  const uint32_t h = pack_e4m3x2(x, y);
  const float2 b = unpack_e4m3x2(h);
  return h | pack_e4m3x2(x - b.x, y - b.y) << 16;
}

// A query row of a tile (swizzled rows of 128 bytes, `row` at `tile` + 128 row), bf16, becomes its
// two e4m3 terms in place: the 128 bytes of 64 values become 64 of h and 64 of l. Returns the row's
// scale. An infinity makes all of the row NaN, a NaN itself.
template <int D>
__device__ __forceinline__ float split_row(uint32_t tile, int row) {
  const uint32_t at = tile + row * 128;
  const int sw = row & 7;
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = ld_shared(at + (c / 8) * QuantShape<D>::kQHalf + (((c & 7) ^ sw) << 4));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
  }
  const int e = scale_exponent(m);
  const float f = m <= 3.4e38f ? power_of_two(-e) : __uint_as_float(0x7fffffffu);
#pragma unroll 1
  for (uint32_t half = at; half < at + D / 64 * QuantShape<D>::kQHalf; half += QuantShape<D>::kQHalf) {
    // chunk c of h and of l, 16 values each, out of chunks 2 c and 2 c + 1 of 8: those that l's
    // first ones overwrite are read before
    uint4 last[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) last[c] = ld_shared(half + (((c + 4) ^ sw) << 4));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 a = c < 2 ? ld_shared(half + (((2 * c) ^ sw) << 4)) : last[2 * (c & 1)];
      const uint4 b = c < 2 ? ld_shared(half + (((2 * c + 1) ^ sw) << 4)) : last[2 * (c & 1) + 1];
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = split_pair(w[2 * i], f), y = split_pair(w[2 * i + 1], f);
        h[i] = __byte_perm(x, y, 0x5410);
        l[i] = __byte_perm(x, y, 0x7632);
      }
      st_shared(half + ((c ^ sw) << 4), make_uint4(h[0], h[1], h[2], h[3]));
      st_shared(half + (((c + 4) ^ sw) << 4), make_uint4(l[0], l[1], l[2], l[3]));
    }
  }
  return m <= 3.4e38f ? power_of_two(e) : 1.f;
}

// Two fp32 values -> one fp16x2 word, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What a score of a group is multiplied by for the softmax's base-2 exponents, K's scale times the row's.
// Never 0: a masked score is -inf, and times 0 it would be NaN.
constexpr float kFactorMin = 1e-37f;

}  // namespace

// POW2: pages of a power of two.
template <int D, bool POW2>
__global__ void __launch_bounds__(kCqThreads, 1)
    chunk_quant_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
  using S = QuantShape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base32 = smem_u32(base);
  QuantBars* bars = reinterpret_cast<QuantBars*>(base + S::kOffBar);
  float2* sML = reinterpret_cast<float2*>(base + S::kOffML);
  Factors* sFactors = reinterpret_cast<Factors*>(base + S::kOffFactors);
  float* sQS = reinterpret_cast<float*>(base + S::kOffQS);
  volatile int* abort = &bars->abort;
  const uint32_t bars32 = smem_u32(bars);
  auto bar = [&](size_t member, uint32_t i = 0) { return bars32 + (uint32_t)member + 8 * i; };
  auto wait = [&](uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, abort, p.status); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kQ; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_ready[i], 4);
      mbar_init(&bars->q_empty[i], 2 + 8);  // the groups' last scores, and every softmax warp has its rows' scales
    }
    for (int i = 0; i < S::kK; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);
    }
    for (int i = 0; i < S::kC; ++i) {
      mbar_init(&bars->c_full[i], 1);
      mbar_init(&bars->c_empty[i], 4);
    }
    for (int i = 0; i < S::kV; ++i) {
      mbar_init(&bars->v_full[i], 4);
      mbar_init(&bars->v_empty[i], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->s_full[i >> 1][i & 1], 2);  // the product, and the issuer, who has seen the tile's factors
      mbar_init(&bars->p_full[i >> 1][i & 1], 4);
      mbar_init(&bars->pv_done[i >> 1][i & 1], 1);
    }
    for (int i = 0; i < kCqItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], kCqThreads / 32 - 1);  // every warp but the scheduler
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
  pdl_wait_primary();  // the plan's work line, and what the cache was appended by
  // The next item of the scheduler's, in every other warp; and that the warp is done with it.
  uint32_t item_slot = 0, item_turn = 0;
  auto await_item = [&]() -> bool {
    return wait(bar(offsetof(QuantBars, item_full), item_slot), item_turn & 1u) && bars->items[item_slot].tokens > 0;
  };
  auto leave_item = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[item_slot]);
    if (++item_slot == kCqItems) item_slot = 0, ++item_turn;
  };
  auto next_item = [&](ChunkItem& I) -> bool {
    if (!await_item()) return false;
    I = bars->items[item_slot];
    leave_item();
    return true;
  };
  if (warp < 8) {
  if (warp == 0) {
    // ------------------------------------------------------------ scheduler
    ChunkWalk walk;
    const int4 cut = walk.begin(p, take_line(p, base), blockIdx.x);
    if (lane == 0) p.cuts[blockIdx.x] = cut;
    fence_proxy_async_smem();
    __syncwarp();
    ChunkItem I{};
    uint32_t slot = 0, turn = 0;
    for (bool more = true; more;) {
      more = walk.next(p, I);
      if (!more) I.tokens = 0;
      if (!wait(bar(offsetof(QuantBars, item_empty), slot), (turn & 1u) ^ 1u)) break;
      if (lane == 0) {
        bars->items[slot] = I;
        bars->nan[slot] = 0;
        mbar_arrive(&bars->item_full[slot]);
      }
      __syncwarp();
      if (++slot == kCqItems) slot = 0, ++turn;
    }
  } else if (warp == 6 || warp == 2) {
    // ----------------------------------------------------------- K, V loads
    // Four tiles at a time: a lane has one 8-token group of one of them. Their pages are read two
    // such batches ahead, and K's loader reads their scales one ahead and makes the factors of four tiles
    // in one go; read a tile ahead, either kept a tile waiting for about 1000 cycles. The boxes, a page's
    // each, are issued by one thread. A tile's bytes may arrive before they are expected: the
    // barrier waits for the arrival that expects them.
    const bool is_v = warp == 2;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    uint8_t* ring = base + (is_v ? S::kOffC : S::kOffK);
    uint64_t* full_bars = is_v ? bars->c_full : bars->k_full;
    const uint32_t empty = bar(is_v ? offsetof(QuantBars, c_empty) : offsetof(QuantBars, k_empty));
    const uint32_t slots = is_v ? S::kC : S::kK;
    const int pb = page_box(p.page_size), boxes = kN / pb, per_box = pb / 8, blocks = p.page_size / p.scale_block,
              block_shift = 31 - __clz(p.scale_block);
    uint32_t slot = 0, turn = 0, count = 0;
    bool ok = true;
    ChunkItem I;
    while (ok && next_item(I)) {
      const int nt = I.t1 - I.t0;
      if (nt <= 0) continue;
      const int kv_head = I.h / p.group, start = I.tile(0), end = I.tile0 + I.t1;
      const int* list = p.page_indices + I.pbase;
      // the lane's group in the batch from tile i on: its first key, and that key's place in the list (-1: none)
      auto group_key = [&](int i) {
        const int tile = start + i + lane / 8;
        return (tile < end ? tile : tile - nt) * kN + 8 * (lane & 7);
      };
      auto group_idx = [&](int key, int i) {
        const int idx = POW2 ? key >> p.page_shift : key / p.page_size;
        return i + lane / 8 < nt && idx < I.need ? idx : -1;
      };
      auto read_page = [&](int i) {
        const int idx = group_idx(group_key(i), i);
        return idx >= 0 ? __ldg(list + idx) : p.num_pages;
      };
      // pages past the request's end, and ids outside the pools: page num_pages, which TMA reads as zeros
      auto checked = [&](int id, int i) {
        if (id >= 0 && id < p.num_pages) return id;
        if (group_idx(group_key(i), i) >= 0) report(p.status, PD_DEV_BAD_PAGE_TABLE);
        return p.num_pages;
      };
      float scale_k = 0.f, scale_v = 0.f;  // of the next batch
      auto read_scales = [&](int id, int i) {
        const int key = group_key(i), off = key - (POW2 ? key >> p.page_shift : key / p.page_size) * p.page_size;
        scale_k = scale_v = 0.f;
        // (a group that no row of the item sees may have anything as its scale)
        if (id < p.num_pages && key < I.keys.hi && key + 8 > I.keys.lo) {
          const int64_t at = ((int64_t)id * p.hkv + kv_head) * blocks + (POW2 ? off >> block_shift : off / p.scale_block);
          scale_k = __ldg(p.k_scale + at);
          scale_v = __ldg(p.v_scale + at);
        }
      };
      int id = checked(read_page(0), 0), ahead = read_page(4);
      if (!is_v) read_scales(id, 0);
      for (int i0 = 0; ok && i0 < nt; i0 += 4) {
        const int key = group_key(i0), off = key - (POW2 ? key >> p.page_shift : key / p.page_size) * p.page_size;
        const int next = checked(ahead, i0 + 4);
        ahead = read_page(i0 + 8);
        const float a = fmaxf(scale_k, kScaleMin), b = fmaxf(scale_v, kScaleMin);
        if (!is_v) read_scales(next, i0 + 4);
        const int tiles = min(4, nt - i0);
        for (int x = 0; x < tiles; ++x) {
          ok = wait(empty + 8 * slot, (turn & 1u) ^ 1u);
          if (!ok) break;
          int bid[8], boff[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            if (n == boxes) break;
            bid[n] = __shfl_sync(0xffffffffu, id, 8 * x + n * per_box);
            boff[n] = __shfl_sync(0xffffffffu, off, 8 * x + n * per_box);
          }
          if (elect_one()) {
            uint8_t* to = ring + slot * S::kCodes;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              if (n == boxes) break;
              tma_load_4d(to + n * pb * D, map, 0, p.nhd ? kv_head : boff[n], p.nhd ? boff[n] : kv_head, bid[n],
                          &full_bars[slot]);
            }
          }
          __syncwarp();
          if (!is_v && x == 0) {
            Factors& f = sFactors[(count + i0 + lane / 8) & (kScaleTiles - 1)];
            const float lb = fast_log2(b);
            if (lane / 8 < tiles) {
              reinterpret_cast<float*>(f.k)[lane & 7] = a;
              reinterpret_cast<float*>(f.log_v)[lane & 7] = lb;
              reinterpret_cast<float*>(f.inverse)[lane & 7] = inverse_scale(lb);
            }
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(&full_bars[slot], S::kCodes);
          if (++slot == slots) slot = 0, ++turn;
        }
        id = next;
      }
      count += nt;
    }
  } else if (warp == 4) {
    // --------------------------------------------------------------- Q loads
    uint32_t q = 0, qturn = 0;
    bool ok = true;
    ChunkItem I;
    while (ok && next_item(I)) {
      if (I.t1 <= I.t0) continue;
      const int tiles = two_tiles(p, I) ? 2 : 1, tok = p.tile_tokens;
      for (int x = 0; ok && x < tiles; ++x) {
        ok = wait(bar(offsetof(QuantBars, q_empty), q), (qturn & 1u) ^ 1u);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[q], (uint32_t)(D / 64 * tok * p.tile_heads * 128));
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(base + q * S::kQTile + h * S::kQHalf, &tm_q, 64 * h, I.h, I.q0 + x * tok, &bars->q_full[q]);
        }
        __syncwarp();
        if (++q == S::kQ) q = 0, ++qturn;
      }
    }
  } else if (warp == 1 || warp == 5) {
    // -------------------------------------------------------------- S = [h | l] [k | k]^T
    const int g = warp >> 2;
    constexpr uint32_t idesc_s = idesc_e4m3_f32(kM, kN);
    uint32_t q = 0, qturn = 0, ks = 0, kturn = 0;
    uint32_t own = 0;  // scores issued
    bool ok = true;
    ChunkItem I;
    while (ok && next_item(I)) {
      const int nt = I.t1 - I.t0;
      if (nt <= 0) continue;
      const bool two = two_tiles(p, I);
      const int step = two ? 1 : 2;
      uint32_t q_slot = q;  // of the group's query tile
      for (int x = 0; ok && x < (two ? 2 : 1); ++x) {
        ok = wait(bar(offsetof(QuantBars, q_ready), q), qturn & 1u);
        if (x == g || !two) q_slot = q;
        else if (ok && lane == 0) mbar_arrive(&bars->q_empty[q]);  // the other group's
        if (++q == S::kQ) q = 0, ++qturn;
      }
      if (!ok) break;
      const uint64_t dq = sw128_desc(__shfl_sync(0xffffffffu, base32 + q_slot * S::kQTile, 0), 16, 1024);
      for (int i = 0; i < nt; ++i) {
        ok = wait(bar(offsetof(QuantBars, k_full), ks), kturn & 1u);
        if (!ok) break;
        if (two || (i & 1) == g) {
          const uint32_t buf = own & 1u;
          ok = own < 2 || wait(bar(offsetof(QuantBars, pv_done), 2 * g + buf), ((own - 2) >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) mbar_arrive(&bars->s_full[g][buf]);
          const uint32_t at = __shfl_sync(0xffffffffu, base32 + S::kOffK + ks * S::kCodes, 0);
          const uint64_t dk = D == 128 ? sw128_desc(at, 16, 1024) : sw64_desc(at, 512);
          const uint32_t t_s = __shfl_sync(0xffffffffu, tmem + col_s(g, buf), 0);
          if (elect_one()) {
            // 32 values a step: two of h and two of l for each 64 values of the rows
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_f8(t_s, desc_advance(dq, (kk / 4) * S::kQHalf + (kk % 4) * 32),
                        desc_advance(dk, (kk / 4) * 64 + (kk % 2) * 32), idesc_s, kk > 0);
            tc_commit(&bars->s_full[g][buf]);
            tc_commit(&bars->k_empty[ks]);
            if (i + step >= nt) tc_commit(&bars->q_empty[q_slot]);  // the group's last of this item
          }
          __syncwarp();
          ++own;
        } else if (lane == 0) {
          mbar_arrive(&bars->k_empty[ks]);
        }
        if (++ks == S::kK) ks = 0, ++kturn;
      }
      if (ok && !two && g >= nt && lane == 0) mbar_arrive(&bars->q_empty[q_slot]);  // no tile of the item is its own
    }
  } else if (warp == 3 || warp == 7) {
    // --------------------------------------------------------------- O += P V
    const int g = warp >> 2;
    constexpr uint32_t idesc_pv = idesc_f16_f32(kM, D, 1);
    const uint32_t t_o = __shfl_sync(0xffffffffu, tmem + col_o(g), 0);
    uint32_t vs = 0, vturn = 0, own = 0;
    bool ok = true;
    ChunkItem I;
    while (ok && next_item(I)) {
      const int nt = I.t1 - I.t0;
      const bool two = two_tiles(p, I);
      const int i0 = two ? 0 : g;
      for (int i = 0; i < nt; ++i) {
        ok = wait(bar(offsetof(QuantBars, v_full), vs), vturn & 1u);
        if (!ok) break;
        if (two || (i & 1) == g) {
          const uint32_t buf = own & 1u;
          ok = wait(bar(offsetof(QuantBars, p_full), 2 * g + buf), (own >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv =
              sw128_desc(__shfl_sync(0xffffffffu, base32 + S::kOffV + vs * S::kVTile, 0), S::kVHalf, 1024);
          const uint32_t t_p = __shfl_sync(0xffffffffu, tmem + col_s(g, buf), 0);
          const uint32_t more = __shfl_sync(0xffffffffu, i > i0 ? 1u : 0u, 0);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              tc_mma_f16_tmem_a(t_o, t_p + 8 * kk, desc_advance(dv, kk * 2048), idesc_pv, kk > 0 ? 1u : more);
            tc_commit(&bars->pv_done[g][buf]);
          }
          __syncwarp();
          ok = wait(bar(offsetof(QuantBars, pv_done), 2 * g + buf), (own >> 1) & 1u);
          if (!ok) break;
          ++own;
        }
        if (lane == 0) mbar_arrive(&bars->v_empty[vs]);
        if (++vs == S::kV) vs = 0, ++vturn;
      }
    }
  }
  if (warp & 1) {
    // every product completes before TMEM is released; after an abort some may be under way
    if (elect_one()) {
      tc_commit(&bars->drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bars->drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  }
  } else if (warp < 16) {
    // ----------------------------------------------------- softmax, epilogue
    const int g = (warp - 8) >> 2, wq = warp & 3, row = wq * 32 + lane;
    const int tok_row = row / p.tile_heads, head = row - tok_row * p.tile_heads;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    uint32_t own = 0, merges = 0, q = 0, qturn = 0, count = 0;
    bool ok = true;
    while (ok && await_item()) {
      const ChunkItem& I = bars->items[item_slot];  // (where it is: registers are short)
      const int nt = max(I.t1 - I.t0, 0);
      const bool two = two_tiles(p, I);
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
      float rs = 0.f;  // the row's scale, times the softmax's
      for (int x = 0; ok && nt > 0 && x < (two ? 2 : 1); ++x) {
        ok = wait(bar(offsetof(QuantBars, q_ready), q), qturn & 1u);
        if (!ok) break;
        if (x == g || !two) rs = sQS[q * kM + row] * p.scale_log2;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_empty[q]);
        if (++q == S::kQ) q = 0, ++qturn;
      }
      if (!ok) break;
      float m = valid ? -INFINITY : 0.f, l = 0.f;  // (l below 0: minus the sum times kSumFactor)
      const int step = two ? 1 : 2, keys_end = (I.tile0 + I.t1) * kN;
      int k0 = (I.tile0 + I.t0 + I.rot + (two ? 0 : g) - step) * kN;  // first key of the tile before
      for (int i = two ? 0 : g; i < nt; i += step) {  // (with one query tile the others are the other group's)
        k0 += step * kN;
        if (k0 >= keys_end) k0 -= nt * kN;
        const uint32_t buf = own & 1u, t_s = tmem + lanes + col_s(g, buf);
        ok = wait(bar(offsetof(QuantBars, s_full), 2 * g + buf), (own >> 1) & 1u);
        if (!ok) break;
        ++own;
        if (warp_valid) {
          tc_fence_after();
          const int c_lo = lo - k0, c_hi = hi - k0;
          const bool full = __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kN);
          if (!full) hide_scores(t_s, c_lo, c_hi);
          const Factors& factors = sFactors[(count + i) & (kScaleTiles - 1)];
          uint32_t w[kN / 2];
          float most, part;  // the largest sum of 32 of the tile's weights, and the sum of all over V's scales
          // weights of the tile, as fp16 pairs
          auto weights = [&](float nm) {
            most = part = 0.f;
            uint32_t v[2][16];
            tmem_ld16(t_s, v[0]);
            // all of the tile's at once, while the scores are on their way
            float f[kGroups], x0[kGroups];
#pragma unroll
            for (int n = 0; n < kGroups / 4; ++n) {
              const float4 a = factors.k[n], b = factors.log_v[n];
              f[4 * n] = fmaf(a.x, rs, kFactorMin), f[4 * n + 1] = fmaf(a.y, rs, kFactorMin);
              f[4 * n + 2] = fmaf(a.z, rs, kFactorMin), f[4 * n + 3] = fmaf(a.w, rs, kFactorMin);
              x0[4 * n] = b.x + nm, x0[4 * n + 1] = b.y + nm, x0[4 * n + 2] = b.z + nm, x0[4 * n + 3] = b.w + nm;
            }
            tmem_wait_ld(v[0]);
            float sums[kGroups];
#pragma unroll
            for (int c = 0; c < kN / 16; ++c) {
              if (c + 1 < kN / 16) tmem_ld16(t_s + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int n = 2 * c + h;
                const float2 f2 = make_float2(f[n], f[n]), x2 = make_float2(x0[n], x0[n]);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 8 * h; e < 8 * h + 8; e += 2) {
                  const float2 x = ffma2(make_float2(__uint_as_float(v[c & 1][e]), __uint_as_float(v[c & 1][e + 1])), f2, x2);
                  const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                  w[8 * c + e / 2] = pack_f16x2(pe.x, pe.y);
                  sum = e == 8 * h ? pe : fadd2(sum, pe);
                }
                sums[n] = sum.x + sum.y;
              }
              if (c + 1 < kN / 16) tmem_wait_ld(v[(c + 1) & 1]);
            }
#pragma unroll
            for (int n = 0; n < kGroups / 4; ++n) {
              const float4 r = factors.inverse[n];
              const float* x = sums + 4 * n;
              most = fmaxf(most, (x[0] + x[1]) + (x[2] + x[3]));
              part += fmaf(x[0], r.x, x[1] * r.y) + fmaf(x[2], r.z, x[3] * r.w);
            }
          };
          bool stale = __all_sync(0xffffffffu, m > -INFINITY), over = false;
#pragma unroll 1
          while (true) {
            if (stale) {
              weights(m == -INFINITY ? 0.f : -m);
              if (over) break;  // with the tile's own maximum
              over = __any_sync(0xffffffffu, valid && most > kWeightLimit);
              if (!over) break;
            }
            // the tile's own maximum: where weights were over the limit, out of the largest sum of 32, which is between
            // the largest and 2^5 times that; else out of the scores
            float ms = -INFINITY;
            const bool summed = stale && __all_sync(0xffffffffu, !valid || most < 0x1p120f);
            if (summed) ms = m + fast_log2(most) - kSumShift;
#pragma unroll 1
            for (int c = 0; !summed && c < kN / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(t_s + 32 * c, v);
              tmem_wait_ld(v);
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float mx = __uint_as_float(v[e]);
#pragma unroll
                for (int x = 1; x < 7; x += 2) mx = fmax3(mx, __uint_as_float(v[e + x]), __uint_as_float(v[e + x + 1]));
                mx = fmaxf(mx, __uint_as_float(v[e + 7]));
                // (the factor is positive)
                const int n = 4 * c + e / 8;
                ms = fmaxf(ms, fmaf(mx, fmaf(reinterpret_cast<const float*>(factors.k)[n], rs, kFactorMin),
                                    reinterpret_cast<const float*>(factors.log_v)[n]) - kShift);
              }
            }
            float alpha = 1.f;
            if (valid && ms > -INFINITY) {
              if (m == -INFINITY) {
                m = ms;
              } else if (ms > (stale ? m : m + kRaise)) {
                // (a maximum left below a row's weights' limit would do every tile twice)
                alpha = fast_exp2(m - ms);
                m = ms;
              }
            }
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
              // the product of the tile before (own counts this one already) is under way
              ok = wait(bar(offsetof(QuantBars, pv_done), 2 * g + ((own - 2) & 1u)), ((own - 2) >> 1) & 1u);
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
            stale = over = true;
          }
          if (!ok) break;
          l = fmaf(part, l < 0.f ? -kSumFactor : 1.f, l);
          if (l > kSumHigh) l *= -kSumFactor;
          tmem_st32(t_s, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
        }
        // warps without rows leave what is there: only rows that are not stored read it
        if (lane == 0) mbar_arrive(&bars->p_full[g][buf]);
      }
      if (!ok) break;
      count += nt;
      const bool other = !two && nt > 1;  // group 1 has tiles of the same rows
      if (g == 1 && !two) {
        if (nt < 2) {
          leave_item();
          continue;
        }
        ok = wait(bar(offsetof(QuantBars, pv_done), 2 + ((own - 1) & 1u)), ((own - 1) >> 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        sML[row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ml_ready);
        // group 0 has read this group's output: its accumulator may be written again
        ok = wait(bar(offsetof(QuantBars, merged)), merges & 1u);
        tc_fence_after();
        ++merges;
        leave_item();
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      if (nt > 0) {
        ok = wait(bar(offsetof(QuantBars, pv_done), 2 * g + ((own - 1) & 1u)), ((own - 1) >> 1) & 1u);
        if (!ok) break;
      }
      if (other) {
        ok = wait(bar(offsetof(QuantBars, ml_ready)), merges & 1u);
        if (!ok) break;
        const float2 b = sML[row];
        const float top = fmaxf(m, b.x), at = top == -INFINITY ? 0.f : top;
        f0 = exp2f(m - at);
        f1 = exp2f(b.x - at);
        float l1 = b.y;
        if (l < 0.f || l1 < 0.f) {  // both as the one that is held times the factor
          if (l > 0.f) l *= -kSumFactor;
          if (l1 > 0.f) l1 *= -kSumFactor;
        }
        l = l * f0 + l1 * f1;
        m = top;
      }
      tc_fence_after();
      const float inv = l != 0.f ? (l < 0.f ? -kSumFactor : 1.f) / l : 0.f;
      const float lse2 = l != 0.f ? m + (log2f(fabsf(l)) + (l < 0.f ? kSumLog : 0.f)) : -INFINITY;
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
        if (*static_cast<volatile const int*>(&bars->nan[item_slot]) != 0) {
          const int tok = I.first_tok + tok0 + tok_row;
          const KeyRange shared = shared_keys(p, I), k = chunk_keys(p, I.qo, I.kv, tok, tok + 1);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t bad = nan_columns(p, I.pbase, I.h / p.group, max(k.lo, (I.tile0 + I.t0) * kN),
                                       min(k.hi, (I.tile0 + I.t1) * kN), KeyRange{shared.lo + kN, shared.hi - kN}, c);
            for (int e = 16 * c; bad != 0; bad >>= 1, ++e) {
              if ((bad & 1u) == 0) continue;
              if (slot >= 0) p.part_o[(slot * p.rows + mrow) * D + e] = __uint_as_float(kNan);
              else if (p.o_dtype == PD_BF16) static_cast<uint16_t*>(p.o)[orow * D + e] = (uint16_t)kNan;
              else static_cast<float*>(p.o)[orow * D + e] = __uint_as_float(kNan);
            }
          }
        }
      }
      tc_fence_before();
      leave_item();
      if (other) {
        if (lane == 0) mbar_arrive(&bars->merged);
        ++merges;
      }
    }
  } else {
    // ------------------------------------------- q to two e4m3 terms, V to fp16
    // A thread takes 16 values of a row, and of every kStep-th row on: chunks c and c + 1 of the
    // row's 8-value chunks, at the same place of the swizzle each time.
    const int t = threadIdx.x - 512;
    constexpr int kRow = D / 16, kStep = 128 / kRow, kUnits = kN / kStep;
    static_assert(kStep % 8 == 0, "whole swizzles");
    const int row0 = t / kRow, j = t % kRow, c = 2 * (j % 4);
    const uint32_t from0 = base32 + S::kOffC + t * 16;
    const uint32_t to0 = base32 + S::kOffV + (j / 4) * S::kVHalf + row0 * 128;
    const uint32_t to_a = to0 + ((c ^ (row0 & 7)) << 4), to_b = to0 + (((c + 1) ^ (row0 & 7)) << 4);
    uint32_t q = 0, qturn = 0, cs = 0, cturn = 0, vs = 0, vturn = 0;
    bool ok = true;
    ChunkItem I;
    while (ok) {
      volatile int* nan = &bars->nan[item_slot];  // (the softmax warps keep the item until all of its V is used)
      if (!next_item(I)) break;
      const int nt = I.t1 - I.t0;
      if (nt <= 0) continue;
      const KeyRange shared = shared_keys(p, I);
      const int tiles = two_tiles(p, I) ? 2 : 1;
      for (int x = 0; ok && x < tiles; ++x) {
        ok = wait(bar(offsetof(QuantBars, q_full), q), qturn & 1u);
        if (!ok) break;
        sQS[q * kM + t] = split_row<D>(base32 + q * S::kQTile, t);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_ready[q]);
        if (++q == S::kQ) q = 0, ++qturn;
      }
      int tile = I.tile(0);
      const int end = I.tile0 + I.t1;
      for (int i = 0; ok && i < nt; ++i) {
        ok = wait(bar(offsetof(QuantBars, c_full), cs), cturn & 1u);
        if (!ok) break;
        uint4 v[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) v[u] = ld_shared(from0 + cs * S::kCodes + u * (kStep * D));
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->c_empty[cs]);
        const int k0 = tile * kN;
        if (++tile == end) tile = I.tile0 + I.t0;
        if (k0 < shared.lo || k0 + kN > shared.hi) {
          // a weight of 0 would not hide a NaN: none of keys that no row sees, and none for now of the others
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            const int key = k0 + u * kStep + row0;
            if (key < I.keys.lo || key >= I.keys.hi) v[u] = make_uint4(0u, 0u, 0u, 0u);
          }
          if (clear_nan(v)) *nan = 1;
        }
        ok = wait(bar(offsetof(QuantBars, v_empty), vs), (vturn & 1u) ^ 1u);
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          uint32_t w[8];
          to_f16(v[u], w);
          const uint32_t at = vs * S::kVTile + u * (kStep * 128);
          st_shared(to_a + at, make_uint4(w[0], w[1], w[2], w[3]));
          st_shared(to_b + at, make_uint4(w[4], w[5], w[6], w[7]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_full[vs]);
        if (++cs == S::kC) cs = 0, ++cturn;
        if (++vs == S::kV) vs = 0, ++vturn;
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
  const cudaError_t e = allow_smem<chunk_quant_tc_kernel<D, POW2>>(QuantShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_quant_tc_kernel<D, POW2>, dim3((unsigned)p.grid), kCqThreads, QuantShape<D>::kSmem, stream,
                          tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_chunk_quant_tc(const ChunkParams& p, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const int pb = page_box(p.page_size);
  if (!make_rows_map(&tq, p.q, PD_BF16, p.total_qo, p.hq, p.head_dim, 64, p.tile_tokens, true, p.tile_heads,
                     p.q_stride) ||
      !make_code_map(&tk, p.k_pool, p.num_pages, p.hkv, p.page_size, p.head_dim, pb, true, p.nhd != 0) ||
      !make_code_map(&tv, p.v_pool, p.num_pages, p.hkv, p.page_size, p.head_dim, pb, false, p.nhd != 0))
    return cudaErrorInvalidValue;
  last_kernel() = "chunk_quant_tc_kernel";
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
