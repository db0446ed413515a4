// pd_chunk_quant_rows.cu -- chunk attention over a cache held in 8 bits, for few query
// rows (single tokens, a drafted one or two; bf16 queries, pages and blocks of a multiple of 8 tokens).
//
// An item has at most 8 query rows (tokens x heads of a KV head), and its keys pass once, so the cache's bytes
// are the floor. Tiles of 128 rows through tensor memory would keep 8 of them busy at most, a
// softmax warp of 4 and every wait between the roles for them; so here a warp does all of it by itself,
// with products of 8 columns (mma.m16n8k16, fp16 in, fp32 out) that are the query rows, and the CTA's warps
// meet at an item's end only:
//   32 keys a warp in turn, in two halves that do not wait for one another: their 8-bit rows come through a ring of
//     its own in shared memory by cp.async, the scales of their four 8-key groups with them;
//   scores, K q^T: q as fp16 (scaled by a power of two a row, so that its largest lies in (224, 448]; exact but for
//     values under 2^-25 of the largest, off by 2^-32 of it at most), k as fp16 by one conversion a pair, exact. The
//     products' inner index may be any order of the head's values, so a lane takes 16 neighbouring bytes of a key and not
//     2 here and there;
//   weights W = 2^(s + log2 b - m), b the key's scale of V and m the row's running maximum of s + log2 b, fp16 with
//     the largest from 2^4 to 2^12: only a score over that raises m, and has the lanes' maxima
//     exchanged. Their sum over b, in fp32, is the softmax's;
//   o, V^T W: the weights' 8 x 8 blocks turned by movmatrix; a lane takes 16 neighbouring values of 4 keys, and a byte
//     of two keys is one pair.
// An item's first copies are under way while the outputs of the one before are joined (139 us of the case below, 144
// after them).
//
// 128 requests of 512 to 4096 keys, 32 query and 8 KV heads of 128: 104 us, 5.4 TB/s; the cache's bytes take 84 at the
// copy rate. What holds it is each warp's chain from a key's bytes to its weights, at 2 warps a scheduler of 232
// registers (1.6 instructions a cycle and SM; 27 % of the stalls wait for the instruction before, 24 % for global memory, what
// an item's start reads above all). One half a turn and 12 warps took 132; a page's id looked at in the turn that reads it 116 for 109; one CTA
// of 8 warps 109 for 104, of 6 and 7 128 and 119 for 117; three turns in the ring 105; the next item looked up while one is
// worked off 104. D 64 fits three CTAs: 78 us with two of them, 68 with three (103 where the SMs had kept
// less shared memory from the kernel before). (With the rows as the 16 of the products, half of them empty, a turn took twice the
// products and registers: 210.)
#include <math.h>

#include "pd_chunk.cuh"
#include "pd_chunk_quant.cuh"
#include "pd_launch.cuh"
#include "pd_quant.cuh"
#include "pd_tc.cuh"

namespace pd {

namespace {

constexpr int kRqHalves = 2;              // of a warp's turn, 16 keys each: while one waits, the other is worked on
constexpr int kRqKeys = 16 * kRqHalves;
constexpr int kRqGroups = kRqKeys / 8;    // of 8 keys
constexpr float kRqShift = 4.0f, kRqRaise = 12.0f;

template <int D>
struct RowsQuantShape {
  static constexpr int kRows = 8;
  static constexpr int kWarps = 4, kThreads = 32 * kWarps;
  static constexpr int kCtas = rows_quant_ctas(D);                // of an SM
  static constexpr int kSpan = kWarps * kRqKeys;                  // keys of the CTA's turn
  static constexpr int kStages = 2;
  static constexpr int kCodes = kRqKeys * D;                      // K or V of a warp's keys
  static constexpr int kStage = 2 * kCodes + 8 * kRqGroups;       // and the groups' scales
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kJoin = kRows * D * 4;                     // a warp's output
  static constexpr int kRing = kWarps * kWarp;
  static constexpr size_t kSmem = kRing + kWarps * kJoin + 2 * kWarps * kRows * sizeof(float);
  static_assert(kSelfBytes <= kRing && kCtas * (kSmem + 1024) <= 233472, "shared memory of an SM");
};

// An 8 x 8 block of 16-bit values, two of a row a lane, turned.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's bytes from global to shared memory, asynchronously; zeros where not `there`.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool there) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(there ? BYTES : 0)
                 : "memory");
}

// Two bf16 of eight.
__device__ __forceinline__ uint32_t q_pair(uint4 v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Where 16-byte chunk `c` of a key's row lies in a stage, so that the lanes that read together meet in no bank (of
// V with D = 64 two do).
template <int D>
__device__ __forceinline__ int k_chunk(int key, int c) { return D == 128 ? c ^ (key & 1) << 2 : c; }
template <int D>
__device__ __forceinline__ int v_chunk(int key, int c) { return D == 128 ? c ^ (key >> 1 & 3) << 1 : c ^ (key >> 1 & 3); }

}  // namespace

// SINGLE: calls of at most one token a request. Rows of one token see the same keys, so no NaN of V has to be kept
// from any of them (without the code for that four short requests take 6.2 us for 6.5, 128 decodes 102.9 for 103.7).
template <int D, bool SINGLE>
__global__ void __launch_bounds__(RowsQuantShape<D>::kThreads, RowsQuantShape<D>::kCtas) chunk_quant_rows_kernel(const ChunkParams p) {
  using S = RowsQuantShape<D>;
  constexpr int kTiles = D / 16;       // of 16 values of the output
  constexpr int kChunks = D / 16;      // 16-byte chunks of a row
  constexpr int kPer = kRqKeys * kChunks / 32;  // chunks of K (or V) that a lane copies
  extern __shared__ __align__(128) uint8_t rq_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(rq_smem) + warp * S::kWarp;
  float* sAcc = reinterpret_cast<float*>(rq_smem + S::kRing);     // [warp][row][D]
  float* sM = sAcc + S::kWarps * S::kRows * D;                    // [warp][row] maxima, then sums
  float* sL = sM + S::kWarps * S::kRows;
  pdl_launch_dependents();
  pdl_wait_primary();
  ChunkWalk walk;
  {
    const ChunkLine line = take_line(p, rq_smem);
    const int4 cut = walk.begin(p, line, blockIdx.x);
    if (tid == 0) p.cuts[blockIdx.x] = cut;
  }
  const int blocks = p.page_size / p.scale_block, block_shift = 31 - __clz(p.scale_block);
  // What a lane copies of a turn's keys: 16-byte chunk `chunk` of key key0 and of every kStep-th from there on, kEach
  // of each group of 8; where from, after the group's first row, and where to in a stage. (K's place in the swizzle is the
  // same for all of them, V's for every other.)
  constexpr int kStep = 32 / kChunks, kEach = kPer / kRqGroups;
  const uint8_t* k_pool = static_cast<const uint8_t*>(p.k_pool);
  const uint8_t* v_pool = static_cast<const uint8_t*>(p.v_pool);
  const int key0 = lane / kChunks, chunk = lane % kChunks, row_step = p.nhd ? p.hkv : 1;
  const int64_t from0 = (int64_t)key0 * row_step * D + chunk * 16, step = (int64_t)kStep * row_step * D;
  const uint32_t to_k = key0 * D + k_chunk<D>(key0, chunk) * 16;
  const uint32_t to_v[2] = {(uint32_t)(S::kCodes + key0 * D + v_chunk<D>(key0, chunk) * 16),
                            (uint32_t)(S::kCodes + key0 * D + v_chunk<D>(key0 + kStep, chunk) * 16)};
  __syncthreads();  // the line has been read
  ChunkItem I{};
  int kv_head = 0, first = 0, last = 0;  // of the item: its KV head, the warp's first key, the end
  uint4 raw[D / 64][2];                  // row g's values 16 c and on of each 64
  // A warp's keys from k0 on are groups of 8, a run of slots of one page each; lane n has group n % kRqGroups: its page's
  // id, read a turn ahead and looked at only where it is used, then its first row in the pools and its block of the
  // scales (-1: no row of the item sees it).
  struct Group {
    int64_t row, block;
  };
  auto group_key = [&](int k0) { return k0 + 8 * (lane & (kRqGroups - 1)); };
  auto seen = [&](int j) { return j + 8 > I.keys.lo && j < I.keys.hi; };
  auto read_page = [&](int k0) {
    const int j = group_key(k0);
    return seen(j) ? __ldg(p.page_indices + I.pbase + (p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size)) : 0;
  };
  auto place = [&](int page, int k0) -> Group {
    const int j = group_key(k0);
    if (!seen(j)) return Group{-1, -1};
    if (page < 0 || page >= p.num_pages) {
      report(p.status, PD_DEV_BAD_PAGE_TABLE);
      return Group{-1, -1};
    }
    const int slot = p.page_shift >= 0 ? j & (p.page_size - 1) : j % p.page_size;
    const int64_t head = (int64_t)page * p.hkv + kv_head;
    return Group{p.nhd ? ((int64_t)page * p.page_size + slot) * p.hkv + kv_head : head * p.page_size + slot,
                 head * blocks + (p.page_shift >= 0 ? slot >> block_shift : slot / p.scale_block)};
  };
  // Starts the copies of the keys from k0 on into a stage; those that no row of the item sees become zeros.
  auto fetch = [&](const Group& at, int k0, int stage) {
    const uint32_t to = ring + stage * S::kStage;
    int64_t r[kRqGroups];
    bool all = true;
#pragma unroll
    for (int n = 0; n < kRqGroups; ++n) {
      r[n] = __shfl_sync(0xffffffffu, at.row, n);
      all = all && r[n] >= 0;
    }
    if (k0 >= I.keys.lo && k0 + kRqKeys <= I.keys.hi && all) {
#pragma unroll
      for (int n = 0; n < kRqGroups; ++n) {
        const int64_t from = r[n] * D + from0;
        const uint8_t *k = k_pool + from, *v = v_pool + from;
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
          const int i = n * kEach + x;
          copy_async<16>(to + to_k + i * (kStep * D), k + x * step, true);
          copy_async<16>(to + to_v[i & 1] + i * (kStep * D), v + x * step, true);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int key = key0 + i * kStep;
        const int64_t base = r[i / kEach];
        const bool there = base >= 0 && k0 + key >= I.keys.lo && k0 + key < I.keys.hi;
        const int64_t from = there ? (base + (int64_t)((key & 7) * row_step)) * D + chunk * 16 : 0;
        copy_async<16>(to + to_k + i * (kStep * D), k_pool + from, there);
        copy_async<16>(to + to_v[i & 1] + i * (kStep * D), v_pool + from, there);
      }
    }
    if (lane < 2 * kRqGroups)  // K's scales of the groups, and V's
      copy_async<4>(to + 2 * S::kCodes + 4 * lane, (lane < kRqGroups ? p.k_scale : p.v_scale) + (at.block >= 0 ? at.block : 0),
                    at.block >= 0);
  };
  int page = 0;  // of the turn that is fetched next
  // The walk's next item: starts its first turns' copies, and reads q. False: there is none.
  auto start = [&]() -> bool {
    if (!walk.next(p, I)) return false;
    kv_head = I.h / p.group;
    first = (I.tile0 + I.t0) * kChunkKeys + warp * kRqKeys;
    last = (I.tile0 + I.t1) * kChunkKeys;
    page = read_page(first);
    const int tok = g / p.tile_heads;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        raw[h][e] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < I.tokens)
          raw[h][e] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                           (int64_t)(I.q0 + tok) * p.q_stride +
                                                           (int64_t)(I.h + g - tok * p.tile_heads) * D + 64 * h + 16 * c) + e);
      }
    __syncwarp();  // the last item's stages have been read
#pragma unroll 1
    for (int i = 0; i < S::kStages - 1; ++i) {
      const int k0 = first + i * S::kSpan;
      if (k0 < last) fetch(place(page, k0), k0, i);
      asm volatile("cp.async.commit_group;" ::: "memory");
      page = read_page(k0 + S::kSpan);
    }
    return true;
  };
  bool more = start();
  while (more) {
    const int rows = I.tokens * p.tile_heads;
    // q as fp16, scaled
    uint32_t q[D / 8];
    float rs[2];        // of rows 2 c and the next: what a score is multiplied by for base-2 exponents
    int lo[2], hi[2];
    // keys that every row sees (rows that are not there see all, and are not stored)
    int all_lo = 0, all_hi = 0x7fffffff;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint32_t w = q_pair(raw[i / 8][i / 4 % 2], i % 4);
      top = fmaxf(top, fmaxf(fabsf(bf16_lo(w)), fabsf(bf16_hi(w))));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool finite = top <= 3.4e38f;  // an infinity makes all of the row NaN
    const int ex = scale_exponent(finite ? top : 0.f);
    const float f = finite ? power_of_two(-ex) : __uint_as_float(0x7fffffffu);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint32_t w = q_pair(raw[i / 8][i / 4 % 2], i % 4);
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q[i]) : "f"(bf16_hi(w) * f), "f"(bf16_lo(w) * f));
    }
    const float scaled = power_of_two(ex) * p.scale_log2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      rs[e] = __shfl_sync(0xffffffffu, scaled, 4 * (2 * c + e));
      const int row = 2 * c + e, t = I.first_tok + row / p.tile_heads;
      const KeyRange k = chunk_keys(p, I.qo, I.kv, t, t + 1);
      lo[e] = k.lo;
      hi[e] = k.hi;
      if (row < rows) {
        all_lo = max(all_lo, k.lo);
        all_hi = min(all_hi, k.hi);
      }
    }
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);
    float o[kTiles][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float sum_log = 0.f;  // kSumLog once a sum of the warp's is held times kSumFactor: all of them then
    bool nan = false;
    int stage = 0;
#pragma unroll 1
    for (int k0 = first; k0 < last; k0 += S::kSpan) {
      const int ahead = k0 + (S::kStages - 1) * S::kSpan;
      __syncwarp();  // the stage that is filled next has been read
      if (ahead < last) fetch(place(page, ahead), ahead, stage == 0 ? S::kStages - 1 : stage - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      page = read_page(ahead + S::kSpan);
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
      __syncwarp();  // the other lanes' copies too
      const uint32_t from = ring + stage * S::kStage;
      if (++stage == S::kStages) stage = 0;
      const bool masked = k0 < all_lo || k0 + kRqKeys > all_hi;
      if (!SINGLE && masked && rows > p.tile_heads) {
#pragma unroll 1
        for (uint32_t at = from + S::kCodes + 16 * lane; at < from + 2 * S::kCodes; at += 512) {
          uint4 v[1];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w)
                       : "r"(at)
                       : "memory");
          if (!clear_nan(v)) continue;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w)
                       : "memory");
          nan = true;
        }
        __syncwarp();
      }
      float a[kRqGroups], sv[kRqGroups];  // the groups' scales of K and V
#pragma unroll
      for (int n = 0; n < kRqGroups; n += 4) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(a[n]), "=f"(a[n + 1]), "=f"(a[n + 2]), "=f"(a[n + 3])
                     : "r"(from + 2 * S::kCodes + 4 * n)
                     : "memory");
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(sv[n]), "=f"(sv[n + 1]), "=f"(sv[n + 2]), "=f"(sv[n + 3])
                     : "r"(from + 2 * S::kCodes + 4 * (kRqGroups + n))
                     : "memory");
      }
      // scores of keys 16 x + g and 16 x + g + 8 with rows 2 c and the next
      float s[kRqHalves][4];
#pragma unroll
      for (int x = 0; x < kRqHalves; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][e] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t k[2 * kRqHalves][8];
#pragma unroll
        for (int n = 0; n < 2 * kRqHalves; ++n) {
          const int key = 8 * n + g;
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(from + key * D + k_chunk<D>(key, 4 * h + c) * 16)
                       : "memory");
          to_f16(v, k[n]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < kRqHalves; ++x)
            mma_16816(s[x], k[2 * x][2 * i], k[2 * x + 1][2 * i], k[2 * x][2 * i + 1], k[2 * x + 1][2 * i + 1],
                      q[8 * h + 2 * i], q[8 * h + 2 * i + 1]);
      }
      float lb[kRqGroups];
#pragma unroll
      for (int n = 0; n < kRqGroups; ++n) {
        a[n] = fmaxf(a[n], kScaleMin);
        lb[n] = fast_log2(fmaxf(sv[n], kScaleMin));
      }
      float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int n = 0; n < kRqGroups; ++n) {
          // (the factor is not 0: a tiny one stays a number)
          float& y = s[n >> 1][2 * (n & 1) + e];
          y = fmaf(y, fmaf(a[n], rs[e], 1e-37f), lb[n]);
          if (masked) {
            const int j = k0 + 8 * n + g;
            if (j < lo[e] || j >= hi[e]) y = -INFINITY;
          }
          best[e] = fmaxf(best[e], y);
        }
      }
      if (__any_sync(0xffffffffu, best[0] > m[0] + kRqRaise || best[1] > m[1] + kRqRaise || fmaxf(l[0], l[1]) > kSumHigh)) {
        if (__any_sync(0xffffffffu, fmaxf(l[0], l[1]) > kSumHigh)) {
          l[0] *= kSumFactor;
          l[1] *= kSumFactor;
          sum_log = kSumLog;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], d));
          if (best[e] > m[e] + kRqRaise) {
            const float alpha = fast_exp2(m[e] - (best[e] - kRqShift));  // (0 for the first)
            m[e] = best[e] - kRqShift;
            l[e] *= alpha;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              o[t][e] *= alpha;
              o[t][2 + e] *= alpha;
            }
          }
        }
      }
      uint32_t w[kRqGroups];
      const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
      for (int n = 0; n < kRqGroups; ++n) {
        const float inverse = inverse_scale(lb[n] + sum_log);
        const float w0 = fast_exp2(s[n >> 1][2 * (n & 1)] - b0), w1 = fast_exp2(s[n >> 1][2 * (n & 1) + 1] - b1);
        l[0] = fmaf(w0, inverse, l[0]);
        l[1] = fmaf(w1, inverse, l[1]);
        uint32_t pair;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pair) : "f"(w1), "f"(w0));
        w[n] = turned(pair);
      }
      // values: rows of a half's keys 2 c, 2 c + 1, 2 c + 8 and 2 c + 9, values D / 8 g and on
#pragma unroll
      for (int x = 0; x < kRqHalves; ++x) {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 16 * x + 2 * c + (i & 1) + 8 * (i >> 1), byte = (D / 8) * g;
          const uint32_t at = from + S::kCodes + key * D + v_chunk<D>(key, byte >> 4) * 16 + (byte & 15);
          if constexpr (D == 128)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                         : "r"(at)
                         : "memory");
          else
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(at) : "memory");
        }
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t a[4], b[4];  // of four values, of keys 2 c and 2 c + 1, and of the other two
          pairs_to_f16(__byte_perm(v[0][e], v[1][e], 0x5140), __byte_perm(v[0][e], v[1][e], 0x7362), a);
          pairs_to_f16(__byte_perm(v[2][e], v[3][e], 0x5140), __byte_perm(v[2][e], v[3][e], 0x7362), b);
#pragma unroll
          for (int t = 0; t < 2; ++t) mma_16816(o[2 * e + t], a[2 * t], a[2 * t + 1], b[2 * t], b[2 * t + 1], w[2 * x], w[2 * x + 1]);
        }
      }
    }
    if (!SINGLE && __any_sync(0xffffffffu, nan)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // columns D / 8 g and on; turns of 32 keys inside [all_lo, all_hi) were multiplied as they are
        const uint32_t bad = nan_columns(p, I.pbase, kv_head, max(lo[e], (I.tile0 + I.t0) * kChunkKeys), min(hi[e], last),
                                         KeyRange{all_lo + kRqKeys, all_hi - kRqKeys}, D / 8 * g / 16) >>
                             (D / 8 * g % 16);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (bad >> 2 * t & 1u) o[t][e] = __uint_as_float(kNan);
          if (bad >> (2 * t + 1) & 1u) o[t][2 + e] = __uint_as_float(kNan);
        }
      }
    }
    const int64_t part = part_slot(I, blockIdx.x);
    const int64_t q0 = I.q0;
    const int h0 = I.h;
    more = start();   // its copies are under way while the warps' outputs are joined
    __syncthreads();  // the last item's outputs have been read
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 2 * c + e;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
      if (g == 0) {
        sM[warp * S::kRows + row] = m[e];
        sL[warp * S::kRows + row] = sum_log == 0.f ? l[e] : -l[e];
      }
      // tile t has values D / 8 g + 2 t and the next
      float* to = sAcc + (warp * S::kRows + row) * D + (D / 8) * g;
#pragma unroll
      for (int t = 0; t < kTiles; t += 2)
        *reinterpret_cast<float4*>(to + 2 * t) = make_float4(o[t][e], o[t][2 + e], o[t + 1][e], o[t + 1][2 + e]);
    }
    __syncthreads();
    // the warps' outputs of 4 columns of a row
    for (int i = tid; i < rows * (D / 4); i += S::kThreads) {
      const int r = i / (D / 4), col = 4 * (i - r * (D / 4));
      float top = -INFINITY, sum = 0.f, least = 0.f;
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        top = fmaxf(top, sM[w * S::kRows + r]);
        least = fminf(least, sL[w * S::kRows + r]);
      }
      const float plain = least < 0.f ? kSumFactor : 1.f;  // what sums held as they are are multiplied by
      const float base = top == -INFINITY ? 0.f : top;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        const float f = fast_exp2(sM[w * S::kRows + r] - base);
        const float4 a = *reinterpret_cast<const float4*>(sAcc + (w * S::kRows + r) * D + col);
        const float l = sL[w * S::kRows + r];
        sum = fmaf(l < 0.f ? -l : l * plain, f, sum);
        y.x = fmaf(a.x, f, y.x);
        y.y = fmaf(a.y, f, y.y);
        y.z = fmaf(a.z, f, y.z);
        y.w = fmaf(a.w, f, y.w);
      }
      const float inv = sum != 0.f ? plain / sum : 0.f;
      y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      const int tok = r / p.tile_heads;
      const int64_t row = (q0 + tok) * p.hq + h0 + r - tok * p.tile_heads;
      if (part < 0 && p.o_dtype == PD_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + col) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      else
        *reinterpret_cast<float4*>((part < 0 ? static_cast<float*>(p.o) + row * D : p.part_o + (part * p.rows + r) * D) +
                                   col) = y;
      if (col == 0) {
        const float lse2 = sum != 0.f ? top + (log2f(sum) + (least < 0.f ? kSumLog : 0.f)) : -INFINITY;
        if (part >= 0) p.part_lse[part * p.rows + r] = lse2;
        else if (p.lse != nullptr) p.lse[row] = lse2 * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------------- host
namespace {

template <int D, bool SINGLE>
cudaError_t launch_rows(const ChunkParams& p, cudaStream_t stream) {
  const cudaError_t e = allow_smem<chunk_quant_rows_kernel<D, SINGLE>, true>(RowsQuantShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_quant_rows_kernel<D, SINGLE>, dim3((unsigned)p.grid), RowsQuantShape<D>::kThreads,
                          RowsQuantShape<D>::kSmem, stream, p);
}

}  // namespace

cudaError_t launch_chunk_quant_rows(const ChunkParams& p, cudaStream_t stream) {
  last_kernel() = "chunk_quant_rows_kernel";
  profile_begin(stream);
  cudaError_t e;
  if (p.max_qo_len <= 1) e = p.head_dim == 64 ? launch_rows<64, true>(p, stream) : launch_rows<128, true>(p, stream);
  else e = p.head_dim == 64 ? launch_rows<64, false>(p, stream) : launch_rows<128, false>(p, stream);
  profile_end(stream);
  return e;
}

}  // namespace pd
