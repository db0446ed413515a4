// pd_chunk.cu -- attention of a chunk of new tokens over a paged KV cache: the
// plan of the work line, the kernel for fp32 and for pages that the tensor-core
// kernel does not take, and the merge of items cut between CTAs.
//
// Sections "Prefill vs Decode performance" (attention parallelises over requests
// and over the KV length) and "Qwen3-Coder" (grouped-query heads). For token i
// of n new ones at position t = kv_len - n + i and a query head h on KV head
// h / group, over the keys j < kv_len with j <= t (causal) and j >= t - window:
//   s_j = scale <q_ih, k_j>,  o_ih = sum_j softmax(s)_j v_j,  lse = ln sum_j e^{s_j}
// and o = 0, lse = -inf where no key is left.
#include <math.h>

#include "pd_chunk.cuh"
#include "pd_chunk_quant.cuh"
#include "pd_launch.cuh"
#include "pd_quant.cuh"

namespace pd {

namespace {

constexpr int kPlanThreads = 1024;

}  // namespace

// ------------------------------------------------------------------- plan
// One CTA makes the line of a batch that is too large for every CTA to make its own.
__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(const ChunkParams p) {
  __shared__ long long warp_tot[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait_primary();
  const ChunkLine line = plan_line<kPlanThreads>(p, p.req_first, p.pre, p.pos, warp_tot);
  if (threadIdx.x == 0) {
    p.hdr[0] = line.rem;
    p.hdr[1] = line.head;
    p.hdr[2] = line.base;
    p.hdr[3] = line.parts;
    p.hdr[4] = line.whole;
    p.hdr[5] = line.shares;
  }
}

// ------------------------------------------------------------------ merge
// o and lse of the items that the line's cuts fell into: block x has the item
// that part x begins and does not end, if there is one. One warp a row, its lanes
// the parts' sums. Bound by its launch, a chain of three reads and the parts it reads
// from L2 (500 tokens over 32700, cut in 216 pieces of 131 KB: 8 us behind the
// kernel's 162; 13 with a part's sum and output read one after the other).
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkParams p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int c = blockIdx.x;
  const int4 cut = p.cuts[c];  // {row of the first token, rows, query head, last part}
  const int rows = cut.y, last = cut.w;
  if (last <= c) return;
  const int lane = threadIdx.x & 31;
  constexpr int E = D / 32;
  for (int m = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); m < rows;
       m += gridDim.y * (kMergeThreads / 32)) {
    float best = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int x0 = c; x0 <= last; x0 += 32) {
      // 32 parts' sums, a lane each; an empty part has none
      const int mine = x0 + lane;
      const bool there = mine == c || (mine <= last && p.cuts[mine].y >= 0);
      const float lse = there ? p.part_lse[(2 * (int64_t)mine + (mine == c ? 1 : 0)) * p.rows + m] : -INFINITY;
      float top = lse;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(top, best);
      const float base = top == -INFINITY ? 0.f : top;  // (no part has a key yet: every factor is 0)
      const float old = exp2f(best - base), f = exp2f(lse - base);
      best = top;
      float part = f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
      sum = sum * old + part;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= old;
      const int parts = min(32, last - x0 + 1);
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        if (w == 0.f) continue;
        const int x = x0 + i;
        const float* o = p.part_o + ((2 * (int64_t)x + (x == c ? 1 : 0)) * p.rows + m) * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(o);
          acc[0] += w * v.x;
          acc[1] += w * v.y;
          acc[2] += w * v.z;
          acc[3] += w * v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(o);
          acc[0] += w * v.x;
          acc[1] += w * v.y;
        }
      }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int tok = m / p.tile_heads;
    const int64_t row = (int64_t)(cut.x + tok) * p.hq + cut.z + (m - tok * p.tile_heads);
    if (p.o_dtype == PD_BF16) {
      uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * D + lane * E);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) o[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    } else {
      float* o = static_cast<float*>(p.o) + row * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = acc[e] * inv;
    }
    if (lane == 0 && p.lse != nullptr) p.lse[row] = sum != 0.f ? (best + log2f(sum)) * kLn2 : -INFINITY;
  }
}

// ----------------------------------------------------------------- kernel
// fp32 arithmetic on the CUDA cores: R query rows (tokens x heads of a KV head)
// against tiles of 64 keys, K then V of a tile in one shared buffer as fp32.
// 256 threads as 16 x 16: a thread has R / 16 rows and every 16th key of the
// scores, the same rows and D / 16 columns of the output; a row's maximum and
// sum go over its 16 lanes by shuffles. Bound by the fp32 pipes and the shared
// memory that feeds them: 4 x 512 tokens over 4096, 32 / 8 heads, run at 30.6
// TFLOP/s for D 64 and 27 for D 128, two CTAs an SM (one, with the 180 to 230
// registers that a thread would take: 21 and 25; the 128 of D 128 spill a little).
constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = kChunkKeys;

template <int R, int D>
constexpr size_t simt_smem() {
  return sizeof(float) * (size_t)(R * (D + 4) + kSimtKeys * (D + 4) + kSimtKeys * (R + 4));
}

// QUANT: pools of 8-bit values with block scales (the value enters the tile as fp32, times its scale): fp32 queries, and
// pages or blocks that are not of whole groups of 8 tokens. Its 64 keys a tile cost the same arithmetic whatever they
// were held in, so it is bound as above, or, with few rows, by the keys' way through registers and shared memory: 32 / 8
// heads of 128, 64 decodes of 2048 keys 396 us in fp32 and 409 in bf16 over pages of 6, 4 x 512 tokens 340
// and 341 (the kernels for bf16 over pages of 16: 57 and 43).
template <typename T, int R, int D, bool QUANT>
__global__ void __launch_bounds__(kSimtThreads, 2) chunk_simt_kernel(const ChunkParams p) {
  constexpr int RT = R / 16, LD = D + 4, LP = R + 4, CT = D / 64;  // CT: float4 columns of a thread
  extern __shared__ float4 simt_smem_raw[];
  float* sQ = reinterpret_cast<float*>(simt_smem_raw);
  float* sKV = sQ + R * LD;
  float* sP = sKV + kSimtKeys * LD;  // [key][row]
  pdl_launch_dependents();
  pdl_wait_primary();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  ChunkWalk walk;
  {
    const ChunkLine line = take_line(p, simt_smem_raw);
    const int4 cut = walk.begin(p, line, blockIdx.x);
    if (tid == 0) p.cuts[blockIdx.x] = cut;
  }
  constexpr int VE = 16 / sizeof(T), VR = D / VE;  // elements of a 16-byte vector, vectors of a row
  constexpr int KE = QUANT ? 16 : VE, KR = D / KE;     // the same of the pools' rows
  constexpr int NV = kSimtKeys * KR / kSimtThreads;  // vectors of a tile per thread
  ChunkItem I;
  while (walk.next(p, I)) {
    const int rows = I.tokens * p.tile_heads;
    __syncthreads();  // the last item's shared rows have been read
    for (int i = tid; i < R * VR; i += kSimtThreads) {
      const int m = i / VR, c = i - m * VR;
      float f[VE] = {};
      if (m < rows) {
        const int tok = m / p.tile_heads;
        const T* q = static_cast<const T*>(p.q) + (int64_t)(I.q0 + tok) * p.q_stride +
                     (int64_t)(I.h + m - tok * p.tile_heads) * D + c * VE;
        const uint4 v = *reinterpret_cast<const uint4*>(q);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 4) {
            f[e] = __uint_as_float(w[e]);
          } else {
            f[2 * e] = bf16_lo(w[e]);
            f[2 * e + 1] = bf16_hi(w[e]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) sQ[m * LD + c * VE + e] = f[e];
    }
    float m_run[RT], l_run[RT], acc[RT][CT * 4];
    int lo[RT], hi[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m_run[i] = -INFINITY;
      l_run[i] = 0.f;
#pragma unroll
      for (int e = 0; e < CT * 4; ++e) acc[i][e] = 0.f;
      const int m = ty * RT + i;
      const int tok = I.first_tok + m / p.tile_heads;
      const KeyRange k = chunk_keys(p, I.qo, I.kv, tok, tok + 1);
      lo[i] = k.lo;
      hi[i] = m < rows ? k.hi : 0;
    }
    const int kv_head = I.h / p.group;
    // A thread's vectors of the rows of keys [k0, k0 + 64): fetched into
    // registers, K's a tile ahead and V's while the scores are computed, then put
    // into shared memory. Keys that no row of the item sees are zero.
    float factor[NV];  // of a thread's vectors (QUANT)
    auto fetch = [&](const void* pool, const float* scale, int k0, uint4 (&v)[NV]) {
      int page[NV];
#pragma unroll
      for (int x = 0; x < NV; ++x) {
        const int j = k0 + (tid + x * kSimtThreads) / KR;
        page[x] = -1;
        if (j >= I.keys.lo && j < I.keys.hi)
          page[x] = p.page_indices[I.pbase + (p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size)];
      }
#pragma unroll
      for (int x = 0; x < NV; ++x) {
        const int i = tid + x * kSimtThreads, c = i % KR, j = k0 + i / KR;
        v[x] = make_uint4(0u, 0u, 0u, 0u);
        factor[x] = 0.f;
        if (j < I.keys.lo || j >= I.keys.hi) continue;
        if (page[x] < 0 || page[x] >= p.num_pages) {
          report(p.status, PD_DEV_BAD_PAGE_TABLE);
          continue;
        }
        const int slot = p.page_shift >= 0 ? j & (p.page_size - 1) : j % p.page_size;
        const int64_t row = p.nhd ? ((int64_t)page[x] * p.page_size + slot) * p.hkv + kv_head
                                  : ((int64_t)page[x] * p.hkv + kv_head) * p.page_size + slot;
        if constexpr (QUANT) {
          v[x] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) + row * D + c * KE));
          factor[x] = fmaxf(__ldg(scale + ((int64_t)page[x] * p.hkv + kv_head) * (p.page_size / p.scale_block) +
                                  slot / p.scale_block), kScaleMin);
        } else {
          v[x] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(pool) + row * D + c * VE));
        }
      }
    };
    auto put = [&](const uint4 (&v)[NV]) {
#pragma unroll
      for (int x = 0; x < NV; ++x) {
        const int i = tid + x * kSimtThreads;
        float4* to = reinterpret_cast<float4*>(sKV + (i / KR) * LD + (i % KR) * KE);
        if constexpr (QUANT) {
          const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = unpack_e4m3x2(w[e] & 0xffffu), b = unpack_e4m3x2(w[e] >> 16);
            to[e] = make_float4(a.x * factor[x], a.y * factor[x], b.x * factor[x], b.y * factor[x]);
          }
        } else if constexpr (sizeof(T) == 4) {
          to[0] = make_float4(__uint_as_float(v[x].x), __uint_as_float(v[x].y), __uint_as_float(v[x].z),
                              __uint_as_float(v[x].w));
        } else {
          to[0] = make_float4(bf16_lo(v[x].x), bf16_hi(v[x].x), bf16_lo(v[x].y), bf16_hi(v[x].y));
          to[1] = make_float4(bf16_lo(v[x].z), bf16_hi(v[x].z), bf16_lo(v[x].w), bf16_hi(v[x].w));
        }
      }
    };
    const bool has_rows = (tid >> 5) * 2 * RT < rows;  // of this warp's; the others only load
    uint4 kv[NV];
    bool nan = false;
    if (I.t0 < I.t1) fetch(p.k_pool, p.k_scale, (I.tile0 + I.t0) * kSimtKeys, kv);
    for (int t = I.t0; t < I.t1; ++t) {
      const int k0 = (I.tile0 + t) * kSimtKeys;
      __syncthreads();
      put(kv);
      __syncthreads();
      fetch(p.v_pool, p.v_scale, k0, kv);
      if (has_rows) {
        float s[RT][4];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float4 qv[RT], kf[4];
#pragma unroll
          for (int i = 0; i < RT; ++i) qv[i] = *reinterpret_cast<const float4*>(sQ + (ty * RT + i) * LD + d);
#pragma unroll
          for (int j = 0; j < 4; ++j) kf[j] = *reinterpret_cast<const float4*>(sKV + (tx + 16 * j) * LD + d);
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[i][j] = fmaf(qv[i].x, kf[j].x, s[i][j]);
              s[i][j] = fmaf(qv[i].y, kf[j].y, s[i][j]);
              s[i][j] = fmaf(qv[i].z, kf[j].z, s[i][j]);
              s[i][j] = fmaf(qv[i].w, kf[j].w, s[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = k0 + tx + 16 * j;
            s[i][j] = key >= lo[i] && key < hi[i] ? s[i][j] * p.scale_log2 : -INFINITY;
            mx = fmaxf(mx, s[i][j]);
          }
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          const float m_new = fmaxf(m_run[i], mx);
          const float base = m_new == -INFINITY ? 0.f : m_new;
          const float alpha = exp2f(m_run[i] - base);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float w = exp2f(s[i][j] - base);
            sum += w;
            sP[(tx + 16 * j) * LP + ty * RT + i] = w;
          }
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          l_run[i] = l_run[i] * alpha + sum;
          m_run[i] = m_new;
#pragma unroll
          for (int e = 0; e < CT * 4; ++e) acc[i][e] *= alpha;
        }
      }
      if constexpr (QUANT) {
        const KeyRange shared = shared_keys(p, I);
        if (k0 < shared.lo || k0 + kSimtKeys > shared.hi) nan |= clear_nan(kv);
      }
      __syncthreads();  // the scores have read K, and the weights are written
      put(kv);
      __syncthreads();
      if (t + 1 < I.t1) fetch(p.k_pool, p.k_scale, k0 + kSimtKeys, kv);
      if (!has_rows) continue;
#pragma unroll 8
      for (int key = 0; key < kSimtKeys; ++key) {
        float w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = sP[key * LP + ty * RT + i];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(sKV + key * LD + tx * 4 + 64 * c);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            acc[i][4 * c + 0] = fmaf(w[i], v.x, acc[i][4 * c + 0]);
            acc[i][4 * c + 1] = fmaf(w[i], v.y, acc[i][4 * c + 1]);
            acc[i][4 * c + 2] = fmaf(w[i], v.z, acc[i][4 * c + 2]);
            acc[i][4 * c + 3] = fmaf(w[i], v.w, acc[i][4 * c + 3]);
          }
        }
      }
    }
    const int64_t slot = part_slot(I, blockIdx.x);
    if (QUANT && __syncthreads_or(nan)) {
      const KeyRange shared = shared_keys(p, I), skip{shared.lo + kSimtKeys, shared.hi - kSimtKeys};
#pragma unroll
      for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int col = tx * 4 + 64 * c;
          const uint32_t bad = nan_columns(p, I.pbase, kv_head, max(lo[i], (I.tile0 + I.t0) * kSimtKeys),
                                           min(hi[i], (I.tile0 + I.t1) * kSimtKeys), skip, col / 16) >> (col & 15);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (bad >> e & 1u) acc[i][4 * c + e] = __uint_as_float(kNan);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int m = ty * RT + i;
      if (m >= rows) continue;
      const float inv = l_run[i] != 0.f ? 1.f / l_run[i] : 0.f;
      const float lse2 = l_run[i] != 0.f ? m_run[i] + log2f(l_run[i]) : -INFINITY;
      const int tok = m / p.tile_heads;
      const int64_t row = (int64_t)(I.q0 + tok) * p.hq + I.h + m - tok * p.tile_heads;
      if (slot < 0 && p.o_dtype == PD_BF16) {
        uint2* o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + tx * 4);
#pragma unroll
        for (int c = 0; c < CT; ++c)
          o[16 * c] = make_uint2(pack_bf16x2(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv),
                                 pack_bf16x2(acc[i][4 * c + 2] * inv, acc[i][4 * c + 3] * inv));
      } else {
        float* o = slot < 0 ? static_cast<float*>(p.o) + row * D : p.part_o + (slot * p.rows + m) * D;
#pragma unroll
        for (int c = 0; c < CT; ++c)
          *reinterpret_cast<float4*>(o + tx * 4 + 64 * c) =
              make_float4(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv,
                          acc[i][4 * c + 3] * inv);
      }
      if (tx == 0) {
        if (slot >= 0) p.part_lse[slot * p.rows + m] = lse2;
        else if (p.lse != nullptr) p.lse[row] = lse2 * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------ few query rows
// fp32 arithmetic for at most R query rows an item (single tokens, verification):
// HBM bound, so every warp streams keys by itself, 8 of a tile's 64, without a
// barrier of the CTA. A lane has D / 32 columns of q, k, v and o. The products of 4
// rows and 8 keys are 32 sums over the lanes, halved and exchanged until lane i has
// the i-th; each warp keeps its own maximum, sum and output, and the eight are
// joined at an item's end. The next keys are on their way to shared memory meanwhile
// (in registers instead, 2 x 8 keys a warp: 90 us for 82). 16 decodes of 1000 to
// 4096 keys, 32 / 8 heads, D 128, 265 MB, take 68 us in the kernel, 3.9 TB/s. Neither
// the bytes in flight hold it (two stages of three, 128 KB an SM, where HBM's rate
// takes about 45 at a latency of 1 us) nor the issue slots (32 %): each warp's 8 keys
// go through one chain, 31 exchanges, the maximum's three, the exponential and a trip
// of the weights through shared memory, before its next 8, and 8 warps do not cover it.
constexpr int kRowsThreads = 256, kRowsWarps = kRowsThreads / 32;
constexpr int kRowsKeys = kChunkKeys / kRowsWarps;
constexpr int kRowsStages = 3;  // of a warp's 8 keys, K and V
static_assert(kRowsKeys == 8, "4 rows x 8 keys are the 32 lanes");

template <typename T, int R, int D>
struct RowsShape {
  static constexpr size_t kTile = kRowsKeys * D * sizeof(T);          // K or V of a warp's keys
  static constexpr size_t kWarp = kRowsStages * 2 * kTile;
  static constexpr size_t kJoin = sizeof(float) * kRowsWarps * R * D;  // the warps' outputs, once their keys are done
  static constexpr size_t kRing = kRowsWarps * kWarp > kJoin ? kRowsWarps * kWarp : kJoin;
  static constexpr size_t kSmem = kRing + sizeof(float) * (R * D + kRowsWarps * (2 * R + kRowsKeys * R));
  static_assert(kSelfBytes <= kRing && kSmem <= 232448, "shared memory of a CTA");
};

// E consecutive elements as they are in memory, and as fp32.
template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };

template <typename T, int E>
struct Elems {
  typename Raw<E * sizeof(T)>::type raw;
  __device__ __forceinline__ void load(const T* p) {
    raw = __ldg(reinterpret_cast<const typename Raw<E * sizeof(T)>::type*>(p));
  }
  // From global to this thread's place in shared memory, asynchronously; zeros where not `there`.
  static __device__ __forceinline__ void copy_async(T* to, const T* from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(to)), "l"(from),
                 "n"((int)(E * sizeof(T))), "r"(there ? (int)(E * sizeof(T)) : 0)
                 : "memory");
  }
  __device__ __forceinline__ void load_shared(const T* p) {
    raw = *reinterpret_cast<const typename Raw<E * sizeof(T)>::type*>(p);
  }
  __device__ __forceinline__ void zero() { raw = {}; }
  __device__ __forceinline__ float get(int e) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  }
};

// One of a lane's two sums with the lane's across bit `half` added: `high` in the
// lanes that have the bit, `low` in the others.
__device__ __forceinline__ float halve(float low, float high, int half, int lane) {
  const bool up = lane & half;
  return (up ? high : low) + __shfl_xor_sync(0xffffffffu, up ? low : high, half);
}

template <typename T, int R, int D>
__global__ void __launch_bounds__(kRowsThreads) chunk_rows_kernel(const ChunkParams p) {
  using S = RowsShape<T, R, D>;
  constexpr int E = D / 32, SETS = R / 4;
  extern __shared__ float4 rows_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(rows_smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, key = lane & 7;
  T* ring = reinterpret_cast<T*>(smem + warp * S::kWarp) + lane * E;  // [stage][K, V][key][D], from this lane's columns on
  float* sAcc = reinterpret_cast<float*>(smem);                       // [warp][row][D]
  float* sQ = reinterpret_cast<float*>(smem + S::kRing);              // [row][D], scaled
  float* sM = sQ + R * D;                                             // [warp][row] maxima, then sums
  float* sL = sM + kRowsWarps * R;
  float* sP = sL + kRowsWarps * R + warp * kRowsKeys * R;             // [key][row], this warp's
  pdl_launch_dependents();
  pdl_wait_primary();
  ChunkWalk walk;
  {
    const ChunkLine line = take_line(p, rows_smem_raw);
    const int4 cut = walk.begin(p, line, blockIdx.x);
    if (tid == 0) p.cuts[blockIdx.x] = cut;
  }
  ChunkItem I;
  while (walk.next(p, I)) {
    __syncthreads();  // the line, or the last item's outputs, have been read
    const int rows = I.tokens * p.tile_heads;
    for (int r = warp; r < R; r += kRowsWarps) {
      Elems<T, E> x;
      x.zero();
      if (r < rows) {
        const int tok = r / p.tile_heads;
        x.load(static_cast<const T*>(p.q) + (int64_t)(I.q0 + tok) * p.q_stride +
               (int64_t)(I.h + r - tok * p.tile_heads) * D + lane * E);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sQ[r * D + lane * E + e] = x.get(e) * p.scale_log2;
    }
    float acc[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
    // this lane's scores are of rows 4 s + lane / 8
    float m[SETS], l[SETS];
    int lo[SETS], hi[SETS];
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
      m[s] = -INFINITY;
      l[s] = 0.f;
      const int r = 4 * s + lane / 8, tok = I.first_tok + r / p.tile_heads;
      const KeyRange k = chunk_keys(p, I.qo, I.kv, tok, tok + 1);
      lo[s] = k.lo;
      hi[s] = r < rows ? k.hi : 0;
    }
    const int kv_head = I.h / p.group;
    // Element offset of this lane's key of the warp's keys [k0, k0 + 8), or -1 where no row of the item sees it.
    auto place = [&](int k0) -> int64_t {
      const int j = k0 + key;
      if (j < I.keys.lo || j >= I.keys.hi) return -1;
      const int idx = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
      const int page = p.page_indices[I.pbase + idx], slot = j - idx * p.page_size;
      if (page < 0 || page >= p.num_pages) {
        report(p.status, PD_DEV_BAD_PAGE_TABLE);
        return -1;
      }
      return (p.nhd ? ((int64_t)page * p.page_size + slot) * p.hkv + kv_head
                    : ((int64_t)page * p.hkv + kv_head) * p.page_size + slot) * D;
    };
    // Starts the copies of the keys at `at` into a stage; every lane reads only what it copied.
    auto fetch = [&](int64_t at, int stage) {
      T* to = ring + stage * (2 * kRowsKeys * D);
#pragma unroll
      for (int j = 0; j < kRowsKeys; ++j) {
        const int64_t o = __shfl_sync(0xffffffffu, at, j);
        const int64_t from = (o >= 0 ? o : 0) + lane * E;
        Elems<T, E>::copy_async(to + j * D, static_cast<const T*>(p.k_pool) + from, o >= 0);
        Elems<T, E>::copy_async(to + (kRowsKeys + j) * D, static_cast<const T*>(p.v_pool) + from, o >= 0);
      }
    };
    const int first = (I.tile0 + I.t0) * kChunkKeys + warp * kRowsKeys, last = (I.tile0 + I.t1) * kChunkKeys;
    int64_t at = first < last ? place(first) : -1;
#pragma unroll
    for (int i = 0; i < kRowsStages - 1; ++i) {
      const int k0 = first + i * kChunkKeys;
      if (k0 < last) fetch(at, i);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (k0 + kChunkKeys < last) at = place(k0 + kChunkKeys);
    }
    __syncthreads();  // q
    int stage = 0;
    for (int k0 = first; k0 < last; k0 += kChunkKeys) {
      const int ahead = k0 + (kRowsStages - 1) * kChunkKeys;
      if (ahead < last) fetch(at, stage == 0 ? kRowsStages - 1 : stage - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (ahead + kChunkKeys < last) at = place(ahead + kChunkKeys);
      asm volatile("cp.async.wait_group %0;" ::"n"(kRowsStages - 1) : "memory");
      const T* k_at = ring + stage * (2 * kRowsKeys * D);
      const T* v_at = k_at + kRowsKeys * D;
      if (++stage == kRowsStages) stage = 0;
      float s[SETS];
#pragma unroll
      for (int x = 0; x < SETS; ++x) {
        // products with rows 4 x + r and r + 2 at once, so that 16 sums are held and not 32
        float part[16];
#pragma unroll
        for (int j = 0; j < kRowsKeys; ++j) {
          Elems<T, E> k;
          k.load_shared(k_at + j * D);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            Elems<float, E> qa, qb;
            qa.load_shared(sQ + (4 * x + r) * D + lane * E);
            qb.load_shared(sQ + (4 * x + r + 2) * D + lane * E);
            float a = qa.get(0) * k.get(0), b = qb.get(0) * k.get(0);
#pragma unroll
            for (int e = 1; e < E; ++e) {
              a = fmaf(qa.get(e), k.get(e), a);
              b = fmaf(qb.get(e), k.get(e), b);
            }
            part[8 * r + j] = halve(a, b, 16, lane);
          }
        }
#pragma unroll
        for (int half = 8; half > 0; half >>= 1)
#pragma unroll
          for (int i = 0; i < half; ++i) part[i] = halve(part[i], part[i + half], half, lane);
        s[x] = part[0];
      }
#pragma unroll
      for (int x = 0; x < SETS; ++x) {
        const float sc = k0 + key >= lo[x] && k0 + key < hi[x] ? s[x] : -INFINITY;
        float top = sc;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m[x]);
        const float base = top == -INFINITY ? 0.f : top;
        const float alpha = exp2f(m[x] - base), w = exp2f(sc - base);
        l[x] = l[x] * alpha + w;
        m[x] = top;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = __shfl_sync(0xffffffffu, alpha, 8 * r);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[4 * x + r][e] *= f;
          }
        }
        sP[key * R + 4 * x + lane / 8] = w;
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kRowsKeys; ++j) {
        Elems<T, E> v;
        v.load_shared(v_at + j * D);
#pragma unroll
        for (int x = 0; x < SETS; ++x) {
          const float4 w = *reinterpret_cast<const float4*>(sP + j * R + 4 * x);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float y = v.get(e);
            acc[4 * x][e] = fmaf(w.x, y, acc[4 * x][e]);
            acc[4 * x + 1][e] = fmaf(w.y, y, acc[4 * x + 1][e]);
            acc[4 * x + 2][e] = fmaf(w.z, y, acc[4 * x + 2][e]);
            acc[4 * x + 3][e] = fmaf(w.w, y, acc[4 * x + 3][e]);
          }
        }
      }
      __syncwarp();  // the weights have been read
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the warps' outputs go where their keys were
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) l[s] += __shfl_xor_sync(0xffffffffu, l[s], d);
      if (key == 0) {
        sM[warp * R + 4 * s + lane / 8] = m[s];
        sL[warp * R + 4 * s + lane / 8] = l[s];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) sAcc[(warp * R + r) * D + lane * E + e] = acc[r][e];
    __syncthreads();
    // the eight warps' outputs of 4 columns of a row
    const int64_t part = part_slot(I, blockIdx.x);
    for (int i = tid; i < rows * (D / 4); i += kRowsThreads) {
      const int r = i / (D / 4), c = 4 * (i - r * (D / 4));
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, sM[w * R + r]);
      const float base = top == -INFINITY ? 0.f : top;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float f = exp2f(sM[w * R + r] - base);
        const float4 a = *reinterpret_cast<const float4*>(sAcc + (w * R + r) * D + c);
        sum = fmaf(sL[w * R + r], f, sum);
        o.x = fmaf(a.x, f, o.x);
        o.y = fmaf(a.y, f, o.y);
        o.z = fmaf(a.z, f, o.z);
        o.w = fmaf(a.w, f, o.w);
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      const int tok = r / p.tile_heads;
      const int64_t row = (int64_t)(I.q0 + tok) * p.hq + I.h + r - tok * p.tile_heads;
      if (part < 0 && p.o_dtype == PD_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + c) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      else
        *reinterpret_cast<float4*>((part < 0 ? static_cast<float*>(p.o) + row * D : p.part_o + (part * p.rows + r) * D) +
                                   c) = o;
      if (c == 0) {
        const float lse2 = sum != 0.f ? top + log2f(sum) : -INFINITY;
        if (part >= 0) p.part_lse[part * p.rows + r] = lse2;
        else if (p.lse != nullptr) p.lse[row] = lse2 * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------------- host
ChunkLayout chunk_layout(ChunkParams& p, int32_t kv_dtype) {
  // The tensor cores take bf16, in pages of whole groups of the swizzle's 8 rows;
  // the CUDA cores take the rest.
  const bool quant = p.scale_block > 0;
  const int64_t most = (int64_t)p.max_qo_len * p.group;  // rows of a request's KV head
  p.tc = kv_dtype == PD_BF16 && p.page_size % 8 == 0 && p.scale_block % 8 == 0;
  // Few rows of an 8-bit cache have a kernel of their own: up to 8, the columns of its products. Measured against the
  // tensor-core kernel, 8 KV heads, D 128: 4 rows, 4 requests of up to 255 keys 6.3 and 9.5 us, 128 of 512 to 4096 keys 104
  // and 160 us; for 16 rows, its products twice, it took 207 us (when it took 144 for 4) and the other 164.
  p.few = quant && p.tc && most <= 8;
  p.tc = p.tc && !p.few;
  if (p.tc) {
    p.tile_heads = p.group <= 128 ? p.group : 1;
    p.tile_tokens = 128 / p.tile_heads;
    p.item_tokens = 2 * p.tile_tokens;
    p.rows = p.item_tokens * p.tile_heads;
    // (an item's ends, in tiles; of 8-bit pools counted as 2, 6 and 8: 32 requests of 2 to 8 tokens 53.5, 52.4 and
    // 52.1 us, 128 of 1 to 4 166, 159 and 160, 500 tokens over 32700 keys 232, 230 and 230)
    p.item_cost = quant ? 8 : 2;
    p.min_units = 4;
    p.max_parts = device_sm_count();
  } else {
    // Rows of an item: 4 or 16 where that takes a request's rows in one go or in a
    // few (the kernel for few rows), else 64. Of 8-bit pools the tiled kernel takes what
    // theirs does not; in it 16 cost a fourth of 64.
    if (p.few) p.rows = 8;
    else if (quant) p.rows = most <= 16 && p.group <= 16 ? 16 : 64;
    else p.rows = most <= 4 ? 4 : most <= 64 && p.group <= 16 ? 16 : 64;
    p.tile_heads = p.group <= p.rows ? p.group : 1;
    p.item_tokens = p.rows / p.tile_heads;
    // In the kernel for few rows of 8-bit pools an item's ends (its first copies' latency, and the meeting of the warps)
    // cost what 6 tiles do: 128 decodes of 512 to 4096 keys take 105.8, 103.7, 103.5 and 104.3 us counted as 2, 4, 6 and 8,
    // 24 of them 31.6, 31.0, 30.9 and 31.1.
    p.item_cost = p.few ? 6 : 1;
    p.min_units = 1;  // few tiles: one a CTA, as their latencies would add up
    p.max_parts = device_sm_count() * (p.few ? rows_quant_ctas(p.head_dim) : p.rows == 64 || quant ? 2 : 1);  // CTAs that an SM holds
  }
  p.page_shift = -1;
  if ((p.page_size & (p.page_size - 1)) == 0)
    for (p.page_shift = 0; (1 << p.page_shift) < p.page_size;) ++p.page_shift;
  p.item_heads = p.hq / p.tile_heads;
  const int64_t by_len = (int64_t)p.batch * (((int64_t)p.max_qo_len + p.item_tokens - 1) / p.item_tokens);
  const int64_t by_rows = (int64_t)p.total_qo / p.item_tokens + p.batch;
  const int64_t blocks = by_len < by_rows ? by_len : by_rows;
  p.max_blocks = (int32_t)(blocks < 0x7fffffff ? blocks : 0x7fffffff);  // (chunk_fits refuses the bound)
  ChunkLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.hdr = take(32 * sizeof(int32_t));
  L.req_first = take(sizeof(int32_t) * ((size_t)p.batch + 1));
  L.pre = take(sizeof(int32_t) * ((size_t)p.max_blocks + 1));
  L.pos = take(sizeof(int32_t) * ((size_t)p.max_parts + 1));
  L.cuts = take(sizeof(int4) * (size_t)p.max_parts);
  L.part_lse = take(sizeof(float) * 2 * (size_t)p.max_parts * p.rows);
  L.part_o = take(sizeof(float) * 2 * (size_t)p.max_parts * p.rows * p.head_dim);
  L.total = off;
  const int64_t items = (int64_t)p.max_blocks * p.item_heads;
  // Uncut items. Cutting spreads them over all CTAs, and costs the line, the parts
  // and the merge, about as much as `spare` tiles on a CTA. Measured, us uncut / cut,
  // one token a request over 256, 512, 1024 and 2048 keys, D 128, 8 KV heads: on the
  // tensor cores 4 requests 8.3 / 13.0, 10.6 / 13.3, 15.0 / 14.2, 23.9 / 16.9, 16
  // requests 8.9 / 15.0, 11.2 / 17.2, 15.8 / 20.5, 27.4 / 34.4; in fp32 4 requests
  // 10.4 / 10.5, 16.3 / 12.3, 27.9 / 15.8, 16 requests 10.8 / 16.7, 17.4 / 22.6,
  // 38.9 / 43.1, 69.7 / 70.0; fp32 items of 64 rows are better cut from two tiles
  // on. Few rows of 8-bit pools, over 256, 512, 1024 and 2048 keys: 4 requests 7.3 / 12.1, 9.1 / 12.9,
  // 12.5 / 14.4, 18.8 / 15.3, 16 requests 8.4 / 13.4, 10.7 / 14.8, 16.0 / 18.3, 25.3 / 23.6, 32 requests 8.8 / 15.4,
  // 12.0 / 18.3, 18.0 / 24.4, 28.7 / 34.1, but 16 of 10 to 2048 keys 22.6 / 18.6 (of up to 1024 14.7 / 15.8).
  // `most_tiles` bounds what requests shorter than the longest lose by it.
  const int64_t all = ((int64_t)p.max_kv_len + kChunkKeys - 1) / kChunkKeys;
  const int64_t seen = ((int64_t)p.window + p.item_tokens) / kChunkKeys + 2;  // through a window
  const int64_t tiles = p.causal && p.window >= 0 && seen < all ? seen : all;
  const int spare = p.tc ? 13 : p.few ? 16 : p.rows == 64 ? 1 : 4, most_tiles = p.tc || p.few ? 16 : p.rows == 64 ? 1 : 8;
  p.uncut = items <= p.max_parts && tiles <= most_tiles && tiles * (p.max_parts - items) <= (int64_t)spare * p.max_parts;
  p.grid = p.uncut ? (int32_t)items : p.max_parts;
  p.self_plan = p.batch <= kSelfBatch && (p.uncut || (p.max_blocks <= kSelfBlocks && p.max_parts <= kSelfParts));
  return L;
}

// Where whole items are dealt out, all rounds of G but the last are: what they leave the
// line is less than 2 G items and one block's heads. Where they are not, the line has
// less than 2^31 units, or they would be.
bool chunk_fits(const ChunkParams& p) {
  const int64_t most = ((int64_t)p.max_kv_len + kChunkKeys - 1) / kChunkKeys + p.item_cost;  // units of an item
  return (2 * (int64_t)p.max_parts + p.item_heads) * most <= 0x7fffffffLL &&
         (int64_t)p.max_blocks * p.item_heads <= 0x7fffffffLL - p.max_parts;
}

namespace {

template <auto Kernel>
cudaError_t launch_cores(const char* name, int threads, size_t smem, const ChunkParams& p, cudaStream_t stream) {
  cudaError_t e = allow_smem<Kernel>(smem);
  if (e != cudaSuccess) return e;
  last_kernel() = name;
  profile_begin(stream);
  e = launch_dependent(Kernel, dim3(p.grid), threads, smem, stream, p);
  profile_end(stream);
  return e;
}

template <typename T, int D>
cudaError_t launch_simt(const ChunkParams& p, cudaStream_t stream) {
  if (p.rows == 4)
    return launch_cores<chunk_rows_kernel<T, 4, D>>("chunk_rows_kernel", kRowsThreads, RowsShape<T, 4, D>::kSmem, p, stream);
  if (p.rows == 16)
    return launch_cores<chunk_rows_kernel<T, 16, D>>("chunk_rows_kernel", kRowsThreads, RowsShape<T, 16, D>::kSmem, p, stream);
  return launch_cores<chunk_simt_kernel<T, 64, D, false>>("chunk_simt_kernel", kSimtThreads, simt_smem<64, D>(), p, stream);
}

template <typename T, int D>
cudaError_t launch_quant_simt(const ChunkParams& p, cudaStream_t stream) {
  if (p.rows == 16)
    return launch_cores<chunk_simt_kernel<T, 16, D, true>>("chunk_simt_kernel", kSimtThreads, simt_smem<16, D>(), p, stream);
  return launch_cores<chunk_simt_kernel<T, 64, D, true>>("chunk_simt_kernel", kSimtThreads, simt_smem<64, D>(), p, stream);
}

}  // namespace

int launch_chunk(ChunkParams& p, int32_t kv_dtype, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (!p.self_plan) e = launch_dependent(chunk_plan_kernel, dim3(1), kPlanThreads, 0, stream, p);
  if (e != cudaSuccess) return PD_ERR_CUDA;
  const bool d64 = p.head_dim == 64;
  if (p.tc)
    e = p.scale_block > 0 ? launch_chunk_quant_tc(p, stream) : launch_chunk_tc(p, stream);
  else if (p.few)
    e = launch_chunk_quant_rows(p, stream);
  else if (p.scale_block > 0 && kv_dtype == PD_BF16)
    e = d64 ? launch_quant_simt<uint16_t, 64>(p, stream) : launch_quant_simt<uint16_t, 128>(p, stream);
  else if (p.scale_block > 0)
    e = d64 ? launch_quant_simt<float, 64>(p, stream) : launch_quant_simt<float, 128>(p, stream);
  else if (kv_dtype == PD_BF16)
    e = d64 ? launch_simt<uint16_t, 64>(p, stream) : launch_simt<uint16_t, 128>(p, stream);
  else
    e = d64 ? launch_simt<float, 64>(p, stream) : launch_simt<float, 128>(p, stream);
  if (e != cudaSuccess) return PD_ERR_CUDA;
  if (p.max_parts > 1 && !p.uncut) {
    const dim3 grid(p.max_parts - 1, (p.rows + 15) / 16);  // two rows a warp
    e = d64 ? launch_dependent(chunk_merge_kernel<64>, grid, kMergeThreads, 0, stream, p)
            : launch_dependent(chunk_merge_kernel<128>, grid, kMergeThreads, 0, stream, p);
  }
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace pd
