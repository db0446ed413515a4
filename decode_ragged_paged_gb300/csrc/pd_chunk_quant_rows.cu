// pd_chunk_quant_rows.cu -- chunk attention over a cache held in 8 bits, for few query
// rows (single tokens, a few drafted ones; bf16 queries, pages and blocks of a multiple of 8 tokens).
//
// HBM bound: an item has at most 16 query rows (tokens x heads of a KV head), and its keys
// pass once. Tiles of 128 rows through tensor memory would keep 4 of them busy, a
// softmax warp of 4 and every wait between the roles for them (128 decodes of 512 to 4096 keys:
// 160 us); so here a warp does all of it by itself, as the fp32 kernel for few rows does, with
// products of 16 rows (mma.m16n8k16, fp16 in, fp32 out), and the CTA's eight warps meet at an
// item's end only:
//   16 keys of 128 a warp: their 8-bit rows come through a ring of its own in shared memory by
//     cp.async, the scales of their two 8-key groups with them;
//   scores: q as fp16 (scaled by a power of two a row, exact), k as fp16 by one conversion a pair.
//     The products' inner index may be any order of the head's values, so a lane takes 16
//     neighbouring bytes of a key and not 2 here and there;
//   weights W = 2^(s + log2 b - m), b the key's scale of V and m the row's running maximum of s + log2 b
//     (raised where it grew by more than 2^8), fp16 with the largest from 2^4 to 2^12;
//     their sum over b is the softmax's;
//   o += W v: a lane takes 16 neighbouring values of 4 keys, and a byte of two keys is one pair.
#include <math.h>

#include "pd_chunk.cuh"
#include "pd_launch.cuh"
#include "pd_quant.cuh"
#include "pd_tc.cuh"

namespace pd {

namespace {

constexpr int kRqThreads = 256, kRqWarps = kRqThreads / 32;
constexpr int kRqRows = 16, kRqKeys = 16;       // of an item, and of a warp's turn
constexpr int kRqSpan = kRqWarps * kRqKeys;     // keys of the CTA's turn
constexpr int kRqStages = 6;
constexpr float kRqShift = 4.0f, kRqRaise = 8.0f;

template <int D>
struct RowsQuantShape {
  static constexpr int kCodes = kRqKeys * D;                      // K or V of a warp's keys
  static constexpr int kStage = 2 * kCodes + 16;                  // and four scales
  static constexpr int kWarp = kRqStages * kStage;
  static constexpr int kJoin = kRqRows * D * 4;                   // a warp's output
  static constexpr int kRing = kRqWarps * (kWarp > kJoin ? kWarp : kJoin);
  static constexpr size_t kSmem = kRing + 2 * kRqWarps * kRqRows * sizeof(float);
  static_assert(kSelfBytes <= kRing && kSmem <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Where 16-byte chunk `c` of a key's row lies in a stage, so that the lanes that read together meet in no bank (of
// V with D = 64 two do).
template <int D>
__device__ __forceinline__ int k_chunk(int key, int c) { return D == 128 ? c ^ (key & 1) << 2 : c; }
template <int D>
__device__ __forceinline__ int v_chunk(int key, int c) { return D == 128 ? c ^ (key >> 1 & 3) << 1 : c ^ (key >> 1 & 3); }

}  // namespace

template <int D>
__global__ void __launch_bounds__(kRqThreads, 1) chunk_quant_rows_kernel(const ChunkParams p) {
  using S = RowsQuantShape<D>;
  constexpr int kSteps = D / 16;       // products of 16 values of a head
  constexpr int kTiles = D / 8;        // of 8 columns of the output
  constexpr int kChunks = D / 16;      // 16-byte chunks of a row
  constexpr int kPer = kRqKeys * kChunks / 32;  // chunks of K (or V) that a lane copies
  extern __shared__ __align__(128) uint8_t rq_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;  // the lane's rows g and g + 8, and its place among the four that share them
  const uint32_t ring = smem_u32(rq_smem) + warp * S::kWarp;
  float* sAcc = reinterpret_cast<float*>(rq_smem);                // [warp][row][D]
  float* sM = reinterpret_cast<float*>(rq_smem + S::kRing);       // [warp][row] maxima, then sums
  float* sL = sM + kRqWarps * kRqRows;
  pdl_launch_dependents();
  pdl_wait_primary();
  ChunkWalk walk;
  {
    const ChunkLine line = take_line(p, rq_smem);
    const int4 cut = walk.begin(p, line, blockIdx.x);
    if (tid == 0) p.cuts[blockIdx.x] = cut;
  }
  const int blocks = p.page_size / p.scale_block;
  ChunkItem I;
  while (walk.next(p, I)) {
    __syncthreads();  // the line, or the last item's outputs, have been read
    const int rows = I.tokens * p.tile_heads;
    const int kv_head = I.h / p.group;
    // A lane's key of the warp's 16 from k0 on (lanes 16 to 31 as lanes 0 to 15): its row of the pools and its block of
    // the scales, -1 where no row of the item sees it.
    auto place = [&](int k0, int64_t& block) -> int64_t {
      const int j = k0 + (lane & 15);
      block = -1;
      if (j < I.keys.lo || j >= I.keys.hi) return -1;
      const int idx = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
      const int page = p.page_indices[I.pbase + idx], slot = j - idx * p.page_size;
      if (page < 0 || page >= p.num_pages) {
        report(p.status, PD_DEV_BAD_PAGE_TABLE);
        return -1;
      }
      const int64_t head = (int64_t)page * p.hkv + kv_head;
      block = head * blocks + slot / p.scale_block;
      return p.nhd ? ((int64_t)page * p.page_size + slot) * p.hkv + kv_head : head * p.page_size + slot;
    };
    // Starts the copies of the keys at `at` into a stage.
    auto fetch = [&](int64_t at, int64_t block, int stage) {
      const uint32_t to = ring + stage * S::kStage;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int key = (lane + 32 * i) / kChunks, ch = lane % kChunks;
        const int64_t row = __shfl_sync(0xffffffffu, at, key);
        const int64_t from = (row >= 0 ? row : 0) * D + ch * 16;
        copy_async<16>(to + key * D + k_chunk<D>(key, ch) * 16, static_cast<const uint8_t*>(p.k_pool) + from, row >= 0);
        copy_async<16>(to + S::kCodes + key * D + v_chunk<D>(key, ch) * 16, static_cast<const uint8_t*>(p.v_pool) + from,
                       row >= 0);
      }
      // lanes 0 to 3: K's scales of the two groups, and V's. A group's block is that of any key of it that is seen.
      int64_t seen = block;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const int64_t o = __shfl_xor_sync(0xffffffffu, seen, d);
        seen = o > seen ? o : seen;
      }
      const int64_t mine = __shfl_sync(0xffffffffu, seen, 8 * (lane & 1));
      if (lane < 4)
        copy_async<4>(to + 2 * S::kCodes + 4 * lane, (lane < 2 ? p.k_scale : p.v_scale) + (mine >= 0 ? mine : 0), mine >= 0);
    };
    const int first = (I.tile0 + I.t0) * kChunkKeys + warp * kRqKeys, last = (I.tile0 + I.t1) * kChunkKeys;
    int64_t block = -1, at = first < last ? place(first, block) : -1;
#pragma unroll 1
    for (int i = 0; i < kRqStages - 1; ++i) {
      const int k0 = first + i * kRqSpan;
      if (k0 < last) fetch(at, block, i);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (k0 + kRqSpan < last) at = place(k0 + kRqSpan, block);
    }
    // q of rows g and g + 8: values 16 c and on of each 64, scaled and as fp16
    uint32_t q[kSteps][4];
    float rs[2];
    int lo[2], hi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = g + 8 * x, tok = r / p.tile_heads;
      uint4 v[D / 64][2];
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[h][e] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows)
            v[h][e] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                           (int64_t)(I.q0 + tok) * p.q_stride +
                                                           (int64_t)(I.h + r - tok * p.tile_heads) * D + 64 * h + 16 * c) + e);
          const uint32_t w[4] = {v[h][e].x, v[h][e].y, v[h][e].z, v[h][e].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool finite = top <= 3.4e38f;  // an infinity makes all of the row NaN
      const int e = scale_exponent(finite ? top : 0.f);
      const float f = finite ? power_of_two(-e) : __uint_as_float(0x7fffffffu);
      rs[x] = power_of_two(e) * p.scale_log2;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // pair i of the 16: step 4 h + i / 2, its first or second pair
          const uint4 u = v[h][i / 4];
          const uint32_t w = i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w;
          uint32_t r16;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r16) : "f"(bf16_hi(w) * f), "f"(bf16_lo(w) * f));
          q[4 * h + i / 2][2 * (i & 1) + x] = r16;
        }
      }
      const KeyRange k = chunk_keys(p, I.qo, I.kv, I.first_tok + tok, I.first_tok + tok + 1);
      lo[x] = k.lo;
      hi[x] = r < rows ? k.hi : 0;
    }
    float o[kTiles][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int stage = 0;
#pragma unroll 1
    for (int k0 = first; k0 < last; k0 += kRqSpan) {
      const int ahead = k0 + (kRqStages - 1) * kRqSpan;
      __syncwarp();  // the stage that is filled next has been read
      if (ahead < last) fetch(at, block, stage == 0 ? kRqStages - 1 : stage - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (ahead + kRqSpan < last) at = place(ahead + kRqSpan, block);
      asm volatile("cp.async.wait_group %0;" ::"n"(kRqStages - 1) : "memory");
      __syncwarp();  // the other lanes' copies too
      const uint32_t from = ring + stage * S::kStage;
      if (++stage == kRqStages) stage = 0;
      float4 scale;  // K's of the two groups, V's of the two
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(scale.x), "=f"(scale.y), "=f"(scale.z), "=f"(scale.w)
                   : "r"(from + 2 * S::kCodes)
                   : "memory");
      // scores of the two groups of 8 keys: columns 2 c and 2 c + 1 of rows g and g + 8
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int key = 8 * n + g;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(from + key * D + k_chunk<D>(key, 4 * h + c) * 16)
                       : "memory");
          uint32_t k[8];
          to_f16(v, k);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_16816(s[n], q[4 * h + i], k[2 * i], k[2 * i + 1]);
        }
      }
      const float lb[2] = {fast_log2(fmaxf(scale.z, kScaleMin)), fast_log2(fmaxf(scale.w, kScaleMin))};
      bool raise = false;
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          // (the factor is not 0: a masked score is -inf below, and a tiny one stays a number)
          const float f = fmaf(n ? scale.y : scale.x, rs[x], 1e-37f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = k0 + 8 * n + 2 * c + e;
            float& y = s[n][2 * x + e];
            y = j >= lo[x] && j < hi[x] ? fmaf(y, f, lb[n]) : -INFINITY;
            top = fmaxf(top, y);
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) - kRqShift;
        if (top > m[x] + kRqRaise || (m[x] == -INFINITY && top > -INFINITY)) {
          alpha[x] = fast_exp2(m[x] - top);  // (0 for the first)
          m[x] = top;
          raise = true;
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          l[x] *= alpha[x];
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            o[t][2 * x] *= alpha[x];
            o[t][2 * x + 1] *= alpha[x];
          }
        }
      }
      uint32_t w[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float base = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float a = fast_exp2(s[n][2 * x] - base), b = fast_exp2(s[n][2 * x + 1] - base);
          l[x] = fmaf(a + b, fast_exp2(-lb[n]), l[x]);
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[2 * n + x]) : "f"(b), "f"(a));
        }
      }
      // values: rows of keys 2 c, 2 c + 1, 2 c + 8 and 2 c + 9, values D / 8 g and on
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 2 * c + (i & 1) + 8 * (i >> 1), byte = (D / 8) * g;
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
        uint32_t b0[4], b1[4];  // of four columns
        pairs_to_f16(__byte_perm(v[0][e], v[1][e], 0x5140), __byte_perm(v[0][e], v[1][e], 0x7362), b0);
        pairs_to_f16(__byte_perm(v[2][e], v[3][e], 0x5140), __byte_perm(v[2][e], v[3][e], 0x7362), b1);
#pragma unroll
        for (int t = 0; t < 4; ++t) mma_16816(o[4 * e + t], w, b0[t], b1[t]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the warps' outputs go where their keys were
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (c == 0) {
        sM[warp * kRqRows + g + 8 * x] = m[x];
        sL[warp * kRqRows + g + 8 * x] = l[x];
      }
      // columns 2 c and 2 c + 1 of tile t are values D / 8 * (2 c) + t and D / 8 * (2 c + 1) + t
      float* to = sAcc + (warp * kRqRows + g + 8 * x) * D + (D / 8) * 2 * c;
#pragma unroll
      for (int t = 0; t < kTiles; t += 4) {
        *reinterpret_cast<float4*>(to + t) =
            make_float4(o[t][2 * x], o[t + 1][2 * x], o[t + 2][2 * x], o[t + 3][2 * x]);
        *reinterpret_cast<float4*>(to + D / 8 + t) =
            make_float4(o[t][2 * x + 1], o[t + 1][2 * x + 1], o[t + 2][2 * x + 1], o[t + 3][2 * x + 1]);
      }
    }
    __syncthreads();
    // the eight warps' outputs of 4 columns of a row
    const int64_t part = part_slot(I, blockIdx.x);
    for (int i = tid; i < rows * (D / 4); i += kRqThreads) {
      const int r = i / (D / 4), col = 4 * (i - r * (D / 4));
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kRqWarps; ++w) top = fmaxf(top, sM[w * kRqRows + r]);
      const float base = top == -INFINITY ? 0.f : top;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRqWarps; ++w) {
        const float f = fast_exp2(sM[w * kRqRows + r] - base);
        const float4 a = *reinterpret_cast<const float4*>(sAcc + (w * kRqRows + r) * D + col);
        sum = fmaf(sL[w * kRqRows + r], f, sum);
        y.x = fmaf(a.x, f, y.x);
        y.y = fmaf(a.y, f, y.y);
        y.z = fmaf(a.z, f, y.z);
        y.w = fmaf(a.w, f, y.w);
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      const int tok = r / p.tile_heads;
      const int64_t row = (int64_t)(I.q0 + tok) * p.hq + I.h + r - tok * p.tile_heads;
      if (part < 0 && p.o_dtype == PD_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + col) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      else
        *reinterpret_cast<float4*>((part < 0 ? static_cast<float*>(p.o) + row * D : p.part_o + (part * p.rows + r) * D) +
                                   col) = y;
      if (col == 0) {
        const float lse2 = sum != 0.f ? top + log2f(sum) : -INFINITY;
        if (part >= 0) p.part_lse[part * p.rows + r] = lse2;
        else if (p.lse != nullptr) p.lse[row] = lse2 * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------------- host
namespace {

template <int D>
cudaError_t launch_rows(const ChunkParams& p, cudaStream_t stream) {
  const cudaError_t e = allow_smem<chunk_quant_rows_kernel<D>>(RowsQuantShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_quant_rows_kernel<D>, dim3((unsigned)p.grid), kRqThreads, RowsQuantShape<D>::kSmem, stream, p);
}

}  // namespace

cudaError_t launch_chunk_quant_rows(const ChunkParams& p, cudaStream_t stream) {
  last_kernel() = "chunk_quant_rows_kernel";
  profile_begin(stream);
  const cudaError_t e = p.head_dim == 64 ? launch_rows<64>(p, stream) : launch_rows<128>(p, stream);
  profile_end(stream);
  return e;
}

}  // namespace pd
