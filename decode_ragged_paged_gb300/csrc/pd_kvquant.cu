// pd_kvquant.cu -- append of new keys and values to a cache held in 8 bits: e4m3
// values with a scale for each block of scale_block tokens of a page and each head.
//
// (Section "KV Messenger": a layer's new KV entries go to their pages.) For a block
// with new tokens x of a head, amax the largest |x| of them:
//   s = the smallest power of two >= max(amax / 448, 2^-100);
//   a block that holds earlier tokens of the request takes the larger of s and its own
//   scale s', and, if it grew, its earlier values c become rn(c s' / s);
//   c = rn(x / s), rounded to the nearest e4m3 value, ties to even.
// What is not finite does not count in amax and becomes NaN, so that one such value
// spoils its own row and not its block. All of it is exact in fp32 but the one rounding: scales are powers of two, and
// where a caller's own are not, quotient and product are rounded to odd first (odd()).
//
// A block has to be read whole before its first value can be written, so a team of warps
// takes (block, head, K or V), holds its new values in registers, exchanges the
// maximum and writes them. One warp holds 16 tokens of 128 bf16 values (8 vectors a
// lane); larger blocks take 2, 4 or 8. The CTA's first warp finds the blocks that
// its rows begin: a request's row is looked for with 32 probes at a time, as one
// after another they would cost a decode more than everything else.
//
// Bound: HBM, every new value read once and half or a quarter of that written. Measured (cold caches): 4096
// tokens of 2 x 40 heads of 128, bf16, 126 MB, 29 us (4.3 TB/s, 65 % of the copy rate); 24 requests of 37 to 700 fp32
// tokens, 2 x 8 heads of 64, 37 MB, 14 us, two rounds of CTAs that each wait for their places, values and
// maximum in turn; 128 decodes 4.1 us, the launch. 80 registers, 3 CTAs an SM: with 64 and 4 the three take 29, 14.8
// and 4.6 us; CTAs of 128 threads 35, 19 and 4.0.
#include <cfloat>
#include <type_traits>

#include <cuda_bf16.h>

#include "pd_common.cuh"
#include "pd_internal.h"
#include "pd_quant.cuh"
#include "pd_tc.cuh"

namespace pd {

namespace {

constexpr int kQaThreads = 256, kQaWarps = kQaThreads / 32;
constexpr int kQaRows = 32;  // rows of a CTA at most: a lane each

// 8 consecutive elements of type T (bf16 bits or fp32).
template <typename T>
struct Vec8 {
  static constexpr int N = sizeof(T) / 2;
  uint4 raw[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                   : "l"(reinterpret_cast<const uint4*>(p) + i));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // Elements 2 i and 2 i + 1.
  __device__ __forceinline__ float2 get(int i) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
  }
  // The largest |x| of them and of m (an infinity among them; a NaN is passed over), in T's own arithmetic.
  using Max = std::conditional_t<sizeof(T) == 4, float, __nv_bfloat162>;
  __device__ __forceinline__ void largest(Max& m) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
    for (int e = 0; e < 4 * N; ++e) {
      if constexpr (sizeof(T) == 4) m = fmaxf(m, fabsf(__uint_as_float(w[e])));
      else m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
    }
  }
  static __device__ __forceinline__ Max none() {
    if constexpr (sizeof(T) == 4) return 0.f;
    else return __float2bfloat162_rn(0.f);
  }
  static __device__ __forceinline__ float of(Max m) {
    if constexpr (sizeof(T) == 4) return m;
    else return fmaxf(__low2float(m), __high2float(m));
  }
  // Times a power of two, as e4m3.
  __device__ __forceinline__ uint2 encode(float inv) const {
    uint32_t v[4];
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = fmul2(get(e), inv2);
      v[e] = pack_e4m3x2(f.x, f.y);
    }
    return make_uint2(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410));
  }
};

// The largest finite |x| of a lane's share of a block's new values, one by one: only where some are not finite.
template <typename T>
__device__ __noinline__ float largest_finite(const T* src, int64_t stride, int count, int D, int at, int step) {
  float m = 0.f;
  for (int i = at; i < count * D; i += step) {
    const T x = src[(i / D) * stride + i % D];
    float a;
    if constexpr (sizeof(T) == 4) a = fabsf(x);
    else a = fabsf(bf16_lo(x));
    if (a <= FLT_MAX) m = fmaxf(m, a);
  }
  return m;
}

// x, which is y cut towards 0, with its last bit set where y - x, `left`, is not 0: rounded from there to far fewer bits it
// gives what y would, as a tie of those is never made and never lost.
__device__ __forceinline__ float odd(float x, float left) {
  return left != 0.f ? __uint_as_float(__float_as_uint(x) | 1u) : x;
}

// Stores a lane's share of a block's new values one by one, with a division: where some are not finite (what is
// not becomes NaN), or the caller's own scale is no power of two, whose inverse would not be exact.
template <typename T>
__device__ __noinline__ void store_slowly(const T* src, int64_t stride, int count, int D, float s, uint8_t* to, int64_t to_step,
                                          int at, int step) {
  for (int i = at; i < count * D; i += step) {
    const int tok = i / D, d = i - tok * D;
    float x;
    if constexpr (sizeof(T) == 4) x = src[tok * stride + d];
    else x = bf16_lo(src[tok * stride + d]);
    if (fabsf(x) <= FLT_MAX) {
      // (s is not below |x| / 448; where both are small, what the quotient leaves would be below fp32's smallest)
      const float up = s < 1.f ? 0x1p64f : 1.f, y = x * up, t = s * up, q = __fdiv_rz(y, t);
      x = odd(q, fmaf(-q, t, y));
    } else {
      x = __uint_as_float(0x7fffffffu);
    }
    to[tok * to_step + d] = (uint8_t)pack_e4m3x2(x, 0.f);
  }
}

// What a CTA's rows begin: `count` new tokens from row `row` on, at places i0 and on of a block of the page that
// is number `entry` of the page lists.
struct Begun {
  int row, count, i0, entry, block;
};

// The last request whose rows begin at or before `row`, by a whole warp (0 if the indptr starts behind it).
__device__ __forceinline__ int request_of(const int32_t* indptr, int batch, int row, int lane) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned before = __ballot_sync(0xffffffffu, lane * step < n && __ldg(indptr + at) <= row);
    const int k = max(__popc(before) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

}  // namespace

template <typename T, int NV>
__global__ void __launch_bounds__(kQaThreads, 3) kv_append_quant_kernel(const KvQuantParams p) {
  __shared__ Begun begun[kQaRows];
  __shared__ int num_begun;
  __shared__ uint32_t red[kQaWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = p.page_size, S = p.scale_block, D = p.head_dim;
  pdl_launch_dependents();
  pdl_wait_primary();
  if (warp == 0) {
    const int r0 = blockIdx.x * p.rows, row = r0 + lane;
    const bool mine = lane < p.rows && row < p.total;
    int r = request_of(p.new_indptr, p.batch, r0, lane);
    bool leads = false;
    Begun w{};
    if (mine) {
      if (lane > 0 && r + 1 < p.batch && __ldg(p.new_indptr + r + 1) <= row) {
        int hi = p.batch;
        while (hi - r > 1) {
          const int mid = (r + hi) >> 1;
          if (__ldg(p.new_indptr + mid) <= row) r = mid;
          else hi = mid;
        }
      }
      const int a = __ldg(p.new_indptr + r), b = __ldg(p.new_indptr + r + 1);
      if (row >= a && row < b) {  // else a row past the last request's tokens
        const int fresh = b - a, n = __ldg(p.kv_len + r);
        const int pa = __ldg(p.page_indptr + r), pb = __ldg(p.page_indptr + r + 1);
        const int t = n - fresh + (row - a);
        if (a < 0 || b > p.total || pa < 0 || pb < pa) {
          report(p.status, PD_DEV_BAD_INDPTR);
        } else if (fresh > n || n > p.max_kv_len) {
          report(p.status, PD_DEV_BAD_LENGTH);
        } else if ((int64_t)(pb - pa) * P < n) {
          report(p.status, PD_DEV_BAD_PAGE_TABLE);
        } else if (row == a || t % S == 0) {
          leads = true;
          w.entry = pa + t / P;
          w.row = row;
          w.i0 = t % S;
          w.block = t % P / S;
          w.count = min(S - w.i0, b - row);
        }
      }
    }
    const unsigned some = __ballot_sync(0xffffffffu, leads);
    if (leads) begun[__popc(some & ((1u << lane) - 1))] = w;
    if (lane == 0) num_begun = __popc(some);
  }
  __syncthreads();
  const int team_warps = p.team_warps, teams = kQaWarps / team_warps, team = warp / team_warps;
  const int tw = team_warps * 32, tl = threadIdx.x - team * tw;
  auto team_sync = [&] {
    if (team_warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(tw) : "memory");
  };
  const int c0 = blockIdx.y * p.per_slice, per = min(p.per_slice, 2 * p.hkv - c0);
  const int vpr = D / 8;  // vectors of a row
  const int items = num_begun * per;
  for (int it = team; it < items; it += teams) {
    const Begun w = begun[it / per];
    const int c = c0 + it % per;
    const bool is_v = c >= p.hkv;
    const int h = is_v ? c - p.hkv : c;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const T* src = static_cast<const T*>(is_v ? p.v_new : p.k_new) + w.row * stride + (int64_t)h * D;
    const int page = __ldg(p.page_indices + w.entry);  // (on its way with the new values)
    const int vecs = w.count * vpr;
    Vec8<T> x[NV];
    // vector i of the block: its row
    auto row_of = [&](int i) { return p.vpr_shift >= 0 ? i >> p.vpr_shift : i / vpr; };
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (i0 + u * tw >= vecs) break;  // (none of the team's)
        const int i = i0 + tl + u * tw, tok = row_of(i);
        if (i < vecs) x[u].load(src + tok * stride + (i - tok * vpr) * 8);
        else x[u].zero();
      }
    };
    auto whole_team = [&](float m) {  // the largest of the team's
      uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
      if (team_warps > 1) {
        if (lane == 0) red[warp] = bits;
        team_sync();
        for (int i = 0; i < team_warps; ++i) bits = max(bits, red[team * team_warps + i]);
        team_sync();  // (before the next maximum)
      }
      return __uint_as_float(bits);
    };
    auto m = Vec8<T>::none();
    float was = 0.f;
    float* scale = nullptr;
    for (int i0 = 0; i0 < vecs; i0 += NV * tw) {
      load(i0);
      if (i0 == 0) {
        if (page < 0 || page >= p.num_pages) {
          if (tl == 0) report(p.status, PD_DEV_BAD_PAGE_TABLE);
          break;
        }
        scale = (is_v ? p.v_scale : p.k_scale) + ((int64_t)page * p.hkv + h) * (P / S) + w.block;
        if (w.i0 > 0) was = *scale;
      }
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (i0 + u * tw >= vecs) break;
        x[u].largest(m);
      }
    }
    if (scale == nullptr) continue;  // (the whole team's)
    float amax = whole_team(Vec8<T>::of(m));
    const bool finite = amax <= FLT_MAX;
    if (!finite) amax = whole_team(largest_finite(src, stride, w.count, D, tl, tw));
    float s = power_of_two(scale_exponent(amax));
    if (w.i0 > 0) s = fmaxf(s, was);
    uint8_t* pool = static_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool);
    const int slot0 = w.block * S;
    const int64_t at = p.nhd ? (((int64_t)page * P + slot0) * p.hkv + h) * D
                             : (((int64_t)page * p.hkv + h) * P + slot0) * D;
    const int64_t step = p.nhd ? (int64_t)p.hkv * D : D;  // from one slot to the next
    if (w.i0 > 0 && s != was) {
      const float f = was / s;
      for (int i = tl; i < w.i0 * vpr; i += tw) {
        const int tok = row_of(i);
        uint2* to = reinterpret_cast<uint2*>(pool + at + tok * step + (i - tok * vpr) * 8);
        const uint2 old = *to;
        uint32_t v[4] = {old.x & 0xffffu, old.x >> 16, old.y & 0xffffu, old.y >> 16};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = unpack_e4m3x2(v[e]);
          const float lo = __fmul_rz(y.x, f), hi = __fmul_rz(y.y, f);
          v[e] = pack_e4m3x2(odd(lo, fmaf(y.x, f, -lo)), odd(hi, fmaf(y.y, f, -hi)));
        }
        *to = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
      }
    }
    uint8_t* to = pool + at + w.i0 * step;
    if (finite && (__float_as_uint(s) & 0x7fffffu) == 0) {
      const float inv = 1.f / s;
      for (int i0 = 0; i0 < vecs; i0 += NV * tw) {
        if (vecs > NV * tw) load(i0);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          if (i0 + u * tw >= vecs) break;
          const int i = i0 + tl + u * tw, tok = row_of(i);
          if (i < vecs) *reinterpret_cast<uint2*>(to + tok * step + (i - tok * vpr) * 8) = x[u].encode(inv);
        }
      }
    } else {
      store_slowly(src, stride, w.count, D, s, to, step, tl, tw);
    }
    if (tl == 0) *scale = s;
  }
}

// ------------------------------------------------------------------- host
int launch_kv_append_quant(KvQuantParams& p, int32_t elem_size, cudaStream_t stream) {
  const int nv = elem_size == 2 ? 8 : 4;  // vectors of a lane: 32 registers
  const int vpr = p.head_dim / 8;
  p.vpr_shift = -1;
  if ((vpr & (vpr - 1)) == 0)
    for (p.vpr_shift = 0; (1 << p.vpr_shift) < vpr;) ++p.vpr_shift;
  // New tokens of a block: as many as it holds, but a batch of few rows a request (a decode) brings fewer.
  // (A guess that sizes teams; a team takes more than it holds in several rounds.)
  const int64_t each = ((int64_t)p.total + p.batch - 1) / p.batch;
  const int64_t most = each < p.scale_block ? each : p.scale_block;
  p.team_warps = 1;
  while (p.team_warps < kQaWarps && (int64_t)p.team_warps * 32 * nv < most * vpr) p.team_warps *= 2;
  // Rows of a CTA: about a block's.
  p.rows = (int32_t)(most < kQaRows ? most : kQaRows);
  const int64_t windows = ((int64_t)p.total + p.rows - 1) / p.rows;
  // Heads of a CTA: two items a team where there is work enough to fill the GPU (they share what the
  // first warp finds), one where there is not.
  const int teams = kQaWarps / p.team_warps, all = 2 * p.hkv;
  const int64_t enough = 4LL * device_sm_count();
  p.per_slice = windows * ((all + 2 * teams - 1) / (2 * teams)) >= enough ? 2 * teams : teams;
  if (p.per_slice > all) p.per_slice = all;
  const unsigned slices = (unsigned)((all + p.per_slice - 1) / p.per_slice);
  last_kernel() = "kv_append_quant_kernel";
  profile_begin(stream);
  const dim3 grid((unsigned)windows, slices);
  const cudaError_t e = elem_size == 2
                            ? launch_dependent(kv_append_quant_kernel<uint16_t, 8>, grid, kQaThreads, 0, stream, p)
                            : launch_dependent(kv_append_quant_kernel<float, 4>, grid, kQaThreads, 0, stream, p);
  profile_end(stream);
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace pd
