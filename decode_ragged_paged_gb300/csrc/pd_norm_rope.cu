// pd_norm_rope.cu -- per-head RMS norms of queries and keys, the position
// rotation, and the write of keys and values into their pages, in one pass.
//
// For a head x of D values (section "Qwen3-Coder" names the model family whose
// queries and keys are normed per head before the rotation):
//   y_e = x_e / sqrt(mean(x^2) + eps) * w_e           (w NULL: y = x)
//   (z_a, z_b) = (y_a cos t - y_b sin t, y_a sin t + y_b cos t)
// for the R/2 pairs i < R/2 with t = position * inv_freq[i]: (a, b) =
// (i, R/2 + i), or (2i, 2i + 1) when interleaved; values past R stay y. All of
// it is computed in fp32 and rounded once, when z is stored. Values v are
// copied.
//
// Angle. t in turns is position * (inv_freq / 2 pi) mod 1: the frequency is
// held as a 64-bit fraction of a turn and multiplied by the position in
// 64-bit integers, whose overflow is the reduction modulo one turn; fp32
// products of far positions would be off by whole turns. The fraction comes from
// a double, so an angle is off by at most position * 2^-53 of its frequency.
//
// Bound: HBM. Every element is read once and written once; a head is D / (2 V)
// lanes, each with V elements of both halves of its pairs, so both loads and
// both stores of a lane are wide and no lane needs another's elements; the sum
// of squares is the only exchange. Cosines and sines are made once per token
// and reused over the heads that the warp takes.
#include "pd_common.cuh"
#include "pd_internal.h"

namespace pd {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrUnroll = 2;  // head groups of a token in flight per warp

template <int BYTES>
struct Vec;
template <>
struct Vec<16> { using type = uint4; };
template <>
struct Vec<8> { using type = uint2; };
template <>
struct Vec<4> { using type = uint32_t; };

// V consecutive elements of type T (bf16 bits or fp32) to fp32 and back.
template <typename T, int V>
struct Pack {
  typename Vec<V * sizeof(T)>::type raw;
  __device__ __forceinline__ void load(const T* p) {
    raw = *reinterpret_cast<const typename Vec<V * sizeof(T)>::type*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    *reinterpret_cast<typename Vec<V * sizeof(T)>::type*>(p) = raw;
  }
  __device__ __forceinline__ void unpack(float* f) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        f[2 * e] = bf16_lo(w[e]);
        f[2 * e + 1] = bf16_hi(w[e]);
      }
    }
  }
  __device__ __forceinline__ void pack(const float* f) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = __float_as_uint(f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    }
  }
};

// cos and sin of a fraction of a turn given in 2^-64: the quadrant from the top
// two bits (rounded to the nearest), the rest, at most an eighth of a turn,
// through sincospif.
__device__ __forceinline__ void cos_sin_turns(uint64_t turns, float& c, float& s) {
  const uint32_t t = (uint32_t)(turns >> 32);
  const uint32_t quad = (t + (1u << 29)) >> 30;
  const int32_t rest = (int32_t)(t - (quad << 30));
  float s0, c0;
  sincospif((float)rest * 4.656612873077393e-10f, &s0, &c0);  // 2^-31: halves of a turn
  const bool odd = quad & 1;
  c = odd ? s0 : c0;
  s = odd ? c0 : s0;
  if ((quad + 1) & 2) c = -c;
  if (quad & 2) s = -s;
}

}  // namespace

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  const int lane = threadIdx.x & 31;
  const int warp = (blockIdx.x * kNrThreads + threadIdx.x) >> 5;
  const int nwarps = gridDim.x * (kNrThreads / 32);
  const int sub = lane / p.lanes, u = lane - sub * p.lanes;  // head of the group, unit of the head
  const int D = p.head_dim, half = p.rope_dim / 2;
  const bool active = u * 2 * V < D;
  // the unit's two runs of V elements
  int ea, eb;
  bool rot;
  if constexpr (INTERLEAVED) {
    ea = 2 * V * u;
    eb = ea + V;
    rot = ea < p.rope_dim;
  } else {
    rot = u * V < half;
    ea = rot ? u * V : p.rope_dim + 2 * V * (u - half / V);
    eb = rot ? half + u * V : ea + V;
  }
  rot = rot && active;
  uint64_t freq[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    freq[e] = 0;
    if (rot) {
      double x = (double)p.inv_freq[u * V + e] * 0.15915494309189535;  // 1 / (2 pi)
      x -= floor(x);
      freq[e] = (uint64_t)(x * 18446744073709551616.0);
    }
  }
  Pack<T, V> qwa, qwb, kwa, kwb;
  if (p.q_weight != nullptr && active) {
    qwa.load(static_cast<const T*>(p.q_weight) + ea);
    qwb.load(static_cast<const T*>(p.q_weight) + eb);
  }
  if (p.k_weight != nullptr && active) {
    kwa.load(static_cast<const T*>(p.k_weight) + ea);
    kwb.load(static_cast<const T*>(p.k_weight) + eb);
  }

  const int heads = p.heads;  // q heads, then k heads, then v heads (when v is written)
  const int64_t items = (int64_t)p.tokens * p.blocks;
  for (int64_t it = warp; it < items; it += nwarps) {
    const int t = (int)(it / p.blocks), blk = (int)(it - (int64_t)t * p.blocks);
    int64_t page_at = 0;  // element offset of the token's slot, head 0
    bool cached = false;
    if (p.slot_map != nullptr) {
      const int64_t slot = p.slot_map[t];
      if (slot < 0) continue;  // a padding row: nothing of it is written
      const int64_t page = slot <= 0xffffffffLL ? (int64_t)((uint32_t)slot / (uint32_t)p.page_size)
                                                : slot / p.page_size;
      cached = page < p.num_pages;
      const int64_t s = slot - page * p.page_size;
      page_at = (p.nhd ? slot * p.hkv : page * p.hkv * p.page_size + s) * D;
      if (!cached && lane == 0) report(p.status, PD_DEV_BAD_PAGE_TABLE);
    }
    float cs[V], sn[V];
    if (rot) {
      const uint64_t pos = (uint64_t)(int64_t)p.positions[t];
#pragma unroll
      for (int e = 0; e < V; ++e) cos_sin_turns(freq[e] * pos, cs[e], sn[e]);
    }
    const int g0 = blk * p.groups_per_block;
    const int g1 = min(g0 + p.groups_per_block, p.groups);
    for (int g = g0; g < g1; g += kNrUnroll) {
      Pack<T, V> a[kNrUnroll], b[kNrUnroll];
      T* out[kNrUnroll];
      int kind[kNrUnroll];  // 0 q, 1 k, 2 v
#pragma unroll
      for (int x = 0; x < kNrUnroll; ++x) {
        const int head = (g + x) * p.heads_per_group + sub;
        const T* src = nullptr;
        out[x] = nullptr;
        kind[x] = 0;
        if (g + x < g1 && head < heads && active) {
          if (head < p.hq) {
            src = static_cast<const T*>(p.q) + (int64_t)t * p.q_stride + (int64_t)head * D;
            out[x] = static_cast<T*>(p.q_out) + (int64_t)t * p.q_out_stride + (int64_t)head * D;
          } else {
            const bool is_v = head >= p.hq + p.hkv;
            const int h = head - p.hq - (is_v ? p.hkv : 0);
            kind[x] = is_v ? 2 : 1;
            src = static_cast<const T*>(is_v ? p.v : p.k) + (int64_t)t * (is_v ? p.v_stride : p.k_stride) +
                  (int64_t)h * D;
            T* dst = static_cast<T*>(is_v ? p.v_out : p.k_out);
            if (p.slot_map == nullptr) out[x] = dst + (int64_t)t * p.k_out_stride + (int64_t)h * D;
            else if (cached) out[x] = dst + page_at + (int64_t)h * (p.nhd ? D : (int64_t)p.page_size * D);
          }
        }
        if (out[x] != nullptr) {
          a[x].load(src + ea);
          b[x].load(src + eb);
        }
      }
#pragma unroll
      for (int x = 0; x < kNrUnroll; ++x) {
        float fa[V], fb[V];
        float ss = 0.f;
        if (out[x] != nullptr) {
          a[x].unpack(fa);
          b[x].unpack(fb);
#pragma unroll
          for (int e = 0; e < V; ++e) ss += fa[e] * fa[e] + fb[e] * fb[e];
        }
        for (int d = p.lanes >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (out[x] == nullptr) continue;
        if (kind[x] < 2) {
          if ((kind[x] == 0 ? p.q_weight : p.k_weight) != nullptr) {
            const float inv = rsqrtf(ss * p.inv_dim + p.eps);
            float ga[V], gb[V];
            (kind[x] == 0 ? qwa : kwa).unpack(ga);
            (kind[x] == 0 ? qwb : kwb).unpack(gb);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              fa[e] *= inv * ga[e];
              fb[e] *= inv * gb[e];
            }
          }
          if (rot) {
            if constexpr (INTERLEAVED) {
#pragma unroll
              for (int e = 0; e < V; ++e) {
                float* f = e < V / 2 ? fa + 2 * e : fb + 2 * e - V;
                const float y0 = f[0], y1 = f[1];
                f[0] = y0 * cs[e] - y1 * sn[e];
                f[1] = y0 * sn[e] + y1 * cs[e];
              }
            } else {
#pragma unroll
              for (int e = 0; e < V; ++e) {
                const float y0 = fa[e], y1 = fb[e];
                fa[e] = y0 * cs[e] - y1 * sn[e];
                fb[e] = y0 * sn[e] + y1 * cs[e];
              }
            }
          }
          a[x].pack(fa);
          b[x].pack(fb);
        }
        a[x].store(out[x] + ea);
        b[x].store(out[x] + eb);
      }
    }
  }
}

// ------------------------------------------------------------------- host
namespace {

template <typename T, int V>
void launch_v(const NormRopeParams& p, unsigned grid, cudaStream_t stream) {
  if (p.interleaved) norm_rope_kernel<T, V, true><<<grid, kNrThreads, 0, stream>>>(p);
  else norm_rope_kernel<T, V, false><<<grid, kNrThreads, 0, stream>>>(p);
}

}  // namespace

// Elements of a lane's run: the widest (at most 16 bytes) that divides the
// halves of the head and of its rotated part, keeps every row aligned, and
// gives a head to at most 32 lanes; 0 if there is none.
int32_t norm_rope_vec(const NormRopeParams& p, int32_t elem_size, uintptr_t addresses) {
  const int64_t strides = p.q_stride | p.k_stride | p.v_stride | p.q_out_stride | p.k_out_stride;
  for (int v = 16 / elem_size; v >= 2; v >>= 1) {
    if (p.head_dim % (2 * v) != 0 || p.rope_dim % (2 * v) != 0 || strides % v != 0) continue;
    if (addresses % (uintptr_t)(v * elem_size) != 0) continue;
    return p.head_dim / (2 * v) <= 32 ? v : 0;
  }
  return 0;
}

int launch_norm_rope(NormRopeParams& p, int32_t elem_size, int32_t vec, cudaStream_t stream) {
  const int units = p.head_dim / (2 * vec);
  p.lanes = 1;
  while (p.lanes < units) p.lanes <<= 1;
  p.heads_per_group = 32 / p.lanes;
  p.groups = (p.heads + p.heads_per_group - 1) / p.heads_per_group;
  p.inv_dim = 1.0f / (float)p.head_dim;
  // A warp takes as many of a token's head groups as leave every SM 32 warps:
  // more would reuse its cosines further, but leave SMs without work.
  const int64_t warps = (int64_t)device_sm_count() * 32;
  int64_t blocks = (warps + p.tokens - 1) / p.tokens;
  const int max_blocks = (p.groups + kNrUnroll - 1) / kNrUnroll;
  if (blocks > max_blocks) blocks = max_blocks;
  p.groups_per_block = (int32_t)((p.groups + blocks - 1) / blocks);
  p.groups_per_block = (p.groups_per_block + kNrUnroll - 1) / kNrUnroll * kNrUnroll;
  p.blocks = (p.groups + p.groups_per_block - 1) / p.groups_per_block;
  const int64_t items = (int64_t)p.tokens * p.blocks;
  int64_t grid = (items * 32 + kNrThreads - 1) / kNrThreads;
  const int64_t most = (int64_t)device_sm_count() * (2048 / kNrThreads);
  if (grid > most) grid = most;
  last_kernel() = "norm_rope_kernel";
  profile_begin(stream);
  if (elem_size == 2) {
    if (vec == 8) launch_v<uint16_t, 8>(p, (unsigned)grid, stream);
    else if (vec == 4) launch_v<uint16_t, 4>(p, (unsigned)grid, stream);
    else launch_v<uint16_t, 2>(p, (unsigned)grid, stream);
  } else {
    if (vec == 4) launch_v<float, 4>(p, (unsigned)grid, stream);
    else launch_v<float, 2>(p, (unsigned)grid, stream);
  }
  profile_end(stream);
  return cudaGetLastError() == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace pd
