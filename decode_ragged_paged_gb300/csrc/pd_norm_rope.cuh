// pd_norm_rope.cuh -- per-head RMS norms of queries and keys, the position
// rotation, and the write of keys and values into their pages, in one pass: the kernel.
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
// Positions with several axes (AXES: time, height and width of a token of an image or a
// video): frequency i turns by the position of its axis, positions[axis(i)][token]. Every lane
// reads the positions of the frequencies that it makes the cosines of, an item ahead as the
// single position is; the axes are two bits each of the launch's parameters. Each lane has a position
// for each of its cosines and not one for all: 16384 tokens of 32 + 2 x 8 heads 85 us with three axes, 79 with one;
// 4099 tokens of 28 + 2 x 4 heads 25 us, 128 of 32 + 2 x 8 5.5 us.
//
// Angle. t in turns is position * (inv_freq / 2 pi) mod 1: the frequency is
// held as a 64-bit fraction of a turn and multiplied by the position in
// 64-bit integers, whose overflow is the reduction modulo one turn, exactly; fp32
// products of far positions would be off by whole turns. The fraction comes from
// a double: 1 / 2 pi and its product with the frequency are each rounded (2^-52 of
// it together), and the product is cut to 2^-64 of a turn, so an angle is off by at
// most position * (inv_freq * 2^-52 + 2 pi * 2^-64) before fp32's cosine. (A frequency
// below zero is off by 2 pi * 2^-54 more: 1 - x is rounded too.)
//
// Bound: HBM; every element is read once and written once. What stands in the
// way is the instructions (at one warp a head group, a first form with scalar
// arithmetic was held at half of HBM's rate by them), so:
//   a head is D / (2 V) lanes, each with V elements of both halves of its pairs:
//     loads and stores are wide and the sum of squares is the only exchange;
//   the weights are multiplied into the token's cosines and sines once, for all
//     the heads that the warp takes: z_a = (x_a (c w_a) - x_b (s w_b)) / rms;
//   the lanes of the heads that a warp holds side by side share the cosines out;
//   the arithmetic is in packed pairs.
// Measured (bf16, D 128, cold caches): 4096 tokens of 40 + 2 x 40 heads, 252 MB,
// 46 us in the kernel, 51 us a call back to back (4.9 TB/s, 73 % of HBM's rate);
// 16384 tokens of 32 + 2 x 8 heads, 403 MB, 79 us (5.1 TB/s); 128 tokens 5.6 us,
// the launch. What is left: half of the issue slots are taken, at the 16 warps
// that 128 registers allow, and a launch's ramp is 7 us of either.
#pragma once

#include "pd_common.cuh"
#include "pd_internal.h"
#include "pd_launch.cuh"
#include "pd_tc.cuh"

namespace pd {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrUnroll = 4;  // head groups of a token in flight per warp (without staging)
// With staging: shared-memory stages of a warp, and the head groups (1 KiB each
// at most) that a stage holds.
constexpr int kNrStages = 2, kNrStageGroups = 7;
constexpr uint32_t kNrStageBytes = kNrStageGroups * 1024;
constexpr size_t kNrSmem = (size_t)(kNrThreads / 32) * kNrStages * (kNrStageBytes + sizeof(uint64_t)) + 128;

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
  // Elements 2 i and 2 i + 1.
  __device__ __forceinline__ float2 get(int i) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
  }
  __device__ __forceinline__ void set(int i, float2 v) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    } else {
      w[i] = pack_bf16x2(v.x, v.y);
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

// C: heads side by side in a warp that share a token's cosines out (a lane makes
// V / C of its unit's V pairs).
// STAGED: a warp's inputs come through shared memory by bulk copies, a stage per
// work item and kNrStages items under way, so that what is in flight is not
// limited by registers; its rows must be 16-byte aligned.
template <typename T, int V, bool INTERLEAVED, int C, bool STAGED, bool AXES>
__global__ void __launch_bounds__(kNrThreads, 2) norm_rope_kernel(const NormRopeParams p) {
  constexpr int U = STAGED ? 1 : kNrUnroll, H = V / 2;  // groups loaded together, packed pairs of a run
  extern __shared__ __align__(128) uint8_t nr_smem[];
  __shared__ int give_up;
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
  const int kinds = p.slot_map != nullptr ? 3 : 2;
  uint8_t* stages = nr_smem + (threadIdx.x >> 5) * (kNrStages * kNrStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(nr_smem + (kNrThreads / 32) * kNrStages * kNrStageBytes) +
                   (threadIdx.x >> 5) * kNrStages;
  const int hpg = p.heads_per_group;
  // Groups [a0, a1) of a kind's heads that the item's groups [g0, g1) cover; `first` is the kind's first group.
  auto cover = [&](int kind, int first, int g0, int g1, int& a0, int& a1) -> int {
    const int groups = kind == 0 ? p.q_groups : p.kv_groups;
    a0 = max(g0 - first, 0);
    a1 = min(g1 - first, groups);
    return groups;
  };
  auto source = [&](int kind, int64_t t) -> const T* {
    return kind == 0   ? static_cast<const T*>(p.q) + t * p.q_stride
           : kind == 1 ? static_cast<const T*>(p.k) + t * p.k_stride
                       : static_cast<const T*>(p.v) + t * p.v_stride;
  };
  // A warp's items are nwarps apart: (token, block) moves on by (step_t, step_b), without a division.
  const int step_t = nwarps / p.blocks, step_b = nwarps - step_t * p.blocks;
  auto move_on = [&](int& t, int& blk) {
    blk += step_b;
    t += step_t;
    if (blk >= p.blocks) blk -= p.blocks, ++t;
  };
  // Starts the copies of an item into stage `st` (one lane).
  auto fetch = [&](int t, int blk, int st) {
    if (t >= p.tokens) return;
    const int g0 = blk * p.groups_per_block, g1 = min(g0 + p.groups_per_block, p.groups);
    const void* from[3];
    uint32_t bytes[3], total = 0;
    int first = 0, a0, a1;
#pragma unroll
    for (int kind = 0; kind < 3; ++kind) {
      bytes[kind] = 0;
      if (kind >= kinds) continue;
      first += cover(kind, first, g0, g1, a0, a1);
      if (a0 >= a1) continue;
      const int h0 = a0 * hpg, h1 = min(a1 * hpg, kind == 0 ? p.hq : p.hkv);
      from[kind] = source(kind, t) + (int64_t)h0 * D;
      bytes[kind] = (uint32_t)((h1 - h0) * D * sizeof(T));
      total += bytes[kind];
    }
    mbar_arrive_expect_tx(&full[st], total);
    uint8_t* to = stages + st * kNrStageBytes;
    const uint64_t once = make_evict_first();
#pragma unroll
    for (int kind = 0; kind < 3; ++kind) {
      if (bytes[kind] == 0) continue;
      bulk_g2s_hint(to, from[kind], bytes[kind], &full[st], once);
      to += bytes[kind];
    }
  };
  pdl_launch_dependents();
  if constexpr (STAGED) {
    if (threadIdx.x == 0) give_up = 0;
    if (lane == 0) {
      for (int i = 0; i < kNrStages; ++i) mbar_init(&full[i], 1);
      fence_barrier_init();
    }
    __syncthreads();
  }
  pdl_wait_primary();
  int t = warp / p.blocks, blk = warp - t * p.blocks;
  int ft = t, fb = blk;  // the next item to fetch
  if constexpr (STAGED) {
    for (int i = 0; i < kNrStages; ++i) {
      if (lane == 0) fetch(ft, fb, i);
      move_on(ft, fb);
    }
  }
  int st = 0;
  uint32_t parity = 0;
  int64_t next_slot = p.slot_map != nullptr && t < p.tokens ? p.slot_map[t] : 0;
  constexpr int A = AXES ? V / C : 1;  // positions that a lane needs of a token
  int64_t axis_at[A];                  // where their axes' begin
#pragma unroll
  for (int j = 0; j < A; ++j) {
    axis_at[j] = 0;
    if (AXES && rot) {
      const int i = u * V + C * j + (sub & (C - 1));
      axis_at[j] = (int64_t)((p.axis_bits[i >> 4] >> (2 * (i & 15))) & 3u) * p.axis_stride;
    }
  }
  int32_t next_pos[A];
#pragma unroll
  for (int j = 0; j < A; ++j) next_pos[j] = p.rope_dim > 0 && t < p.tokens ? p.positions[axis_at[j] + t] : 0;
  // (made while the first inputs are on their way)
  uint64_t freq[V / C];  // of pairs C j + sub % C
#pragma unroll
  for (int j = 0; j < V / C; ++j) {
    freq[j] = 0;
    if (rot) {
      double x = (double)p.inv_freq[u * V + C * j + (sub & (C - 1))] * 0.15915494309189535;  // 1 / (2 pi)
      x -= floor(x);
      freq[j] = (uint64_t)(x * 18446744073709551616.0);
    }
  }
  while (t < p.tokens) {
    const int64_t slot = next_slot;
    int32_t position[A];
#pragma unroll
    for (int j = 0; j < A; ++j) position[j] = next_pos[j];
    int tn = t, bn = blk;
    move_on(tn, bn);
    if (tn < p.tokens) {  // read an item ahead
      if (p.slot_map != nullptr) next_slot = p.slot_map[tn];
      if (p.rope_dim > 0) {
#pragma unroll
        for (int j = 0; j < A; ++j) next_pos[j] = p.positions[axis_at[j] + tn];
      }
    }
    int64_t place = 0;  // element offset of the token's k and v, head 0
    bool cached = true;
    if (p.slot_map != nullptr) {
      const int64_t page = (uint64_t)slot <= 0xffffffffULL ? (int64_t)((uint32_t)slot / (uint32_t)p.page_size)
                                                           : slot / p.page_size;
      cached = slot >= 0 && page < p.num_pages;
      place = (p.nhd ? slot * p.hkv : page * p.hkv * p.page_size + (slot - page * p.page_size)) * D;
      if (slot >= 0 && !cached && lane == 0) report(p.status, PD_DEV_BAD_PAGE_TABLE);
    } else {
      place = (int64_t)t * p.k_out_stride;
    }
    const int64_t head_step = p.slot_map != nullptr && !p.nhd ? (int64_t)p.page_size * D : D;
    float cs[V], sn[V];
    if (p.rope_dim > 0) {
      float c[V / C], s[V / C];
#pragma unroll
      for (int j = 0; j < V / C; ++j)
        cos_sin_turns(freq[j] * (uint64_t)(int64_t)position[AXES ? j : 0], c[j], s[j]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int from = (e % C) * p.lanes + u;
        cs[e] = C == 1 ? c[e / C] : __shfl_sync(0xffffffffu, c[e / C], from);
        sn[e] = C == 1 ? s[e / C] : __shfl_sync(0xffffffffu, s[e / C], from);
      }
    }
    const int g0 = blk * p.groups_per_block, g1 = min(g0 + p.groups_per_block, p.groups);
    const T* staged = reinterpret_cast<const T*>(stages + st * kNrStageBytes);
    if constexpr (STAGED) {
      if (!warp_mbar_wait(&full[st], parity, &give_up, p.status)) break;
    }
    int first = 0;  // the kind's first group
    // q heads, then k heads, then v heads: one body, or its registers would add up
#pragma unroll 1
    for (int kind = 0; kind < kinds; ++kind) {
      const int count = kind == 0 ? p.hq : p.hkv;
      int a0, a1;
      first += cover(kind, first, g0, g1, a0, a1);
      if (a0 >= a1) continue;
      const T* src;  // of head a0 * hpg
      if constexpr (STAGED) {
        src = staged;
        staged += (min(a1 * hpg, count) - a0 * hpg) * D;
      } else {
        src = source(kind, t) + (int64_t)a0 * hpg * D;
      }
      // a padding row: nothing of it is written; a slot past the pools: no k and v
      if (slot < 0 || (kind > 0 && !cached)) continue;
      T* dst = kind == 0 ? static_cast<T*>(p.q_out) + t * p.q_out_stride
                         : static_cast<T*>(kind == 1 ? p.k_out : p.v_out) + place;
      const int64_t step = kind == 0 ? D : head_step;
      const T* weight = static_cast<const T*>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
      const bool turn = kind < 2 && p.rope_dim > 0;
      // the rotation of this token, weights multiplied in
      float2 aa[H], ab[H], ba[H], bb[H];
      const bool mix = turn && rot;
      {
        Pack<T, V> wa, wb;
        if (weight != nullptr && active) {
          wa.load(weight + ea);
          wb.load(weight + eb);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const float2 one = make_float2(1.f, 1.f);
          const float2 fa = weight != nullptr ? wa.get(i) : one, fb = weight != nullptr ? wb.get(i) : one;
          aa[i] = fa;
          bb[i] = fb;
          if (!mix) continue;
          if constexpr (INTERLEAVED) {
            // pairs i of run a and i of run b: z = (x0 c - x1 s, x0 s + x1 c), in four products
            const float ca = cs[i], sa = sn[i], cb = cs[H + i], sb = sn[H + i];
            aa[i] = make_float2(fa.x * ca, fa.y * ca);   // x0 -> z0, x1 -> z1
            ab[i] = make_float2(-fa.y * sa, fa.x * sa);  // x1 -> z0, x0 -> z1
            bb[i] = make_float2(fb.x * cb, fb.y * cb);
            ba[i] = make_float2(-fb.y * sb, fb.x * sb);
          } else {
            const float2 c2 = make_float2(cs[2 * i], cs[2 * i + 1]), s2 = make_float2(sn[2 * i], sn[2 * i + 1]);
            aa[i] = fmul2(fa, c2);
            ab[i] = fmul2(fb, make_float2(-s2.x, -s2.y));  // of x_b in z_a
            ba[i] = fmul2(fa, s2);                         // of x_a in z_b
            bb[i] = fmul2(fb, c2);
          }
        }
      }
      const T* s_at = src + sub * D + ea;
      T* d_at = dst + (int64_t)(a0 * hpg + sub) * step + ea;
      const int run = eb - ea, s_step = hpg * D;
      const int64_t d_step = hpg * step;
      int head = a0 * hpg + sub;
      for (int g = a0; g < a1; g += U) {
        Pack<T, V> a[U], b[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
          if (g + x < a1 && head + x * hpg < count && active) {
            a[x].load(s_at + x * s_step);
            b[x].load(s_at + x * s_step + run);
          }
        }
        s_at += U * s_step;
#pragma unroll
        for (int x = 0; x < U; ++x, head += hpg, d_at += d_step) {
          if (g + x >= a1) break;
          const bool here = head < count && active;
          if (turn || weight != nullptr) {
            float2 xa[H], xb[H], sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
              xa[i] = a[x].get(i);
              xb[i] = b[x].get(i);
            }
            float inv = 1.f;
            if (weight != nullptr) {
#pragma unroll
              for (int i = 0; i < H; ++i) {
                sum = ffma2(xa[i], xa[i], sum);
                sum = ffma2(xb[i], xb[i], sum);
              }
              float ss = active ? sum.x + sum.y : 0.f;  // lanes past the head's units have nothing
              for (int d = p.lanes >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
              inv = rsqrtf(ss * p.inv_dim + p.eps);
            }
            const float2 inv2 = make_float2(inv, inv);
#pragma unroll
            for (int i = 0; i < H; ++i) {
              float2 za = fmul2(xa[i], aa[i]), zb = fmul2(xb[i], bb[i]);
              if (mix) {
                if constexpr (INTERLEAVED) {
                  za = ffma2(make_float2(xa[i].y, xa[i].x), ab[i], za);
                  zb = ffma2(make_float2(xb[i].y, xb[i].x), ba[i], zb);
                } else {
                  za = ffma2(xb[i], ab[i], za);
                  zb = ffma2(xa[i], ba[i], zb);
                }
              }
              a[x].set(i, fmul2(za, inv2));
              b[x].set(i, fmul2(zb, inv2));
            }
          }
          if (here) {
            a[x].store(d_at);
            b[x].store(d_at + run);
          }
        }
      }
    }
    if constexpr (STAGED) {
      __syncwarp();  // every lane has read the stage
      if (lane == 0) fetch(ft, fb, st);
      move_on(ft, fb);
      if (++st == kNrStages) {
        st = 0;
        parity ^= 1u;
      }
    }
    t = tn;
    blk = bn;
  }
  if constexpr (STAGED) {
    if (*static_cast<volatile int*>(&give_up)) {  // copies may be under way: let them land before shared memory is freed
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  }
}

// ------------------------------------------------------------------- host
namespace {

template <auto Kernel>
cudaError_t launch_k(const NormRopeParams& p, unsigned grid, size_t smem, cudaStream_t stream) {
  const cudaError_t e = smem > 0 ? allow_smem<Kernel>(smem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  return launch_dependent(Kernel, dim3(grid), kNrThreads, smem, stream, p);
}

template <typename T, int V, int C, bool STAGED, bool AXES>
cudaError_t launch_s(const NormRopeParams& p, unsigned grid, cudaStream_t stream) {
  const size_t smem = STAGED ? kNrSmem : 0;
  return p.interleaved ? launch_k<norm_rope_kernel<T, V, true, C, STAGED, AXES>>(p, grid, smem, stream)
                       : launch_k<norm_rope_kernel<T, V, false, C, STAGED, AXES>>(p, grid, smem, stream);
}

template <typename T, int V, int C, bool AXES>
cudaError_t launch_c(const NormRopeParams& p, unsigned grid, cudaStream_t stream) {
  if constexpr (V * sizeof(T) == 16)
    if (p.staged) return launch_s<T, V, C, true, AXES>(p, grid, stream);
  return launch_s<T, V, C, false, AXES>(p, grid, stream);
}

template <typename T, int V, bool AXES>
cudaError_t launch_v(const NormRopeParams& p, unsigned grid, cudaStream_t stream) {
  if (V >= 4 && p.heads_per_group >= 4) return launch_c<T, V, V >= 4 ? 4 : 2, AXES>(p, grid, stream);
  if (p.heads_per_group >= 2) return launch_c<T, V, 2, AXES>(p, grid, stream);
  return launch_c<T, V, 1, AXES>(p, grid, stream);
}

}  // namespace

// The forms with one axis (pd_norm_rope.cu) and with several (pd_norm_rope_axes.cu): compiled side by side.
template <bool AXES>
cudaError_t launch_norm_rope_form(const NormRopeParams& p, int32_t elem_size, int32_t vec, unsigned grid,
                                  cudaStream_t stream) {
  if (elem_size == 2)
    return vec == 8   ? launch_v<uint16_t, 8, AXES>(p, grid, stream)
           : vec == 4 ? launch_v<uint16_t, 4, AXES>(p, grid, stream)
                      : launch_v<uint16_t, 2, AXES>(p, grid, stream);
  return vec == 4 ? launch_v<float, 4, AXES>(p, grid, stream) : launch_v<float, 2, AXES>(p, grid, stream);
}

}  // namespace pd
