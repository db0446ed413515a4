// pd_chunk_quant.cuh -- values of V that are NaN, in the kernels over 8-bit pools (the append makes them of
// what is not finite).
//
// Such a value belongs into its column of the rows that see its key, but in a product it would reach all
// rows of the item, as a weight of 0 times NaN is NaN. So where some row of the item does not see all of a tile's
// keys, the tile's NaNs enter the product as 0, and an item that had any has them put into its outputs
// afterwards, row by row, out of the pool. In other tiles, where all rows see every key, the product itself does it.
#pragma once

#include "pd_chunk.cuh"

namespace pd {

namespace {

// Keys that every row of the item sees.
__device__ __forceinline__ KeyRange shared_keys(const ChunkParams& p, const ChunkItem& I) {
  const int last = I.first_tok + I.tokens - 1;
  const KeyRange a = chunk_keys(p, I.qo, I.kv, I.first_tok, I.first_tok + 1), b = chunk_keys(p, I.qo, I.kv, last, last + 1);
  return KeyRange{b.lo, a.hi};
}

// Bit 7 of every byte of four e4m3 values that is NaN (0x7f or 0xff); other bits are anything.
__device__ __forceinline__ uint32_t nan_bits(uint32_t v) { return (v & 0x7f7f7f7fu) + 0x01010101u; }

// Four e4m3 values with 0 for those that are NaN.
__device__ __forceinline__ uint32_t without_nan(uint32_t v) {
  const uint32_t nan = nan_bits(v) & 0x80808080u;
  return v & ~(nan | (nan - (nan >> 7)));
}

// Puts 0 for the NaNs among them; whether there were any.
template <int N>
__device__ __forceinline__ bool clear_nan(uint4 (&v)[N]) {
  uint32_t found = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) found |= (nan_bits(v[i].x) | nan_bits(v[i].y)) | (nan_bits(v[i].z) | nan_bits(v[i].w));
  if ((found & 0x80808080u) == 0) return false;
#pragma unroll
  for (int i = 0; i < N; ++i)
    v[i] = make_uint4(without_nan(v[i].x), without_nan(v[i].y), without_nan(v[i].z), without_nan(v[i].w));
  return true;
}

// Which of 16 columns of a row, from 16 * chunk on, have a NaN in V among keys [lo, hi); keys [skip_lo, skip_hi)
// need not be looked at. A function of its own, as it runs once in a long while.
__device__ __noinline__ uint32_t find_nan(const uint8_t* v_pool, const int32_t* pages, int num_pages, int page_size, int hkv,
                                          int kv_head, int nhd, int head_dim, int lo, int hi, int skip_lo, int skip_hi,
                                          int chunk) {
  uint32_t found[4] = {};
#pragma unroll 1
  for (int j = lo; j < hi; ++j) {
    if (j >= skip_lo && j < skip_hi) {
      j = skip_hi - 1;
      continue;
    }
    const int page = __ldg(pages + j / page_size), slot = j % page_size;
    if (page < 0 || page >= num_pages) continue;
    const int64_t row = nhd ? ((int64_t)page * page_size + slot) * hkv + kv_head
                            : ((int64_t)page * hkv + kv_head) * page_size + slot;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(v_pool + row * head_dim) + chunk);
    found[0] |= nan_bits(v.x);
    found[1] |= nan_bits(v.y);
    found[2] |= nan_bits(v.z);
    found[3] |= nan_bits(v.w);
  }
  uint32_t columns = 0;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = i == 0 ? found[0] : i == 1 ? found[1] : i == 2 ? found[2] : found[3];
    columns |= ((f >> 7 & 1u) | (f >> 14 & 2u) | (f >> 21 & 4u) | (f >> 28 & 8u)) << (4 * i);
  }
  return columns;
}

__device__ __forceinline__ uint32_t nan_columns(const ChunkParams& p, int pbase, int kv_head, int lo, int hi, KeyRange skip,
                                                int chunk) {
  return find_nan(static_cast<const uint8_t*>(p.v_pool), p.page_indices + pbase, p.num_pages, p.page_size, p.hkv, kv_head,
                  p.nhd, p.head_dim, lo, hi, skip.lo, skip.hi, chunk);
}

constexpr uint32_t kNan = 0x7fffffffu;

}  // namespace

}  // namespace pd
