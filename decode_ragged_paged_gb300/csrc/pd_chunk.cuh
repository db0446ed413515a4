// pd_chunk.cuh -- the work line of the chunk attention: how (request, token
// block, head) items become units, and how a CTA walks its part of the line.
//
// The blocks of a request follow one another, its heads follow one another
// around them (all blocks of a head, then the next head), the requests around
// those. pre[b] holds the units of one head before block b, so request r's
// units start at item_heads * pre[first(r)], its head h at + h * (pre[first(r +
// 1)] - pre[first(r)]), and a position is found by two binary searches.
#pragma once

#include "pd_common.cuh"
#include "pd_internal.h"

namespace pd {

// Keys a block of tokens [t0, t1) of a request may see: [lo, hi).
struct KeyRange {
  int lo, hi;
};

__device__ __forceinline__ KeyRange chunk_keys(const ChunkParams& p, int qo, int kv, int t0, int t1) {
  KeyRange k;
  k.hi = p.causal ? min(kv, kv - qo + t1) : kv;
  k.lo = p.window >= 0 ? max(0, kv - qo + t0 - p.window) : 0;
  return k;
}

__device__ __forceinline__ int chunk_tiles(const ChunkParams& p, KeyRange k) {
  return k.hi > k.lo ? (k.hi + p.key_tile - 1) / p.key_tile - k.lo / p.key_tile : 0;
}

// A CTA's share of one item: key tiles [t0, t1) of its n.
struct ChunkItem {
  int r, q0, tokens, first_tok, h, qo, kv, pbase, need;  // q0: row of its first token; first_tok: that token's index
  int n, t0, t1;
  KeyRange keys;
  int tile0;  // first key tile of the item (absolute)
};

__device__ __forceinline__ int64_t part_start(int64_t units, int64_t parts, int64_t c) { return units * c / parts; }

struct ChunkWalk {
  int64_t u, u1;  // units left: [u, u1)
  int64_t item_start;
  int r, b, b0, b1, h;

  // To unit `at` of the line; the part ends before unit `end`.
  __device__ __forceinline__ void seek(const ChunkParams& p, int64_t at, int64_t end) {
    u = at;
    u1 = end;
    if (u >= u1) return;
    // last request whose units start at or before `at` (requests without blocks start where the next one does)
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.pre[p.req_first[mid]] * p.item_heads <= at) lo = mid;
      else hi = mid;
    }
    r = lo;
    b0 = p.req_first[r];
    b1 = p.req_first[r + 1];
    const int64_t start = p.pre[b0] * p.item_heads, per_head = p.pre[b1] - p.pre[b0];
    h = (int)((at - start) / per_head);
    const int64_t head_start = start + h * per_head;
    const int64_t rest = at - head_start + p.pre[b0];
    lo = b0;
    hi = b1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.pre[mid] <= rest) lo = mid;
      else hi = mid;
    }
    b = lo;
    item_start = head_start + p.pre[b] - p.pre[b0];
  }

  // The next item of the part that has keys here, or none at all to see.
  __device__ __forceinline__ bool next(const ChunkParams& p, ChunkItem& I) {
    while (u < u1) {
      const int64_t units = p.pre[b + 1] - p.pre[b];
      I.n = (int)units - p.item_cost;
      I.t0 = (int)(u - item_start);
      I.t1 = (int)min((int64_t)I.n, u1 - item_start);
      const bool some = I.n > 0 ? I.t0 < I.n : I.t0 == 0;
      if (some) {
        const int a = p.qo_indptr[r];
        I.r = r;
        I.qo = p.qo_indptr[r + 1] - a;
        I.kv = p.kv_len[r];
        I.first_tok = (b - b0) * p.item_tokens;
        I.tokens = min(p.item_tokens, I.qo - I.first_tok);
        I.q0 = a + I.first_tok;
        I.h = h * p.tile_heads;
        I.pbase = p.page_indptr[r];
        I.need = (I.kv + p.page_size - 1) / p.page_size;
        I.keys = chunk_keys(p, I.qo, I.kv, I.first_tok, I.first_tok + I.tokens);
        I.tile0 = I.keys.lo / p.key_tile;
      }
      // on to the next item
      item_start += units;
      u = item_start;
      if (++b == b1) {
        b = b0;
        if (++h == p.item_heads) {
          h = 0;
          while (++r < p.batch) {
            b0 = b1;
            b1 = p.req_first[r + 1];
            if (b1 > b0) break;
          }
          b = b0;
        }
      }
      if (some) return true;
    }
    return false;
  }
};

// Where a cut item's part goes: 2 c for the part that an earlier CTA began, 2 c
// + 1 for the one that CTA c begins; -1 for a whole item.
__device__ __forceinline__ int64_t part_slot(const ChunkItem& I, int c) {
  if (I.t0 == 0 && I.t1 == I.n) return -1;
  return 2 * (int64_t)c + (I.t0 == 0 ? 1 : 0);
}

}  // namespace pd
