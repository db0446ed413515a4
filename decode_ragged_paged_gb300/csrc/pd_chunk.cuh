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
  int q0, tokens, first_tok, h;  // row of its first token, tokens, that token's index in the request, query head
  int qo, kv, pbase, need;       // of its request: new tokens, cached ones, page list
  int n, t0, t1, tile0;          // tile0: its first key tile
  KeyRange keys;
};

// A request as the work line sees it; no blocks if it is skipped.
struct ChunkRequest {
  int row, qo, kv, pbase, blocks;
};

__device__ __forceinline__ ChunkRequest chunk_request(const ChunkParams& p, int r, bool say) {
  const int a = p.qo_indptr[r], b = p.qo_indptr[r + 1], n = p.kv_len[r];
  const int pa = p.page_indptr[r], pb = p.page_indptr[r + 1];
  int code = PD_DEV_OK;
  if (a < 0 || b < a || b > p.total_qo || pa < 0 || pb < pa) code = PD_DEV_BAD_INDPTR;
  else if (n < 0 || n > p.max_kv_len || b - a > p.max_qo_len) code = PD_DEV_BAD_LENGTH;
  else if ((long long)(pb - pa) * p.page_size < n) code = PD_DEV_BAD_PAGE_TABLE;
  if (code != PD_DEV_OK) {
    if (say) report(p.status, code);
    return ChunkRequest{0, 0, 0, 0, 0};
  }
  return ChunkRequest{a, b - a, n, pa, (b - a + p.item_tokens - 1) / p.item_tokens};
}

// Units of one head of a request's block.
__device__ __forceinline__ int block_units(const ChunkParams& p, int qo, int kv, int block) {
  const int t0 = block * p.item_tokens;
  return p.item_cost + chunk_tiles(p, chunk_keys(p, qo, kv, t0, min(qo, t0 + p.item_tokens)));
}

__device__ __forceinline__ int64_t part_start(int64_t units, int64_t parts, int64_t c) { return units * c / parts; }

// Exclusive scan over a CTA of NT threads, and the total; warp_tot: NT / 32 words of shared memory.
template <int NT>
__device__ __forceinline__ long long scan_exclusive(long long v, long long* warp_tot, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the totals of an earlier scan have been read
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  long long w = lane < NT / 32 ? warp_tot[lane] : 0;
#pragma unroll
  for (int d = 1; d < NT / 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, NT / 32 - 1);
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp > 0 ? before : 0) + x - v;
}

// The work line of a batch, by one CTA: checks the requests, numbers their
// blocks (first [B + 1]) and sums the blocks' units (pre [blocks + 1]), both in
// global memory or in the CTA's own shared memory. Ends with a barrier.
struct ChunkLine {
  int64_t units, parts;
};

template <int NT>
__device__ ChunkLine plan_line(const ChunkParams& p, int32_t* first, int64_t* pre, long long* warp_tot) {
  const int tid = threadIdx.x;
  long long carry = 0, total;
  for (int r0 = 0; r0 < p.batch; r0 += NT) {
    const int r = r0 + tid;
    const long long n = r < p.batch ? chunk_request(p, r, true).blocks : 0;
    const long long at = carry + scan_exclusive<NT>(n, warp_tot, total);
    if (r < p.batch) first[r] = (int)min(at, (long long)p.max_blocks);
    carry += total;
  }
  if (carry > p.max_blocks) {
    // more blocks than rows allow: requests whose rows overlap. None is worked on.
    if (tid == 0) report(p.status, PD_DEV_BAD_INDPTR);
    __syncthreads();
    return ChunkLine{0, 1};
  }
  const int blocks = (int)carry;
  if (tid == 0) first[p.batch] = blocks;
  __syncthreads();
  carry = 0;
  for (int b0 = 0; b0 < blocks; b0 += NT) {
    const int b = b0 + tid;
    long long units = 0;
    if (b < blocks) {
      int lo = 0, hi = p.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= b) lo = mid;
        else hi = mid;
      }
      units = block_units(p, p.qo_indptr[lo + 1] - p.qo_indptr[lo], p.kv_len[lo], b - first[lo]);
    }
    const long long at = carry + scan_exclusive<NT>(units, warp_tot, total);
    if (b < blocks) pre[b] = at;
    carry += total;
  }
  if (tid == 0) pre[blocks] = carry;
  ChunkLine line;
  line.units = carry * p.item_heads;
  line.parts = (line.units + p.min_units - 1) / p.min_units;  // at least so many units a part
  if (line.parts > p.max_parts) line.parts = p.max_parts;
  if (line.parts < 1) line.parts = 1;
  __syncthreads();
  return line;
}

// A small batch's line is made by every CTA for itself, in `scratch` (kSelfBytes
// of its shared memory); a large one's has been left in the workspace by the plan
// kernel. The seek that follows reads it where this returns it.
constexpr int kSelfBatch = 256, kSelfBlocks = 1024;
constexpr size_t kSelfBytes = 32 * 8 + (kSelfBlocks + 2) * 8 + (kSelfBatch + 2) * 4;

template <int NT>
__device__ __forceinline__ ChunkLine take_line(const ChunkParams& p, void* scratch, const int32_t*& first,
                                               const int64_t*& pre) {
  if (!p.self_plan) {
    first = p.req_first;
    pre = p.pre;
    return ChunkLine{p.hdr[0], p.hdr[1]};
  }
  long long* warp_tot = static_cast<long long*>(scratch);
  int64_t* own_pre = reinterpret_cast<int64_t*>(warp_tot + 32);
  int32_t* own_first = reinterpret_cast<int32_t*>(own_pre + kSelfBlocks + 2);
  first = own_first;
  pre = own_pre;
  return plan_line<NT>(p, own_first, own_pre, warp_tot);
}

struct ChunkWalk {
  int64_t u = 0, u1 = 0;  // units left: [u, u1)
  int64_t item_start;
  int r, b, h;  // request, block of it, item head
  ChunkRequest q;

  // To unit `at` of the line; the part ends before unit `end`.
  __device__ __forceinline__ void seek(const ChunkParams& p, const int32_t* first, const int64_t* pre, int64_t at,
                                       int64_t end) {
    u = at;
    u1 = end;
    if (u >= u1) return;
    // last request whose units start at or before `at` (requests without blocks start where the next one does)
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[first[mid]] * p.item_heads <= at) lo = mid;
      else hi = mid;
    }
    r = lo;
    const int b0 = first[r], b1 = first[r + 1];
    const int64_t start = pre[b0] * p.item_heads, per_head = pre[b1] - pre[b0];
    h = (int)((at - start) / per_head);
    const int64_t head_start = start + h * per_head;
    const int64_t rest = at - head_start + pre[b0];
    lo = b0;
    hi = b1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= rest) lo = mid;
      else hi = mid;
    }
    b = lo - b0;
    item_start = head_start + pre[lo] - pre[b0];
    q = chunk_request(p, r, false);
  }

  // The next item of the part that has keys here, or none at all to see; `at`: its first unit.
  __device__ __forceinline__ bool next(const ChunkParams& p, ChunkItem& I, int64_t& at) {
    while (u < u1) {
      I.first_tok = b * p.item_tokens;
      I.tokens = min(p.item_tokens, q.qo - I.first_tok);
      I.q0 = q.row + I.first_tok;
      I.h = h * p.tile_heads;
      I.qo = q.qo;
      I.kv = q.kv;
      I.pbase = q.pbase;
      I.need = (q.kv + p.page_size - 1) / p.page_size;
      I.keys = chunk_keys(p, q.qo, q.kv, I.first_tok, I.first_tok + I.tokens);
      I.tile0 = I.keys.lo / p.key_tile;
      I.n = chunk_tiles(p, I.keys);
      at = item_start;
      I.t0 = (int)(u - item_start);
      I.t1 = (int)min((int64_t)I.n, u1 - item_start);
      const bool some = I.n > 0 ? I.t0 < I.n : I.t0 == 0;
      item_start += I.n + p.item_cost;
      u = item_start;
      if (++b == q.blocks) {
        b = 0;
        if (++h == p.item_heads) {
          h = 0;
          do {
            if (++r == p.batch) {
              u = u1;
              break;
            }
            q = chunk_request(p, r, false);
          } while (q.blocks == 0);
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

// What the merge has to know of an item that part c begins and does not end:
// {row of its first token, rows, query head, part that holds its last tile}.
__device__ __forceinline__ int4 cut_of(const ChunkParams& p, const ChunkLine& line, const ChunkItem& I, int64_t at,
                                       int c) {
  int last = c + 1;
  while (last + 1 < line.parts && part_start(line.units, line.parts, last + 1) < at + I.n) ++last;
  return make_int4(I.q0, I.tokens * p.tile_heads, I.h, last);
}

}  // namespace pd
