// pd_chunk.cuh -- the work of the chunk attention: how (request, token block,
// head) items are dealt to the CTAs.
//
// An item's work is counted in units, one per key tile and item_cost more; pre[b]
// holds the units of one head before block b of the batch.
//   The line. The items in a row, head by head, a head's blocks in batch order,
// cut into equal parts, one per CTA, anywhere between two key tiles: every CTA
// has the same work, and an item that a cut falls into is merged afterwards.
//   Short items. Where there is an item a CTA at most, and none of more than a few
// tiles, they are not cut, and there is no line and no merge.
//   Whole items. Blocks of one request read the same keys. Where there are
// several times more items than CTAs, the first `whole` blocks are dealt out
// item by item, block by block with its heads: the CTAs then stream the same
// keys at the same time, out of L2. What is left makes the line, cut so that
// every CTA's whole items and part come to the same. More work than 32 bits of
// units is dealt out like that too, so that the line stays inside them.
#pragma once

#include <type_traits>

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
  return k.hi > k.lo ? (k.hi - 1) / kChunkKeys + 1 - k.lo / kChunkKeys : 0;
}

// A CTA's share of one item: key tiles [t0, t1) of its n, in turn from t0 + rot on and
// around (tile()).
struct ChunkItem {
  int q0, tokens, first_tok, h;  // row of its first token, tokens, that token's index in the request, query head
  int qo, kv, pbase, need;       // of its request: new tokens, cached ones, page list
  int n, t0, t1, rot, tile0;     // tile0: its first key tile
  KeyRange keys;

  // Key tile that comes i-th.
  __device__ __forceinline__ int tile(int i) const {
    const int t = t0 + rot + i;
    return tile0 + (t < t1 ? t : t - (t1 - t0));
  }
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

// A CTA of NT threads, or with NT = 32 a warp by itself.
template <int NT>
__device__ __forceinline__ void sync_of() {
  if constexpr (NT == 32) __syncwarp();
  else __syncthreads();
}

// Exclusive scan over them, and the total; warp_tot: NT / 32 words of shared memory.
template <int NT, typename V>
__device__ __forceinline__ V scan_exclusive(V v, V* warp_tot, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if constexpr (NT == 32) {
    total = __shfl_sync(0xffffffffu, x, 31);
    return x - v;
  }
  __syncthreads();  // the totals of an earlier scan have been read
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  V w = lane < NT / 32 ? warp_tot[lane] : 0;
#pragma unroll
  for (int d = 1; d < NT / 32; d <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, NT / 32 - 1);
  const V before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp > 0 ? before : 0) + x - v;
}

// What a CTA has to know of the line. Its units are counted in 32 bits (chunk_fits), those of
// all blocks before one (pre) modulo 2^32: only differences inside the line are used.
struct ChunkLine {
  int rem, head, base;  // units of the line, of one head of it, and of one head before it
  int parts, whole;     // parts of the line; blocks dealt out whole before it
  int shares;           // what pos counts up to: the sum of the parts' shares, or 0 if pos is in units
  const int32_t* first; // first block of every request
  const int32_t* pre;   // units of one head before every block
  const int32_t* pos;   // where every part starts

  // Units of one head of the line before its block b.
  __device__ __forceinline__ int before(int b) const { return (int)((uint32_t)pre[b] - (uint32_t)base); }

  // First unit of part c. The shares come to the line's units, or (rounding, CTAs
  // with too much already) to nearly that, and are stretched to it here.
  __device__ __forceinline__ int start(int c) const {
    if (shares == 0) return pos[c];
    return c == parts ? rem : (int)((int64_t)pos[c] * rem / shares);
  }
};

// The line of a batch, by one CTA or one warp: checks the requests, numbers their blocks
// (first [B + 1]), sums the blocks' units (pre [blocks + 1]) and cuts the line
// (pos [max_parts + 1]), in global memory or in the CTA's own shared memory. Every
// word gets one value only, as several warps may make the same line in the same
// place, one still writing what another reads. Ends with a barrier.
template <int NT>
__device__ ChunkLine plan_line(const ChunkParams& p, int32_t* first, int32_t* pre, int32_t* pos, long long* warp_tot) {
  const int tid = threadIdx.x & (NT - 1);
  ChunkLine line{0, 1, 0, 0, 0, 0, first, pre, pos};
  // Blocks are summed in 64 bits: 1024 requests with the same rows (an indptr that falls in between) may have
  // more than 2^31. (The 32 requests of a warp have no more than kSelfBlocks or max_parts each.)
  using Count = std::conditional_t<NT == 32, int, long long>;
  Count carry = 0, total;
  bool over = false;
  for (int r0 = 0; r0 < p.batch; r0 += NT) {
    const int r = r0 + tid;
    const Count n = r < p.batch ? chunk_request(p, r, true).blocks : 0;
    const Count at = carry + scan_exclusive<NT>(n, reinterpret_cast<Count*>(warp_tot), total);
    if (r < p.batch) first[r] = (int)min(at, (Count)p.max_blocks);
    carry += total;
    over = over || carry > p.max_blocks;
    if (over) break;
  }
  const int blocks = (int)carry;  // (unless over)
  if (!over && tid == 0) first[p.batch] = blocks;
  sync_of<NT>();
  if (p.uncut && !over) {
    line.whole = blocks;
    return line;
  }
  long long sum = 0;
  for (int b0 = 0; !over && b0 < blocks; b0 += NT) {
    const int b = b0 + tid;
    int units = 0;
    if (b < blocks) {
      int lo = 0, hi = p.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= b) lo = mid;
        else hi = mid;
      }
      units = block_units(p, p.qo_indptr[lo + 1] - p.qo_indptr[lo], p.kv_len[lo], b - first[lo]);
    }
    int tiles;  // kChunkMaxKeys keeps the sum of NT blocks inside 32 bits
    const int at = scan_exclusive<NT>(units, reinterpret_cast<int*>(warp_tot), tiles);
    if (b < blocks) pre[b] = (int)((uint32_t)sum + (uint32_t)at);
    sum += tiles;
  }
  if (over || sum == 0) {
    // more blocks than rows allow (requests whose rows overlap): none is worked on
    if (tid == 0 && over) report(p.status, PD_DEV_BAD_INDPTR);
    sync_of<NT>();
    return line;
  }
  if (tid == 0) pre[blocks] = (int)(uint32_t)sum;
  sync_of<NT>();
  const int G = p.max_parts, H = p.item_heads;
  const long long units = sum * H;
  // whole items: all rounds but the last, whose items the line evens out
  if ((blocks >= 2 * p.batch && (int64_t)blocks * H >= 3 * (int64_t)G) || units > 0x7fffffffLL)
    line.whole = (int)(((int64_t)blocks * H / G - 1) * G / H);
  line.base = pre[line.whole];
  line.head = line.before(blocks);
  line.rem = line.head * H;
  if (line.whole == 0) {
    line.parts = (int)min((long long)G, (units + p.min_units - 1) / p.min_units);  // at least so many units a part
    const int each = line.rem / line.parts, left = line.rem - each * line.parts;
    for (int c = tid; c <= line.parts; c += NT) pos[c] = each * c + left * c / line.parts;
  } else {
    line.parts = G;
    int shares = 0;
    for (int c0 = 0; c0 < G; c0 += NT) {
      const int c = c0 + tid;
      int share = 0;
      if (c < G) {
        long long has = 0;  // units of this CTA's whole items
        for (int i = c; i < line.whole * H; i += G) has += (uint32_t)pre[i / H + 1] - (uint32_t)pre[i / H];
        share = (int)min(max(units / G - has, 0LL), (long long)(0x7fffffff / G));  // (a sum of 32 bits)
      }
      int some;
      const int at = shares + scan_exclusive<NT>(share, reinterpret_cast<int*>(warp_tot), some);
      if (c < G) pos[c] = at;
      shares += some;
    }
    line.shares = max(shares, 1);  // (no shares: every part but the last starts at 0)
  }
  sync_of<NT>();
  return line;
}

// A small batch's line is made by every warp that needs it for itself, in
// `scratch` (kSelfBytes of shared memory; warps that share it write the same): no
// launch more, and no barrier of the CTA. It takes the warp about 200 cycles per
// 32 requests and per 32 blocks, so a large batch's (over 4 us that way) is left
// in the workspace by the plan kernel, which takes that long to launch and run.
constexpr int kSelfBatch = 128, kSelfBlocks = 512, kSelfParts = 512;
constexpr size_t kSelfBytes = 4 * (kSelfBlocks + 2 + kSelfParts + 2 + kSelfBatch + 2);

__device__ __forceinline__ ChunkLine take_line(const ChunkParams& p, void* scratch) {
  if (!p.self_plan) return ChunkLine{p.hdr[0], p.hdr[1], p.hdr[2], p.hdr[3], p.hdr[4], p.hdr[5], p.req_first, p.pre, p.pos};
  int32_t* pre = static_cast<int32_t*>(scratch);
  int32_t* pos = pre + kSelfBlocks + 2;
  return plan_line<32>(p, pos + kSelfParts + 2, pre, pos, nullptr);
}

// A place among the items: block b of request r, item head h.
struct ChunkPlace {
  int r, b, h;
  ChunkRequest q;

  // The place that lane `x` of the warp has.
  __device__ __forceinline__ ChunkPlace from(int x) const {
    auto get = [x](int v) { return __shfl_sync(0xffffffffu, v, x); };
    return ChunkPlace{get(r), get(b), get(h), {get(q.row), get(q.qo), get(q.kv), get(q.pbase), get(q.blocks)}};
  }

  // `n` blocks on, over requests without any; false past the last request.
  __device__ __forceinline__ bool skip(const ChunkParams& p, int n) {
    b += n;
    while (b >= q.blocks) {
      b -= q.blocks;
      if (++r >= p.batch) return false;
      q = chunk_request(p, r, false);
    }
    return true;
  }
};

struct ChunkWalk {
  // whole items: number `item` of `whole_items`, at place w
  int item = 0, whole_items = 0;
  ChunkPlace w;
  // the part of the line: units [u, u1) from u0 on, in the item that starts at item_start, at place l
  int u = 0, u1 = 0, u0 = 0, item_start = 0;
  ChunkPlace l, line_first;  // line_first: the line's first block

  // To CTA c's work; a whole warp calls it. Returns what the merge has to know of
  // the item that its part begins and does not end: {row of its first token, rows,
  // query head, part that holds its last tile}, the last -1 if there is none; rows
  // -1: the part is empty. The four places that have to be found (the first whole
  // item, both ends of the part, the line's first block) are found by four lanes,
  // so that their searches and reads take the time of one.
  __device__ __forceinline__ int4 begin(const ChunkParams& p, const ChunkLine& line, int c) {
    int4 cut = make_int4(0, 0, 0, -1);
    const int lane = threadIdx.x & 31;
    whole_items = line.whole * p.item_heads;
    item = c;
    const bool has_part = c < line.parts;
    if (has_part) {
      u = line.start(c);
      u1 = line.start(c + 1);
      u0 = u;
    }
    if (!has_part && item >= whole_items) return cut;
    // lane 0: unit u of the line; 1: unit u1 (or the last); 2: the line's first block; 3: the first whole item
    const int at = lane == 1 ? min(u1, line.rem - 1) : min(u, line.rem - 1);
    ChunkPlace here;
    here.h = at / line.head;
    int lo = line.whole, hi = line.first[p.batch], start = 0;
    if (lane < 2) {
      const int rest = at - here.h * line.head;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (line.before(mid) <= rest) lo = mid;
        else hi = mid;
      }
      start = here.h * line.head + line.before(lo);
    } else if (lane == 3) {
      lo = min(c, max(whole_items - 1, 0)) / p.item_heads;
      here.h = c % p.item_heads;
    }
    // last request whose blocks start at or before it (requests without blocks start where the next one does)
    int r0 = 0, r1 = p.batch;
    while (r1 - r0 > 1) {
      const int mid = (r0 + r1) >> 1;
      if (line.first[mid] <= lo) r0 = mid;
      else r1 = mid;
    }
    here.r = r0;
    here.b = lo - line.first[r0];
    here.q = chunk_request(p, r0, false);
    l = here.from(0);
    item_start = __shfl_sync(0xffffffffu, start, 0);
    line_first = here.from(2);
    line_first.h = 0;
    w = here.from(3);
    if (!has_part || u == u1) {
      cut.y = has_part ? -1 : 0;
    } else if (u1 < line.rem) {
      const ChunkPlace e = here.from(1);
      const int s = __shfl_sync(0xffffffffu, start, 1);
      const int end = s + block_units(p, e.q.qo, e.q.kv, e.b) - p.item_cost;  // of its tiles
      if (s >= u && s < u1 && u1 < end) {
        const int t0 = e.b * p.item_tokens;
        cut = make_int4(e.q.row + t0, min(p.item_tokens, e.q.qo - t0) * p.tile_heads, e.h * p.tile_heads, c + 1);
        while (cut.w + 1 < line.parts && line.start(cut.w + 1) < end) ++cut.w;
      }
    }
    return cut;
  }

  static __device__ __forceinline__ void describe(const ChunkParams& p, const ChunkPlace& at, ChunkItem& I) {
    I.first_tok = at.b * p.item_tokens;
    I.tokens = min(p.item_tokens, at.q.qo - I.first_tok);
    I.q0 = at.q.row + I.first_tok;
    I.h = at.h * p.tile_heads;
    I.qo = at.q.qo;
    I.kv = at.q.kv;
    I.pbase = at.q.pbase;
    I.need = (at.q.kv + p.page_size - 1) / p.page_size;
    I.keys = chunk_keys(p, at.q.qo, at.q.kv, I.first_tok, I.first_tok + I.tokens);
    I.tile0 = I.keys.lo / kChunkKeys;
    I.n = chunk_tiles(p, I.keys);
  }

  // The next item that has keys here, or none at all to see.
  __device__ __forceinline__ bool next(const ChunkParams& p, ChunkItem& I) {
    if (item < whole_items) {
      describe(p, w, I);
      I.t0 = I.rot = 0;
      I.t1 = I.n;
      const int block = item / p.item_heads;
      item += (int)gridDim.x;
      if (item < whole_items) {
        w.h = item % p.item_heads;
        if (!w.skip(p, item / p.item_heads - block)) item = whole_items;
      }
      return true;
    }
    while (u < u1) {
      describe(p, l, I);
      I.t0 = u - item_start;
      I.t1 = min(I.n, u1 - item_start);
      const bool some = I.n > 0 ? I.t0 < I.n : I.t0 == 0;
      // Blocks of one request read the same keys, a part each of them, and parts are
      // about as long as one another: so a CTA that has worked off x units goes on at
      // a tile that is x modulo a part's length (where its tiles have one), and the
      // CTAs read the same keys at about the same time, once from HBM.
      I.rot = 0;
      if (I.qo > p.item_tokens) {
        const int length = u1 - u0, ahead = (u - u0 - (I.tile0 + I.t0)) % length;
        I.rot = ahead < 0 ? ahead + length : ahead;
        if (I.rot >= I.t1 - I.t0) I.rot = 0;
      }
      item_start += I.n + p.item_cost;
      u = item_start;
      if (u < u1 && !l.skip(p, 1)) {  // the next head, from the line's first block on
        const int h = l.h + 1;
        l = line_first;
        l.h = h;
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
