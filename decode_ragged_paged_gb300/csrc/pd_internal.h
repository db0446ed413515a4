// pd_internal.h -- launch parameters and launcher declarations shared between
// the C-ABI layer (pd_api.cu) and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pd.h"

namespace pd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ decode
// Workspace of the split-KV decode (all offsets 256-byte aligned):
//   hdr       int32[64]            hdr[0] = work items, hdr[1] = chunks in total
//   req_info  int4[B]              {first chunk, chunks, chunk length, q row or -1 if skipped}
//   rc_list   int2[max_chunks]     (request, chunk index) of every chunk, longest chunks first
//   part_o    float[max_chunks][Hq][D]   normalised partial outputs
//   part_lse  float[max_chunks][Hq]      their log2-sum-exp2 of scaled scores
struct DecodeParams {
  int32_t batch, hq, hkv, head_dim, page_size, group, heads_per_item, items_per_chunk;
  int32_t nhd;  // pools [page][slot][head][dim] instead of [page][head][slot][dim]
  int32_t total_qo, max_kv_len, num_pages, chunk_target, max_chunks;
  int32_t o_dtype;
  float scale_log2;  // softmax scale times log2(e)
  const int32_t* qo_indptr;  // may be null: row r = request r
  const int32_t* kv_len;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  void* o;
  float* lse;
  int32_t* hdr;
  int4* req_info;
  int2* rc_list;
  float* part_o;
  float* part_lse;
  int32_t* status;
};

struct DecodeLayout {
  size_t hdr, req_info, rc_list, part_o, part_lse, total;
  int32_t chunk_target, max_chunks;
};

// Chunk length and workspace layout of a decode over `batch` requests of at
// most max_kv_len tokens; `sm_count` sizes the split.
DecodeLayout decode_layout(int32_t batch, int32_t hq, int32_t head_dim, int32_t max_kv_len,
                           int32_t items_per_chunk, int32_t sm_count);

// Heads of one group processed together by a decode work item.
int32_t decode_heads_per_item(int32_t group, int32_t head_dim);

// Plans and runs a decode. Returns a pd_status.
int launch_decode(DecodeParams& p, int32_t kv_dtype, cudaStream_t stream);

// ----------------------------------------------------------------- prefill
// Workspace of the tensor-core prefill (offsets 256-byte aligned):
//   hdr      int32[64]     hdr[0] = work items (q tiles x query heads)
//   rq_list  int2[max_rq]  (request, q tile) ordered by decreasing KV-tile count
struct PrefillParams {
  int32_t batch, hq, hkv, group, page_size, num_pages, total_qo, max_qo_len, max_kv_len, causal, o_dtype;
  int32_t max_rq;
  // GQA packing: a 128-row tile holds tile_rows query rows x tile_heads query
  // heads of one KV head (tile_heads = the group, or 1); items per q tile =
  // item_heads = hq / tile_heads
  int32_t tile_heads, tile_rows, item_heads;
  int32_t nhd;       // pools [page][slot][head][dim] instead of [page][head][slot][dim]
  float scale_log2;  // softmax scale times log2(e)
  const int32_t* qo_indptr;
  const int32_t* kv_len;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  void* o;
  float* lse;
  int32_t* hdr;
  int2* rq_list;
  int32_t* status;
};

struct PrefillLayout {
  size_t hdr, rq_list, total;
  int32_t max_rq;
};

// Query heads a prefill tile packs for this group size (the group when it
// divides 128, else 1).
int32_t prefill_tile_heads(int32_t group);
PrefillLayout prefill_layout(int32_t batch, int32_t total_qo, int32_t max_qo_len, int32_t tile_heads);

// Workspace of pd_attn_mixed_split: the prefill part at 0, the decode part at
// `decode` (bytes).
struct MixedSplitLayout {
  size_t decode, total;
};
MixedSplitLayout mixed_split_layout(const pd_attn_desc* d, const pd_batch* b);

// Checks what the tensor-core prefill supports; returns a pd_status.
int prefill_supported(int32_t kv_dtype, int32_t head_dim, int32_t page_size);

// Plans and runs a prefill over bf16 q / pools. Returns a pd_status.
int launch_prefill(PrefillParams& p, const void* q, const void* k_pool, const void* v_pool, cudaStream_t stream);

// --------------------------------------------------------------- KV copies
struct KvCopyParams {
  int32_t batch, hkv, head_dim, page_size, num_layers, num_pages, elem_size;
  int32_t head_begin, head_count;    // pack / unpack: pool heads [head_begin, head_begin + head_count)
  int32_t layer_begin, layer_count;  // pack: layers [layer_begin, layer_begin + layer_count) of num_layers
  int32_t max_kv_len, max_new;
  int32_t nhd;                       // pools [page][slot][head][dim] instead of [page][head][slot][dim]
  int64_t layer_stride;
  const int32_t* new_indptr;   // append only
  const int32_t* kv_len;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  const void* src;             // append: k_new; pack: k pool; unpack: packed buffer
  const void* src2;            // append: v_new; pack: v pool
  void* dst;                   // append: k pool; pack: packed buffer; unpack: k pool
  void* dst2;                  // append: v pool; unpack: v pool
  const int64_t* offsets;      // pack: dst offsets; unpack: src offsets
  int64_t buf_bytes;           // size of the packed buffer
  int32_t* status;
};

int launch_kv_append(const KvCopyParams& p, cudaStream_t stream);
int launch_kv_pack(const KvCopyParams& p, cudaStream_t stream);
int launch_kv_unpack(const KvCopyParams& p, cudaStream_t stream);

// -------------------------------------------------------------- MLA decode
// Workspace (offsets 256-byte aligned):
//   hdr        int32[64]   hdr[0] = chunks listed, hdr[1] = chunk length
//   req_info   int4[B]     {first chunk, chunks, kv_len or -1 if invalid, 0}
//   chunk_list int2[max_chunks]  (request, chunk) longest first
//   part_lse   float[max_chunks][Hq]        log2-sum-exp2 of scaled scores
//   part_o     float[max_chunks][Hq][512]   normalised partial outputs
struct MlaParams {
  int32_t batch, hq, page_size, num_pages, max_kv_len, o_dtype, pairs, max_chunks;
  float scale_log2;  // softmax scale times log2(e)
  const int32_t* kv_len;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  void* o;
  float* lse;
  int32_t* hdr;
  int4* req_info;
  int2* chunk_list;
  int32_t* split_list;  // requests cut into several chunks (hdr[2] of them)
  float* part_lse;
  float* part_o;
  int32_t* status;
};

struct MlaLayout {
  size_t hdr, req_info, chunk_list, split_list, part_lse, part_o, total;
  int32_t max_chunks;
};

// What the MLA kernel supports (latent 512 + rope 64, bf16, 1..128 heads,
// page size a power of two in [16, 256]); returns a pd_status.
int mla_supported(int32_t d_c, int32_t d_r, int32_t dtype, int32_t hq, int32_t page_size);
// CTA pairs of the persistent MLA grid (one CTA per SM).
int mla_pairs();
MlaLayout mla_layout(int32_t batch, int32_t hq);
int launch_mla(MlaParams& p, const void* q, const void* kv_pool, cudaStream_t stream);

// ------------------------------------------------------------------ tables
struct TablesParams {
  int32_t batch, page_size, num_pages, table_rows, table_cols, total_qo, max_page_indices, free_capacity;
  int32_t hash_size;  // entries of the duplicate-row table in shared memory (0: rows == NULL)
  const int32_t* rows;
  const int32_t* cached_len;
  const int32_t* new_len;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* qo_indptr;
  int32_t* kv_len;
  int32_t* page_indptr;
  int32_t* page_indices;
  int32_t* positions;
  int64_t* slot_map;
  int32_t* status;
};
constexpr int32_t kTablesMaxBatch = 8192;  // the sums of a batch stay in shared memory
int launch_batch_tables(TablesParams& p, cudaStream_t stream);

struct SlotMapParams {
  int32_t batch, page_size, num_pages, total_qo, max_kv_len;
  const int32_t* qo_indptr;
  const int32_t* kv_len;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  int32_t* positions;
  int64_t* slot_map;
  int32_t* status;
};
int launch_slot_map(const SlotMapParams& p, cudaStream_t stream);

// ----------------------------------------------------------- norm and rope
struct NormRopeParams {
  int32_t tokens, hq, hkv, head_dim, rope_dim, interleaved, page_size, num_pages, nhd;
  // set by the launcher: lanes of a head, heads of a warp's group, groups of a
  // token, groups a work item covers, work items of a token
  int32_t lanes, heads_per_group, q_groups, kv_groups, groups, groups_per_block, blocks;
  int32_t staged;  // inputs through shared memory
  float eps, inv_dim;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements between tokens
  const void* q;
  const void* k;
  const void* v;
  const void* q_weight;
  const void* k_weight;
  const float* inv_freq;
  const int32_t* positions;
  const int64_t* slot_map;  // null: k goes to rows of k_out
  void* q_out;
  void* k_out;  // rows or pool
  void* v_out;  // pool
  int32_t* status;
};
int32_t norm_rope_vec(const NormRopeParams& p, int32_t elem_size, uintptr_t addresses);
int launch_norm_rope(NormRopeParams& p, int32_t elem_size, int32_t vec, cudaStream_t stream);

// --------------------------------------------------------- chunk attention
// An item is (request, block of item_tokens query tokens, tile_heads query
// heads of one KV head); its keys are cut into tiles of kChunkKeys. How the items
// are dealt to the CTAs: pd_chunk.cuh.
// Workspace (offsets 256-byte aligned):
//   hdr        int32[32]        the line's {units, units of a head, units before it, parts, whole blocks, shares}
//   req_first  int32[B + 1]     first block of every request
//   pre        int32[max_blocks + 1]  units of one head before every block, modulo 2^32
//   pos        int32[parts + 1]  where every part of the line starts: its first unit, or
//              with whole items before the line, the shares of the parts before it
//   cuts       int4[parts]       the item that a part begins and does not end
//   part_lse   float[2 * parts][rows]     log2-sum-exp2 of a cut item's part
//   part_o     float[2 * parts][rows][D]  its normalised output
constexpr int kChunkKeys = 64;
// Keys of a request: 2^24 are 2^18 tiles of at most about 0.8 us, so that a warp
// that waits for the item before its own to end stays far below the limit of a wait.
constexpr int kChunkMaxKeys = 1 << 24;
struct ChunkParams {
  int32_t batch, hq, hkv, group, head_dim, page_size, num_pages, total_qo, max_qo_len, max_kv_len;
  int32_t causal, window, o_dtype, nhd;
  int32_t tc;          // the tensor-core kernel takes the call
  int32_t page_shift;  // log2 of a page size that is a power of two, else -1
  int32_t aligned32;   // o and the workspace are 32-byte aligned
  int32_t self_plan;   // every CTA makes the work line for itself
  int32_t uncut;       // an item is one CTA's, and a CTA has one at most: no line, no merge
  int32_t grid;        // CTAs
  int32_t tile_heads, tile_tokens, item_heads, item_tokens, item_cost, min_units, rows, max_blocks, max_parts;
  float scale_log2;  // softmax scale times log2(e)
  int64_t q_stride;  // elements between query tokens
  const int32_t* qo_indptr;
  const int32_t* kv_len;
  const int32_t* page_indptr;
  const int32_t* page_indices;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  void* o;
  float* lse;
  int32_t* hdr;
  int32_t* req_first;
  int32_t* pre;
  int32_t* pos;
  int4* cuts;
  float* part_lse;
  float* part_o;
  int32_t* status;
};
struct ChunkLayout {
  size_t hdr, req_first, pre, pos, cuts, part_lse, part_o, total;
};
// Fills the tiling of p (its sizes and types are set) and returns the workspace layout.
ChunkLayout chunk_layout(ChunkParams& p, int32_t kv_dtype);
// Whether 32 bits number the items and count the line's units, whatever the lengths are.
bool chunk_fits(const ChunkParams& p);
int launch_chunk(ChunkParams& p, int32_t kv_dtype, cudaStream_t stream);

cudaError_t launch_chunk_tc(const ChunkParams& p, cudaStream_t stream);

// ------------------------------------------------------------ tensor maps
bool make_pool_map(CUtensorMap* map, const void* pool, int32_t dtype, int32_t num_pages, int32_t hkv,
                   int32_t page_size, int32_t head_dim, int32_t box_cols, int32_t box_rows, bool swizzle128,
                   bool nhd = false);
bool make_rows_map(CUtensorMap* map, const void* base, int32_t dtype, int32_t total, int32_t hq, int32_t head_dim,
                   int32_t box_cols, int32_t box_rows, bool swizzle128, int32_t box_heads = 1,
                   int64_t row_stride = 0);

// ------------------------------------------------------------------- misc
// SMs of the device, or of the SM partition (green context) the calling thread
// launches into while partition_sms() is set.
int device_sm_count();
// Set (thread-local) while a call launches into an SM partition: grids are
// sized for the partition's SMs, and the kernels' one-time attribute setup,
// which is per context, runs again.
int& partition_sms();

// Events of pd_profile_events() (per host thread); recorded around main kernels.
struct ProfileEvents {
  cudaEvent_t start = nullptr, stop = nullptr;
};
ProfileEvents& profile_events();
// Name of the main kernel the last call of this host thread launched.
const char*& last_kernel();
inline void profile_begin(cudaStream_t s) {
  if (profile_events().start) cudaEventRecord(profile_events().start, s);
}
inline void profile_end(cudaStream_t s) {
  if (profile_events().stop) cudaEventRecord(profile_events().stop, s);
}

// Launches a kernel as a programmatic dependent of the one before it on the
// stream: its CTAs are placed while that one drains, and wait for it (with
// pdl_wait_primary(), before they touch global memory). Not while launches are
// timed alone through the profiling events. An error is the caller's to return and is
// not left behind as the thread's last one, where a later call would find it.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = profile_events().start != nullptr ? 0 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace pd
