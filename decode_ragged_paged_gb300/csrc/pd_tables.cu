// pd_tables.cu -- block tables, page lists, positions and slots of a serving
// step, built on the GPU from the requests' lengths.
//
// The section "KV Messenger" has the model append a layer's new KV entries to
// their pages; every call of the library finds those pages through a CSR page
// table. This file makes that table, and the slot of every new token, without
// a round trip through the host.
//
// With c cached and n new tokens per request (kv = c + n), pages of P tokens
// and exclusive prefix sums over the requests,
//   qo_indptr   = prefix(n)            page_indptr = prefix(ceil(kv / P))
//   base        = prefix(ceil(kv / P) - ceil(c / P))
//   page j of a request = its block-table entry, or for j >= ceil(c / P) the
//                         free page free[count - 1 - (base + j - ceil(c / P))]
//   position(i) = c + i                slot = page * P + position % P
// Free pages are taken in request order, so a call's result depends on nothing
// but its inputs.
//
// Bound: the launch. The bytes are small (a decode step of 128 requests moves
// 0.15 MB, a server of 1000 long requests 9 MB), so everything is one launch:
// every CTA makes the prefix sums of the whole batch in shared memory for
// itself (three loads and one block scan) and then fills its share of the page
// list and of the rows. No CTA waits on another. Back to back a step takes 4.7 us
// (128 requests), 9.8 us for the 1000 (1 million pages: the search for each entry's
// request, 11.4 over all of them; one search for a run of entries left the others of
// a thread waiting for it, 12.1 us, and 6.2 us for the 128).
#include "pd_common.cuh"
#include "pd_internal.h"
#include "pd_launch.cuh"

namespace pd {

namespace {

constexpr int kTabThreads = 1024;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kFill = 4;  // entries of the page list or rows that a thread works on together
constexpr int kHints = 512;  // places of the page list whose requests are looked up ahead

// Prefix sums over the batch.
struct Sums {
  long long rows, pages, need;
};

__device__ __forceinline__ long long shfl_up64(long long v, int d) {
  return __shfl_up_sync(0xffffffffu, v, d);
}

// Exclusive block scan of three sums; every thread calls it.
__device__ Sums block_scan(Sums v, Sums* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long a = shfl_up64(x.rows, d), b = shfl_up64(x.pages, d), c = shfl_up64(x.need, d);
    if (lane >= d) {
      x.rows += a;
      x.pages += b;
      x.need += c;
    }
  }
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_tot[lane];
    const Sums own = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long a = shfl_up64(w.rows, d), b = shfl_up64(w.pages, d), c = shfl_up64(w.need, d);
      if (lane >= d) {
        w.rows += a;
        w.pages += b;
        w.need += c;
      }
    }
    warp_tot[lane] = Sums{w.rows - own.rows, w.pages - own.pages, w.need - own.need};
  }
  __syncthreads();
  const Sums o = warp_tot[warp];
  return Sums{o.rows + x.rows - v.rows, o.pages + x.pages - v.pages, o.need + x.need - v.need};
}

// Last r in [lo, hi) with pre[r] <= at (pre ascending, pre[lo] <= at).
__device__ __forceinline__ int owner(const int* pre, int lo, int hi, int at) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

constexpr int32_t tables_hash_size(int32_t batch) {
  int32_t n = 64;
  while (n < 2 * batch) n <<= 1;
  return n;
}

constexpr size_t tables_smem(int32_t batch, int32_t hash_size) {
  return sizeof(int) * ((size_t)5 * batch + 2 + hash_size);
}
// What the kernel is allowed, whatever a call's batch takes: a limit of its own for
// each call would be another thread's as well.
constexpr size_t kTabSmem = tables_smem(kTablesMaxBatch, tables_hash_size(kTablesMaxBatch));
static_assert(kTabSmem + kTabWarps * sizeof(Sums) + (kHints + 2) * sizeof(int) <= 232448, "shared memory of a CTA");

}  // namespace

// COMMIT: the batch's sums only, and the free count written in place, for
// calls whose count is read and written in the same word (a second launch, so
// that no CTA of the first reads a count that another has written).
template <bool COMMIT>
__global__ void __launch_bounds__(kTabThreads, 1) batch_tables_kernel(const TablesParams p) {
  extern __shared__ int tab_smem[];
  __shared__ Sums warp_tot[kTabWarps];
  __shared__ int hint[kHints + 1];
  __shared__ unsigned int taken;
  const int B = p.batch, tid = threadIdx.x;
  int* qo = tab_smem;               // [B + 1] rows before request r, at most total_qo
  int* pg = qo + B + 1;             // [B + 1] pages before it, at most max_page_indices
  int* need = pg + B + 1;           // [B] free pages taken before it
  int* old_pages = need + B;        // [B] pages it holds already, -1 for a refused request
  int* table_row = old_pages + B;   // [B] its row of the block table
  int* hash = table_row + B;        // [hash_size] first request of every block-table row
  const bool pops = p.free_pages != nullptr;
  pdl_launch_dependents();
  pdl_wait_primary();
  int avail = pops ? *p.free_count : 0;
  avail = min(max(avail, 0), p.free_capacity);
  if (tid == 0) taken = 0;

  // Every thread takes a run of consecutive requests. The first of them (the only
  // one up to 1024 requests) is read here, ahead of what the rows go through.
  const int per = (B + kTabThreads - 1) / kTabThreads;
  const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
  struct Req {
    int n, c, row;
  };
  auto read = [&](int r) -> Req { return {p.new_len[r], p.cached_len[r], p.rows != nullptr ? p.rows[r] : r}; };
  Req mine0{};
  if (r0 < r1) mine0 = read(r0);

  if (p.rows != nullptr) {
    for (int i = tid; i < p.hash_size; i += kTabThreads) hash[i] = -1;
    __syncthreads();
    // a row listed twice belongs to the first request that lists it
    for (int r = r0; r < r1; ++r) {
      const int row = r == r0 ? mine0.row : p.rows[r];
      if (row < 0 || row >= p.table_rows) continue;
      for (unsigned h = (unsigned)row * 2654435761u;; ++h) {
        int* at = &hash[h & (unsigned)(p.hash_size - 1)];
        const int cur = atomicCAS(at, -1, r);
        if (cur == -1) break;
        if (p.rows[cur] == row) {
          atomicMin(at, r);
          break;
        }
      }
    }
    __syncthreads();
  }

  auto look = [&](int r, const Req& q, int& code) -> Sums {
    Sums s{max(q.n, 0), 0, 0};
    code = PD_DEV_OK;
    const long long kv = (long long)q.n + q.c;
    const int P = p.page_size;
    if (q.n < 0 || q.c < 0 || kv > 0x7fffffffLL) {
      code = PD_DEV_BAD_LENGTH;
      return s;
    }
    // both below 2^31 and rounded up without passing it
    const int old = q.c / P + (q.c % P != 0), tot = (int)kv / P + ((int)kv % P != 0);
    if (tot > p.table_cols) {
      code = PD_DEV_BAD_LENGTH;
      return s;
    }
    bool row_ok = q.row >= 0 && q.row < p.table_rows;
    if (row_ok && p.rows != nullptr) {
      // the row's entry: other rows on the way there are other requests'
      unsigned h = (unsigned)q.row * 2654435761u;
      int at;
      while ((at = hash[h & (unsigned)(p.hash_size - 1)]) != r && p.rows[at] != q.row) ++h;
      row_ok = at == r;
    }
    if (!row_ok) {
      code = PD_DEV_BAD_ROW;
      return s;
    }
    s.pages = tot;
    s.need = pops ? tot - old : 0;
    return s;
  };
  Sums mine{0, 0, 0}, first{0, 0, 0};
  int first_code = PD_DEV_OK;
  for (int r = r0; r < r1; ++r) {
    int code;
    const Sums s = look(r, r == r0 ? mine0 : read(r), code);
    if (r == r0) {
      first = s;
      first_code = code;
    }
    mine.rows += s.rows;
    mine.pages += s.pages;
    mine.need += s.need;
  }
  Sums at = block_scan(mine, warp_tot);
  for (int r = r0; r < r1; ++r) {
    Req q = mine0;
    Sums s = first;
    int code = first_code;
    if (r > r0) {
      q = read(r);
      s = look(r, q, code);
    }
    const Sums end{at.rows + s.rows, at.pages + s.pages, at.need + s.need};
    if (code == PD_DEV_OK && (end.rows > p.total_qo || end.pages > p.max_page_indices)) code = PD_DEV_BAD_INDPTR;
    if (code == PD_DEV_OK && s.need > 0 && end.need > avail) code = PD_DEV_NO_PAGES;
    if (code == PD_DEV_OK && s.need > 0) atomicMax(&taken, (unsigned int)end.need);
    if (!COMMIT) {
      qo[r] = (int)min(at.rows, (long long)p.total_qo);
      pg[r] = (int)min(at.pages, (long long)p.max_page_indices);
      need[r] = (int)min(at.need, (long long)0x7fffffff);
      old_pages[r] = code != PD_DEV_OK ? -1 : (int)(s.pages - s.need);
      table_row[r] = q.row;
      if (blockIdx.x == 0) {
        p.kv_len[r] = code != PD_DEV_OK ? -1 : q.c + (int)s.rows;
        p.qo_indptr[r] = qo[r];
        p.page_indptr[r] = pg[r];
        if (code != PD_DEV_OK) report(p.status, code);
      }
      if (r == B - 1) {
        qo[B] = (int)min(end.rows, (long long)p.total_qo);
        pg[B] = (int)min(end.pages, (long long)p.max_page_indices);
        if (blockIdx.x == 0) {
          p.qo_indptr[B] = qo[B];
          p.page_indptr[B] = pg[B];
        }
      }
    }
    at = end;
  }
  if (!COMMIT && B == 0 && tid == 0) {
    qo[0] = pg[0] = 0;
    if (blockIdx.x == 0) p.qo_indptr[0] = p.page_indptr[0] = 0;
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0 && pops && (COMMIT || p.free_count_out != p.free_count))
    *p.free_count_out = avail - (int)taken;
  if (COMMIT) return;

  // The page lists, then the rows: a few entries of a thread at a time, their
  // searches and their reads of the tables side by side.
  const int nnz = pg[B], real_rows = qo[B];
  const int P = p.page_size;
  const int64_t total = (int64_t)nnz + p.total_qo, stride = (int64_t)gridDim.x * kTabThreads;
  // With several entries a thread, the requests of kHints places of the page list are
  // found first, and an entry's is searched for between two of them.
  const bool hinted = nnz >= kFill * stride;
  int shift = 0;
  if (hinted) {
    while ((nnz >> shift) >= kHints) ++shift;
    for (int k = tid; k <= kHints; k += kTabThreads)
      hint[k] = owner(pg, 0, B, (int)min((int64_t)k << shift, (int64_t)nnz - 1));
    __syncthreads();
  }
  for (int64_t e0 = (int64_t)blockIdx.x * kTabThreads + tid; e0 < total; e0 += kFill * stride) {
    int r[kFill], j[kFill], pos[kFill], page[kFill];
#pragma unroll
    for (int x = 0; x < kFill; ++x) {
      const int64_t e = e0 + x * stride;
      r[x] = -1;
      j[x] = pos[x] = 0;
      page[x] = -1;
      if (e < nnz) {
        const int k = (int)e >> shift;
        r[x] = hinted ? owner(pg, hint[k], hint[k + 1] + 1, (int)e) : owner(pg, 0, B, (int)e);
        j[x] = (int)e - pg[r[x]];
      } else if (e < nnz + (int64_t)real_rows) {
        r[x] = owner(qo, 0, B, (int)(e - nnz));
        if (old_pages[r[x]] >= 0) pos[x] = p.cached_len[r[x]] + (int)(e - nnz) - qo[r[x]];
        j[x] = pos[x] / P;
      }
      if (r[x] >= 0 && old_pages[r[x]] >= 0)
        page[x] = j[x] < old_pages[r[x]]
                      ? p.block_table[(int64_t)table_row[r[x]] * p.table_cols + j[x]]
                      : p.free_pages[avail - 1 - (need[r[x]] + j[x] - old_pages[r[x]])];
    }
#pragma unroll
    for (int x = 0; x < kFill; ++x) {
      const int64_t e = e0 + x * stride;
      if (e >= total) break;
      const bool served = r[x] >= 0 && old_pages[r[x]] >= 0, known = page[x] >= 0 && page[x] < p.num_pages;
      if (e < nnz) {
        if (served && j[x] >= old_pages[r[x]]) p.block_table[(int64_t)table_row[r[x]] * p.table_cols + j[x]] = page[x];
        if (served && !known) report(p.status, PD_DEV_BAD_PAGE_TABLE);
        p.page_indices[e] = page[x];
      } else {
        p.positions[e - nnz] = pos[x];
        p.slot_map[e - nnz] = served && known ? (int64_t)page[x] * P + (pos[x] - j[x] * P) : -1;
      }
    }
  }
}

// Positions and slots of the rows of a batch whose page table the caller has:
// one thread per row.
__global__ void __launch_bounds__(256) slot_map_kernel(const SlotMapParams p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.total_qo) return;
  int pos = 0;
  int64_t slot = -1;
  if (p.batch > 0) {
    const int r = owner(p.qo_indptr, 0, p.batch, i);
    const int a = p.qo_indptr[r], b = p.qo_indptr[r + 1];
    if (i >= a && i < b) {
      const int n = p.kv_len[r], pa = p.page_indptr[r], pb = p.page_indptr[r + 1];
      int code = PD_DEV_OK;
      if (a < 0 || pa < 0 || pb < pa) code = PD_DEV_BAD_INDPTR;
      else if (n < b - a || n > p.max_kv_len) code = PD_DEV_BAD_LENGTH;
      else if ((int64_t)(pb - pa) * p.page_size < n) code = PD_DEV_BAD_PAGE_TABLE;
      if (code == PD_DEV_OK) {
        pos = n - (b - a) + (i - a);
        const int page = p.page_indices[pa + pos / p.page_size];
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.page_size + pos % p.page_size;
        else code = PD_DEV_BAD_PAGE_TABLE;
      }
      if (code != PD_DEV_OK) report(p.status, code);
    }
  }
  p.positions[i] = pos;
  p.slot_map[i] = slot;
}

// ------------------------------------------------------------------- host
int launch_batch_tables(TablesParams& p, cudaStream_t stream) {
  p.hash_size = p.rows != nullptr ? tables_hash_size(p.batch) : 0;
  const size_t smem = tables_smem(p.batch, p.hash_size);
  // an entry a thread, up to a CTA per SM
  const int64_t entries = (int64_t)p.max_page_indices + p.total_qo;
  int64_t grid = (entries + kTabThreads - 1) / kTabThreads;
  if (grid > device_sm_count()) grid = device_sm_count();
  if (grid < 1) grid = 1;
  if (allow_smem<batch_tables_kernel<false>>(kTabSmem) != cudaSuccess ||
      allow_smem<batch_tables_kernel<true>>(kTabSmem) != cudaSuccess)
    return PD_ERR_CUDA;
  last_kernel() = "batch_tables_kernel";
  profile_begin(stream);
  cudaError_t e = launch_dependent(batch_tables_kernel<false>, dim3((unsigned)grid), kTabThreads, smem, stream, p);
  profile_end(stream);
  if (e == cudaSuccess && p.free_pages != nullptr && p.free_count == p.free_count_out)
    e = launch_dependent(batch_tables_kernel<true>, dim3(1), kTabThreads, smem, stream, p);
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

int launch_slot_map(const SlotMapParams& p, cudaStream_t stream) {
  last_kernel() = "slot_map_kernel";
  profile_begin(stream);
  const cudaError_t e = launch_dependent(slot_map_kernel, dim3((unsigned)((p.total_qo + 255) / 256)), 256, 0, stream, p);
  profile_end(stream);
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace pd
