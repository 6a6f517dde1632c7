// Pages given back and mapped on the GPU (dflash_pages_map, dflash_pages_release): the page
// table of a cache the caller owns, kept from the requests' lengths without the host.
//
// Mapping is two prefix sums over the batch.  With c_b rows to come behind s_b slots, entry b
// needs  n_b = max(0, ceil((s_b + c_b) / 128) - mapped_b)  pages; its rows start at
// sum_{i<b} c_i, and its new pages are the free list's from
// F - 1 - sum_{i<b} n_i downwards.  Everything is in the entries' order, so equal inputs
// give equal tables, and giving pages back undoes a mapping exactly.
#include "kvq.cuh"
#include "packed.cuh"

namespace dflash {

// One CTA walks the batch (up to kMapBatch entries, kMapPer consecutive ones a thread).
constexpr int kMapThreads = 1024, kMapBatch = 4096, kMapPer = kMapBatch / kMapThreads;
constexpr int kRowThreads = 256;
constexpr int kFusedRows = 4096;  // up to here the same CTA writes the rows' maps

struct PagesK {
  int32_t *table, *mapped, *free, *n_free, *status;
  int n_pages, n_seqs, pps;
};
struct MapK {
  PagesK p;
  const int32_t *seq_ids, *start, *counts;  // release: start holds the slots kept
  int32_t *offsets, *kv_lens, *row_seq, *row_pos, *row_slot;
  int batch, n_rows;
  int hash;  // places of the table of ids, a power of two >= 2 * batch
  int fused;
};

// Shared memory: per entry its id, the pages taken up to and with it, and where in the
// sequence's table its page 0 of that count would lie; then the rows' offsets and starts (-1: no rows),
// then the table of ids.
struct MapSmem {
  int32_t *id, *end, *base, *off, *start, *seen;
};
__host__ __device__ inline size_t map_smem_ints(int batch, int hash) {
  return 5 * (size_t)(batch + 1) + hash;
}

// Inclusive prefix sums of two values over the CTA's threads.
__device__ __forceinline__ void block_scan2(long long& a, long long& b) {
  __shared__ long long part[2][kMapThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    part[0][warp] = a;
    part[1][warp] = b;
  }
  __syncthreads();
  long long pa = lane < warp ? part[0][lane] : 0, pb = lane < warp ? part[1][lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    pa += __shfl_xor_sync(0xffffffffu, pa, o);
    pb += __shfl_xor_sync(0xffffffffu, pb, o);
  }
  a += pa;
  b += pb;
  __syncthreads();
}

// Places in the table of ids: an id's place keeps the first entry that names it.
__device__ __forceinline__ int id_place(const MapK& k, const MapSmem& s, int id, int b, bool insert) {
  uint32_t h = (uint32_t)id * 2654435761u;
  h ^= h >> 15;
  for (int i = 0; i < k.hash; ++i, ++h) {  // (at most half of the places are taken)
    const int at = (int)(h & (uint32_t)(k.hash - 1));
    const int held = insert ? atomicCAS(&s.seen[at], -1, b) : s.seen[at];
    if (held < 0) return -1;
    if (s.id[held] == id) {
      if (insert) atomicMin(&s.seen[at], b);
      return s.seen[at];
    }
  }
  return -1;
}

// Entry b: false when its id is no sequence's, or an earlier entry names the same.
__device__ __forceinline__ bool map_entry(const MapK& k, const MapSmem& s, int b) {
  const int id = s.id[b];
  return id >= 0 && id < k.p.n_seqs && id_place(k, s, id, b, false) == b;
}

__device__ __forceinline__ MapSmem map_begin(const MapK& k, int32_t* sm) {
  MapSmem s;
  const int n = k.batch + 1;
  s.id = sm;
  s.end = sm + n;
  s.base = sm + 2 * n;
  s.off = sm + 3 * n;
  s.start = sm + 4 * n;
  s.seen = sm + 5 * n;
  for (int i = threadIdx.x; i < k.hash; i += kMapThreads) s.seen[i] = -1;
  for (int b = threadIdx.x; b < k.batch; b += kMapThreads) s.id[b] = k.seq_ids ? k.seq_ids[b] : b;
  __syncthreads();
  for (int b = threadIdx.x; b < k.batch; b += kMapThreads)
    if (s.id[b] >= 0 && s.id[b] < k.p.n_seqs) id_place(k, s, s.id[b], b, true);
  __syncthreads();
  return s;
}

// first entry whose `end` is above i
__device__ __forceinline__ int entry_above(const int32_t* end, int batch, int i) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// the three numbers of packed row r of entry b (its rows from `first` on behind `start`
// slots; start < 0: none)
__device__ __forceinline__ void write_row(const MapK& k, int r, int seq, int start, int first) {
  int pos = -1, slot = -1;
  if (start < 0) {
    seq = -1;
  } else {
    pos = start + (r - first);
    const int page = k.p.table[(int64_t)seq * k.p.pps + pos / kPageSlots];
    slot = page >= 0 && page < k.p.n_pages ? page * kPageSlots + pos % kPageSlots : -1;
  }
  if (k.row_seq) k.row_seq[r] = seq;
  if (k.row_pos) k.row_pos[r] = pos;
  if (k.row_slot) k.row_slot[r] = slot;
}

__global__ void __launch_bounds__(kMapThreads) pages_map_kernel(const MapK k) {
  pdl_wait();
  extern __shared__ int32_t map_smem[];
  const MapSmem s = map_begin(k, map_smem);
  const int tid = threadIdx.x, b0 = tid * kMapPer;
  int n_free = *k.p.n_free;
  if (n_free < 0 || n_free > k.p.n_pages) {
    set_dev_status(k.p.status, kDevCheck);
    n_free = 0;
  }
  // what each entry needs: rows and pages
  int rows[kMapPer], need[kMapPer], have[kMapPer], st[kMapPer];
  bool good[kMapPer];
  long long sum_rows = 0, sum_need = 0;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int b = b0 + i;
    rows[i] = need[i] = have[i] = st[i] = 0;
    good[i] = false;
    if (b >= k.batch) continue;
    st[i] = k.start ? k.start[b] : 0;
    rows[i] = max(k.counts[b], 0);
    good[i] = map_entry(k, s, b) && st[i] >= 0 && k.counts[b] >= 0;
    if (good[i]) {
      have[i] = k.p.mapped[s.id[b]];
      good[i] = have[i] >= 0 && have[i] <= k.p.pps;
    }
    if (!good[i]) {
      set_dev_status(k.p.status, kDevCheck);
    } else {
      const long long end = (long long)st[i] + rows[i];
      if (end > (long long)k.p.pps * kPageSlots) {
        set_dev_status(k.p.status, kDevCapacity);
        good[i] = false;
      } else {
        need[i] = max(0, (int)((end + kPageSlots - 1) / kPageSlots) - have[i]);
      }
    }
    sum_rows += rows[i];
    sum_need += need[i];
  }
  long long end_rows = sum_rows, end_need = sum_need;
  block_scan2(end_rows, end_need);
  long long row = end_rows - sum_rows, page = end_need - sum_need;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int b = b0 + i;
    if (b >= k.batch) break;
    const int first = (int)min(row, (long long)k.n_rows);
    if (good[i] && ((need[i] > 0 && page + need[i] > n_free) || row + rows[i] > k.n_rows)) {
      set_dev_status(k.p.status, kDevCapacity);
      good[i] = false;
    }
    k.offsets[b] = first;
    k.kv_lens[b] = good[i] ? st[i] + rows[i] : max(st[i], 0);
    s.off[b] = first;
    s.start[b] = good[i] ? st[i] : -1;
    s.base[b] = good[i] ? need[i] : 0;
    row += rows[i];
    page += need[i];
  }
  // The pages of the entries that get them, counted anew: an entry refused for its rows leaves
  // its pages to nobody.
  long long got = 0, none = 0;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i)
    if (b0 + i < k.batch) got += s.base[b0 + i];
  long long end_got = got;
  block_scan2(end_got, none);
  int at = (int)(end_got - got);
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int b = b0 + i;
    if (b >= k.batch) break;
    const int take = s.base[b];
    s.base[b] = have[i] - at;
    at += take;
    s.end[b] = at;
    if (take > 0) k.p.mapped[s.id[b]] = have[i] + take;
  }
  if (b0 < k.batch && b0 + kMapPer >= k.batch) {  // the last entry's thread
    const int all = (int)min(row, (long long)k.n_rows);
    k.offsets[k.batch] = all;
    s.off[k.batch] = all;
    if (row > k.n_rows) set_dev_status(k.p.status, kDevCapacity);
  }
  __syncthreads();
  const int total = s.end[k.batch - 1];
  for (int i = tid; i < total; i += kMapThreads) {
    const int b = entry_above(s.end, k.batch, i);
    k.p.table[(int64_t)s.id[b] * k.p.pps + s.base[b] + i] = k.p.free[n_free - 1 - i];
    k.p.free[n_free - 1 - i] = -1;
  }
  if (tid == 0 && total > 0) *k.p.n_free = n_free - total;
  if (!k.fused) return;
  __syncthreads();
  for (int r = tid; r < k.n_rows; r += kMapThreads) {
    const bool none_left = r >= s.off[k.batch];
    const int b = none_left ? 0 : entry_above(s.off + 1, k.batch, r);
    write_row(k, r, s.id[b], none_left ? -1 : s.start[b], s.off[b]);
  }
}

// The rows' maps of long batches.
__global__ void __launch_bounds__(kRowThreads) pages_rows_kernel(const MapK k) {
  pdl_wait();
  const int r = blockIdx.x * kRowThreads + threadIdx.x;
  if (r >= k.n_rows) return;
  const bool none_left = r >= k.offsets[k.batch];
  const int b = none_left ? 0 : entry_above(k.offsets + 1, k.batch, r);
  const int first = k.offsets[b];
  int start = -1;
  if (!none_left) {  // an entry that was refused kept its length
    start = k.start ? k.start[b] : 0;
    if (k.kv_lens[b] - start != k.counts[b]) start = -1;
  }
  write_row(k, r, k.seq_ids ? k.seq_ids[b] : b, start, first);
}

__global__ void __launch_bounds__(kMapThreads) pages_release_kernel(const MapK k) {
  pdl_wait();
  extern __shared__ int32_t map_smem[];
  const MapSmem s = map_begin(k, map_smem);
  const int tid = threadIdx.x, b0 = tid * kMapPer;
  const int n_free = *k.p.n_free;
  int give[kMapPer], keep[kMapPer];
  long long sum = 0, none = 0;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int b = b0 + i;
    give[i] = keep[i] = 0;
    if (b >= k.batch) continue;
    const int slots = k.start ? k.start[b] : 0;
    bool good = map_entry(k, s, b) && slots >= 0;
    if (good) {
      const int have = k.p.mapped[s.id[b]];
      good = have >= 0 && have <= k.p.pps;
      keep[i] = (int)(((long long)slots + kPageSlots - 1) / kPageSlots);
      if (good) give[i] = max(0, have - keep[i]);
    }
    if (!good) set_dev_status(k.p.status, kDevCheck);
    sum += give[i];
  }
  long long end = sum;
  block_scan2(end, none);
  long long at = end - sum;
  __shared__ long long s_total;
  if (tid == kMapThreads - 1) s_total = end;
  __syncthreads();
  // more pages than there are: the counts are not this pool's
  const long long total = s_total;
  if (n_free < 0 || total + n_free > k.p.n_pages) {
    if (tid == 0) set_dev_status(k.p.status, kDevCheck);
    return;
  }
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int b = b0 + i;
    if (b >= k.batch) break;
    s.base[b] = keep[i] - (int)at;
    at += give[i];
    s.end[b] = (int)at;
    if (give[i] > 0) k.p.mapped[s.id[b]] = keep[i];
  }
  __syncthreads();
  for (int i = tid; i < (int)total; i += kMapThreads) {
    const int b = entry_above(s.end, k.batch, i);
    int32_t* const e = k.p.table + (int64_t)s.id[b] * k.p.pps + s.base[b] + i;
    k.p.free[n_free + total - 1 - i] = *e;
    *e = -1;
  }
  if (tid == 0 && total > 0) *k.p.n_free = n_free + (int)total;
}

static bool pages_ok(const dflash_pages* p) {
  return p && p->page_table_dev && p->n_mapped_dev && p->free_pages_dev && p->n_free_dev &&
         p->status_dev && p->n_pages >= 1 && p->n_seqs >= 1 && p->pages_per_seq >= 1 &&
         p->pages_per_seq <= (1 << 22) && (int64_t)p->n_pages * kPageSlots < ((int64_t)1 << 31) &&
         kvq_ints_aligned({p->page_table_dev, p->n_mapped_dev, p->free_pages_dev, p->n_free_dev,
                           p->status_dev});
}

// n 32-bit words from p on
struct PagesRange {
  const void* p;
  int64_t n;
};
static bool pages_overlap(const PagesRange& a, const PagesRange& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < (uint64_t)a.n * 4 : x - y < (uint64_t)b.n * 4;
}
// nothing of out[0 .. n_out) overlaps another of them or an input
static bool pages_disjoint(const PagesRange* out, int n_out, const PagesRange* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (pages_overlap(out[i], out[j])) return false;
    for (int j = 0; j < n_in; ++j)
      if (pages_overlap(out[i], in[j])) return false;
  }
  return true;
}

static MapK map_args(const dflash_pages* p, int batch, const int32_t* seq_ids, const int32_t* start) {
  MapK k;
  memset(&k, 0, sizeof(k));
  k.p.table = p->page_table_dev;
  k.p.mapped = p->n_mapped_dev;
  k.p.free = p->free_pages_dev;
  k.p.n_free = p->n_free_dev;
  k.p.status = p->status_dev;
  k.p.n_pages = p->n_pages;
  k.p.n_seqs = p->n_seqs;
  k.p.pps = p->pages_per_seq;
  k.seq_ids = seq_ids;
  k.start = start;
  k.batch = batch;
  k.hash = 64;
  while (k.hash < 2 * batch) k.hash *= 2;
  return k;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_pages_map(const dflash_pages* pages, int32_t batch, int32_t n_rows,
                               const int32_t* seq_ids, const int32_t* start, const int32_t* counts,
                               int32_t* offsets, int32_t* kv_lens, int32_t* row_seq,
                               int32_t* row_pos, int32_t* row_slot, dflash_stream_t stream) {
  if (!pages_ok(pages) || batch < 1 || batch > kMapBatch || n_rows < 0 || n_rows >= (1 << 30) ||
      !counts || !offsets || !kv_lens ||
      !kvq_ints_aligned({seq_ids, start, counts, offsets, kv_lens, row_seq, row_pos, row_slot}))
    return DFLASH_E_INVALID_ARG;
  const PagesRange out[] = {{offsets, batch + 1},
                            {kv_lens, batch},
                            {row_seq, n_rows},
                            {row_pos, n_rows},
                            {row_slot, n_rows},
                            {pages->page_table_dev, (int64_t)pages->n_seqs * pages->pages_per_seq},
                            {pages->n_mapped_dev, pages->n_seqs},
                            {pages->free_pages_dev, pages->n_pages},
                            {pages->n_free_dev, 1},
                            {pages->status_dev, 1}};
  const PagesRange in[] = {{seq_ids, batch}, {start, batch}, {counts, batch}};
  if (!pages_disjoint(out, 10, in, 3)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {out[0].p, out[1].p, out[2].p, out[3].p, out[4].p, out[5].p, out[6].p,
                              out[7].p, out[8].p, out[9].p, seq_ids,  start,    counts};
  DF_TRY(kvq_ptrs_ok(ptrs, 13));
  MapK k = map_args(pages, batch, seq_ids, start);
  k.counts = counts;
  k.offsets = offsets;
  k.kv_lens = kv_lens;
  k.row_seq = row_seq;
  k.row_pos = row_pos;
  k.row_slot = row_slot;
  k.n_rows = n_rows;
  const bool rows = row_seq || row_pos || row_slot;
  k.fused = rows && n_rows <= kFusedRows;
  static std::atomic<bool> smem_done[kMaxDevices];
  if (ensure_smem_attr(smem_done, pages_map_kernel, (int)(map_smem_ints(kMapBatch, 2 * kMapBatch) * 4)) !=
      cudaSuccess)
    return DFLASH_E_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  if (launch_k(true, pages_map_kernel, dim3(1), dim3(kMapThreads), map_smem_ints(batch, k.hash) * 4, st,
               k) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (rows && n_rows > kFusedRows &&
      launch_k(true, pages_rows_kernel, dim3((n_rows + kRowThreads - 1) / kRowThreads),
               dim3(kRowThreads), 0, st, k) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_pages_release(const dflash_pages* pages, int32_t batch, const int32_t* seq_ids,
                                   const int32_t* keep, dflash_stream_t stream) {
  if (!pages_ok(pages) || batch < 1 || batch > kMapBatch || !kvq_ints_aligned({seq_ids, keep}))
    return DFLASH_E_INVALID_ARG;
  const PagesRange out[] = {{pages->page_table_dev, (int64_t)pages->n_seqs * pages->pages_per_seq},
                            {pages->n_mapped_dev, pages->n_seqs},
                            {pages->free_pages_dev, pages->n_pages},
                            {pages->n_free_dev, 1},
                            {pages->status_dev, 1}};
  const PagesRange in[] = {{seq_ids, batch}, {keep, batch}};
  if (!pages_disjoint(out, 5, in, 2)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {out[0].p, out[1].p, out[2].p, out[3].p, out[4].p, seq_ids, keep};
  DF_TRY(kvq_ptrs_ok(ptrs, 7));
  MapK k = map_args(pages, batch, seq_ids, keep);
  static std::atomic<bool> smem_done[kMaxDevices];
  if (ensure_smem_attr(smem_done, pages_release_kernel,
                       (int)(map_smem_ints(kMapBatch, 2 * kMapBatch) * 4)) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (launch_k(true, pages_release_kernel, dim3(1), dim3(kMapThreads),
               map_smem_ints(batch, k.hash) * 4, (cudaStream_t)stream, k) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
