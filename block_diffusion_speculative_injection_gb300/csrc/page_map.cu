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

// Both calls are bound by latency: a launch, and then a chain of dependent reads (ids, the
// sequences' counts, page ids).  A CTA walks the whole batch, kPer consecutive entries a thread.  For
// the maps of many rows a cluster of CTAs does so, each for all entries, and shares the rows out; what
// the call reads and changes is changed after all of them have read it.
// 256 sequences with a block of 16 rows each, given back and mapped: 7.8 us for both calls (9.3
// by one CTA, 8.8 by two); 32 prompts of 512 to 4096 rows (79,838 rows, 0.96 MB of maps): 11.9 us, 8
// SMs' instructions for the maps' rows.  No more CTAs than a cluster has, because what they read (counts,
// table, free list) may change only after all have read it, and a cluster has that barrier without a second
// launch: right for the steps of a server, dear for very many rows (4096 sequences of 200: 76 us, bytes 1.5).
constexpr int kMapThreads = 1024, kMapBatch = 4096;
constexpr int kMapCluster = 8, kMapRows = 1024;  // most CTAs; rows a CTA takes before there is another
constexpr int kMapRuns = 4;                      // rows a thread has under way

struct PagesK {
  int32_t *table, *mapped, *free, *n_free, *status;
  int n_pages, n_seqs, pps;
};
struct MapK {
  PagesK p;
  const int32_t *seq_ids, *start, *counts;  // release: start holds the slots kept
  int32_t *offsets, *kv_lens, *row_seq, *row_pos, *row_slot;
  int batch, n_rows;
  int hash;        // places of the table of ids, a power of two >= 2 * batch
  int hash_shift;  // 32 - log2(hash)
  int runs;        // of 32 rows a warp takes at once, 1..kMapRuns
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

// Sums stay at kMapMany, which is above every count of rows and pages that a call can serve
// (so 32 bits do, and saturating addition is still associative).
constexpr int kMapMany = (1 << 30) - 1;
__device__ __forceinline__ int add_sat(int a, int b) { return min(a + b, kMapMany); }

// Prefix sums of two values (0..kMapMany) over the CTA's threads: what lies before this one; and all.
__device__ __forceinline__ void block_scan2(int& a, int& b, int& all_a, int& all_b) {
  __shared__ int2 part[kMapThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a = add_sat(a, x);
      b = add_sat(b, y);
    }
  }
  if (lane == 31) part[warp] = make_int2(a, b);
  __syncthreads();
  int2 p = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, p.x, o), y = __shfl_up_sync(0xffffffffu, p.y, o);
    if (lane >= o) {
      p.x = add_sat(p.x, x);
      p.y = add_sat(p.y, y);
    }
  }
  static_assert(kMapThreads / 32 == 32, "a lane for each warp");
  all_a = __shfl_sync(0xffffffffu, p.x, 31);
  all_b = __shfl_sync(0xffffffffu, p.y, 31);
  const int wa = __shfl_sync(0xffffffffu, p.x, max(warp - 1, 0));
  const int wb = __shfl_sync(0xffffffffu, p.y, max(warp - 1, 0));
  a = __shfl_up_sync(0xffffffffu, a, 1);
  b = __shfl_up_sync(0xffffffffu, b, 1);
  a = add_sat(lane > 0 ? a : 0, warp > 0 ? wa : 0);
  b = add_sat(lane > 0 ? b : 0, warp > 0 ? wb : 0);
  __syncthreads();
}

// Places in the table of ids: an id's place keeps the first entry that names it.  (Multiples of 2^32
// times the golden ratio fall apart, so neighbouring ids hardly ever meet.)
__device__ __forceinline__ int id_place(const MapK& k, const MapSmem& s, int id, int b, bool insert) {
  uint32_t h = (uint32_t)id * 2654435769u >> k.hash_shift;
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

// This thread's entries, read ahead of everything else: id (-1: none or out of range), the
// first and second number of the call, the pages that the sequence has.
template <int kPer>
struct MapEntries {
  int id[kPer], a[kPer], c[kPer], have[kPer];
  bool mine[kPer], good[kPer];  // there is such an entry; its id is a sequence's, and named first here
};

template <int kPer>
__device__ __forceinline__ MapSmem map_begin(const MapK& k, int32_t* sm, MapEntries<kPer>& e) {
  MapSmem s;
  const int n = k.batch + 1, b0 = threadIdx.x * kPer;
  s.id = sm;
  s.end = sm + n;
  s.base = sm + 2 * n;
  s.off = sm + 3 * n;
  s.start = sm + 4 * n;
  s.seen = sm + 5 * n;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    e.mine[i] = b < k.batch;
    e.id[i] = !e.mine[i] ? -1 : k.seq_ids ? k.seq_ids[b] : b;
    e.a[i] = e.mine[i] && k.start ? k.start[b] : 0;
    e.c[i] = e.mine[i] && k.counts ? k.counts[b] : 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    e.good[i] = e.id[i] >= 0 && e.id[i] < k.p.n_seqs;
    e.have[i] = e.good[i] ? k.p.mapped[e.id[i]] : 0;
    if (e.mine[i]) s.id[b0 + i] = e.id[i];
  }
  if (k.seq_ids) {
    for (int i = threadIdx.x; i < k.hash; i += kMapThreads) s.seen[i] = -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e.good[i]) id_place(k, s, e.id[i], b0 + i, true);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      e.good[i] = e.good[i] && id_place(k, s, e.id[i], b0 + i, false) == b0 + i;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) e.good[i] = e.good[i] && e.have[i] >= 0 && e.have[i] <= k.p.pps;
  return s;
}

// first entry, from lo on, whose `end` is above i
__device__ __forceinline__ int entry_above(const int32_t* end, int batch, int i, int lo = 0) {
  int hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

template <int kPer>
__global__ void __launch_bounds__(kMapThreads, 1) pages_map_kernel(const MapK k, const int C) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ int32_t map_smem[];
  const int tid = threadIdx.x, b0 = tid * kPer, rank = blockIdx.x;
  int n_free = *k.p.n_free;
  MapEntries<kPer> e;
  const MapSmem s = map_begin(k, map_smem, e);
  bool bad = false, full = false;
  if (n_free < 0 || n_free > k.p.n_pages) {
    bad = true;
    n_free = 0;
  }
  // what each entry needs: rows and pages
  int rows[kPer], need[kPer];
  int row = 0, page = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    rows[i] = min(max(e.c[i], 0), kMapMany);
    need[i] = 0;
    e.good[i] = e.good[i] && e.a[i] >= 0 && e.c[i] >= 0;
    bad = bad || (e.mine[i] && !e.good[i]);
    if (e.good[i]) {
      const long long end = (long long)e.a[i] + e.c[i];
      e.good[i] = end <= (long long)k.p.pps * kPageSlots;
      if (e.good[i])
        need[i] = max(0, (int)((end + kPageSlots - 1) / kPageSlots) - e.have[i]);
      else
        full = true;
    }
    row = add_sat(row, rows[i]);
    page = add_sat(page, need[i]);
  }
  int all_rows, all_need;
  block_scan2(row, page, all_rows, all_need);
  int at = page;
  bool odd = false;  // an entry that needs pages does not get them
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    if (!e.mine[i]) break;
    const int first = min(row, k.n_rows);
    row = add_sat(row, rows[i]);
    page = add_sat(page, need[i]);
    const bool no_rows = row > k.n_rows;
    if (e.good[i] && ((need[i] > 0 && page > n_free) || no_rows)) {
      full = true;
      odd = odd || need[i] > 0;
      e.good[i] = false;
    }
    if (!e.good[i]) need[i] = 0;
    if (rank == 0) {
      k.offsets[b] = first;
      k.kv_lens[b] = e.good[i] ? e.a[i] + rows[i] : max(e.a[i], 0);
    }
    s.off[b] = first;
    s.start[b] = e.good[i] ? e.a[i] : -1;
    if (b == k.batch - 1) {
      const int all = min(row, k.n_rows);
      if (rank == 0) k.offsets[k.batch] = all;
      s.off[k.batch] = all;
      full = full || row > k.n_rows;
    }
  }
  if (bad) set_dev_status(k.p.status, kDevCheck);
  if (full) set_dev_status(k.p.status, kDevCapacity);
  // Pages are counted over the entries that get them: anew where some do not.
  if (__syncthreads_or(odd)) {
    int none = 0;
    at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) at += need[i];
    block_scan2(at, none, all_need, all_rows);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    if (!e.mine[i]) break;
    s.base[b] = e.have[i] - at;
    at += need[i];
    s.end[b] = at;
  }
  __syncthreads();
  // The three numbers of each packed row.  A page is the table's, or, not there yet, the free list's.
  // (A warp takes up to kMapRuns runs of 32 rows: a thread's next row is mostly of the same entry.)
  if (k.row_seq || k.row_pos || k.row_slot) {
    const int n_packed = s.off[k.batch];
    const int runs = k.runs;
    for (int r0 = (rank * kMapThreads + (tid & ~31)) * runs + (tid & 31); r0 < k.n_rows;
         r0 += runs * C * kMapThreads) {
      int seq[kMapRuns], pos[kMapRuns], pg[kMapRuns];
      int b = 0;
#pragma unroll
      for (int i = 0; i < kMapRuns; ++i) {
        const int r = r0 + i * 32;
        seq[i] = pos[i] = pg[i] = -1;
        if (i >= runs || r >= n_packed) continue;
        if (i == 0 || s.off[b + 1] <= r) b = entry_above(s.off + 1, k.batch, r, b);
        if (s.start[b] < 0) continue;
        seq[i] = s.id[b];
        pos[i] = s.start[b] + (r - s.off[b]);
        const int in_seq = pos[i] / kPageSlots, in_list = in_seq - s.base[b];
        pg[i] = in_list >= (b > 0 ? s.end[b - 1] : 0)
                    ? k.p.free[n_free - 1 - in_list]
                    : k.p.table[(int64_t)seq[i] * k.p.pps + in_seq];
      }
#pragma unroll
      for (int i = 0; i < kMapRuns; ++i) {
        const int r = r0 + i * 32;
        if (i >= runs || r >= k.n_rows) break;
        if (k.row_seq) k.row_seq[r] = seq[i];
        if (k.row_pos) k.row_pos[r] = pos[i];
        if (k.row_slot)
          k.row_slot[r] = pg[i] >= 0 && pg[i] < k.p.n_pages ? pg[i] * kPageSlots + pos[i] % kPageSlots : -1;
      }
    }
  }
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  // from here on the state changes
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (need[i] > 0) k.p.mapped[e.id[i]] = e.have[i] + need[i];
  }
  const int total = s.end[k.batch - 1];
  for (int i = rank * kMapThreads + tid; i < total; i += C * kMapThreads) {
    const int b = entry_above(s.end, k.batch, i);
    k.p.table[(int64_t)s.id[b] * k.p.pps + s.base[b] + i] = k.p.free[n_free - 1 - i];
    k.p.free[n_free - 1 - i] = -1;
  }
  if (rank == 0 && tid == 0 && total > 0) *k.p.n_free = n_free - total;
}

template <int kPer>
__global__ void __launch_bounds__(kMapThreads, 1) pages_release_kernel(const MapK k) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ int32_t map_smem[];
  const int tid = threadIdx.x, b0 = tid * kPer;
  const int n_free = *k.p.n_free;
  MapEntries<kPer> e;
  const MapSmem s = map_begin(k, map_smem, e);
  int give[kPer], keep[kPer];
  int at = 0, none = 0, total, no_total;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    give[i] = keep[i] = 0;
    e.good[i] = e.good[i] && e.a[i] >= 0;
    bad = bad || (e.mine[i] && !e.good[i]);
    if (!e.good[i]) continue;
    keep[i] = (int)(((long long)e.a[i] + kPageSlots - 1) / kPageSlots);
    give[i] = max(0, e.have[i] - keep[i]);
    at = add_sat(at, give[i]);
  }
  block_scan2(at, none, total, no_total);
  // more pages than there are: the counts are not this pool's
  if (n_free < 0 || n_free > k.p.n_pages || total > k.p.n_pages - n_free) {
    if (tid == 0) set_dev_status(k.p.status, kDevCheck);
    return;
  }
  if (bad) set_dev_status(k.p.status, kDevCheck);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    if (!e.mine[i]) break;
    s.base[b] = keep[i] - at;
    at += give[i];
    s.end[b] = at;
    if (give[i] > 0) k.p.mapped[e.id[i]] = keep[i];
  }
  __syncthreads();
  for (int i = tid; i < total; i += kMapThreads) {
    const int b = entry_above(s.end, k.batch, i);
    int32_t* const entry = k.p.table + (int64_t)s.id[b] * k.p.pps + s.base[b] + i;
    k.p.free[n_free + total - 1 - i] = *entry;
    *entry = -1;
  }
  if (tid == 0 && total > 0) *k.p.n_free = n_free + total;
}

static bool pages_ok(const dflash_pages* p) {
  return p && p->page_table_dev && p->n_mapped_dev && p->free_pages_dev && p->n_free_dev &&
         p->status_dev && p->n_pages >= 1 && p->n_seqs >= 1 && p->pages_per_seq >= 1 &&
         p->pages_per_seq <= (1 << 22) && (int64_t)p->n_pages * kPageSlots < ((int64_t)1 << 31) &&
         kvq_ints_aligned({p->page_table_dev, p->n_mapped_dev, p->free_pages_dev, p->n_free_dev,
                           p->status_dev});
}

// n 32-bit words from p on
static MemRange words(const int32_t* p, int64_t n) { return MemRange{p, 4 * n}; }

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
  k.hash_shift = 26;
  for (; k.hash < 2 * batch; k.hash *= 2) --k.hash_shift;
  return k;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_pages_map(const dflash_pages* pages, int32_t batch, int32_t n_rows,
                               const int32_t* seq_ids, const int32_t* start, const int32_t* counts,
                               int32_t* offsets, int32_t* kv_lens, int32_t* row_seq,
                               int32_t* row_pos, int32_t* row_slot, dflash_stream_t stream) {
  if (!pages_ok(pages) || batch < 1 || batch > kMapBatch || n_rows < 0 || n_rows >= (1 << 29) ||
      !counts || !offsets || !kv_lens ||
      !kvq_ints_aligned({seq_ids, start, counts, offsets, kv_lens, row_seq, row_pos, row_slot}))
    return DFLASH_E_INVALID_ARG;
  const MemRange out[] = {words(offsets, batch + 1),
                          words(kv_lens, batch),
                          words(row_seq, n_rows),
                          words(row_pos, n_rows),
                          words(row_slot, n_rows),
                          words(pages->page_table_dev, (int64_t)pages->n_seqs * pages->pages_per_seq),
                          words(pages->n_mapped_dev, pages->n_seqs),
                          words(pages->free_pages_dev, pages->n_pages),
                          words(pages->n_free_dev, 1),
                          words(pages->status_dev, 1)};
  const MemRange in[] = {words(seq_ids, batch), words(start, batch), words(counts, batch)};
  if (!ranges_apart(out, 10, in, 3)) return DFLASH_E_INVALID_ARG;
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
  int C = 1;
  if (row_seq || row_pos || row_slot)
    while (C < kMapCluster && C * kMapRows < n_rows) C *= 2;
  k.runs = std::max(1, std::min(kMapRuns, n_rows / (C * kMapThreads)));
  static std::atomic<bool> smem_done[2][kMaxDevices];
  const int big = batch > kMapThreads;
  const auto kernel = big ? pages_map_kernel<kMapBatch / kMapThreads> : pages_map_kernel<1>;
  if (ensure_smem_attr(smem_done[big], kernel, (int)(map_smem_ints(kMapBatch, 2 * kMapBatch) * 4)) !=
      cudaSuccess)
    return DFLASH_E_CUDA;
  if (launch_k_cluster(true, dim3(C, 1, 1), kernel, dim3(C), dim3(kMapThreads),
                       map_smem_ints(batch, k.hash) * 4, (cudaStream_t)stream, k, C) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_pages_release(const dflash_pages* pages, int32_t batch, const int32_t* seq_ids,
                                   const int32_t* keep, dflash_stream_t stream) {
  if (!pages_ok(pages) || batch < 1 || batch > kMapBatch || !kvq_ints_aligned({seq_ids, keep}))
    return DFLASH_E_INVALID_ARG;
  const MemRange out[] = {words(pages->page_table_dev, (int64_t)pages->n_seqs * pages->pages_per_seq),
                          words(pages->n_mapped_dev, pages->n_seqs),
                          words(pages->free_pages_dev, pages->n_pages),
                          words(pages->n_free_dev, 1),
                          words(pages->status_dev, 1)};
  const MemRange in[] = {words(seq_ids, batch), words(keep, batch)};
  if (!ranges_apart(out, 5, in, 2)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {out[0].p, out[1].p, out[2].p, out[3].p, out[4].p, seq_ids, keep};
  DF_TRY(kvq_ptrs_ok(ptrs, 7));
  MapK k = map_args(pages, batch, seq_ids, keep);
  static std::atomic<bool> smem_done[2][kMaxDevices];
  const int big = batch > kMapThreads;
  const auto kernel = big ? pages_release_kernel<kMapBatch / kMapThreads> : pages_release_kernel<1>;
  if (ensure_smem_attr(smem_done[big], kernel, (int)(map_smem_ints(kMapBatch, 2 * kMapBatch) * 4)) !=
      cudaSuccess)
    return DFLASH_E_CUDA;
  if (launch_k(true, kernel, dim3(1), dim3(kMapThreads), map_smem_ints(batch, k.hash) * 4,
               (cudaStream_t)stream, k) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
