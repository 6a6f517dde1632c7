// The 8-bit KV cache: writing rows, reading them back, eviction by accumulated
// attention weight, and the host checks that all dflash_kvq_* calls share.
//
// Format: e4m3 codes in pages of 128 slots, one power-of-two exponent per 16
// slots of a head.  With a power of two, x -> x * 2^-e is exact, so the only
// rounding is the one to e4m3, recoding a block under another exponent moves
// codes by whole binades (lossless above the subnormal codes), and attention can
// fold the exponents into its scores.
#include "kvq.cuh"

namespace dflash {

// ---------------------------------------------------------------------------
// a warp's block: 16 rows of 128 values, eight consecutive values of row
// 2 i + lane / 16 in x[i] (columns 8 (lane % 16) ..)
// ---------------------------------------------------------------------------
struct KvqRows {
  float x[8][8];
};

// exponent of the block (rows not in use hold zeros): non-finite values do not count
__device__ __forceinline__ int block_exponent(const KvqRows& r) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(r.x[i][j]);
      a = m < INFINITY ? fmaxf(a, m) : a;
    }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  return kvq_exponent(a);
}

// codes of eight values under exponent e; a non-finite value becomes NaN
__device__ __forceinline__ uint2 code_row(const float* x, int e) {
  const float s = pow2i(-e);
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = fabsf(x[j]) < INFINITY ? x[j] * s : __int_as_float(0x7fffffff);
  return kvq_encode8(y);
}

// ---------------------------------------------------------------------------
// append: one warp per (batch entry, block of 16 slots, head, K or V).  It reads
// its block's committed codes and new rows whole before it writes, so a block
// has one writer.  Bound by memory: 2 B in and 1 B out per new element.
// ---------------------------------------------------------------------------
struct AppendK {
  KvqK c;
  const int32_t *seq_ids, *start, *counts;
  const bf16* in[2];
  long long stride[2];  // elements between rows
  int batch, rows, n_blk;
};

__global__ void __launch_bounds__(128) kvq_append_kernel(const AppendK p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int kv = (int)(w & 1);
  w >>= 1;
  const int head = (int)(w % p.c.Hkv);
  w /= p.c.Hkv;
  const int blk = (int)(w % p.n_blk);
  w /= p.n_blk;
  if (w >= p.batch) return;
  const int b = (int)w;
  const int seq = kvq_seq(p.c, p.seq_ids, b);
  const int s0 = p.start[b], cnt = p.counts ? p.counts[b] : p.rows;
  if (seq < 0) return;
  if (s0 < 0 || cnt < 0 || cnt > p.rows) {
    set_dev_status(p.c.status, kDevCheck);
    return;
  }
  const long long slot0 = ((long long)(s0 / kKvqSub) + blk) * kKvqSub;
  const long long end = (long long)s0 + cnt;
  if (cnt == 0 || slot0 >= end) return;
  const int page = slot0 < (1LL << 31) ? kvq_page(p.c, seq, (int)(slot0 / kPageSlots)) : -1;
  if (page < 0) {
    set_dev_status(p.c.status, kDevCapacity);
    return;
  }
  const int r0 = (int)(slot0 % kPageSlots);
  const int64_t ph = kvq_ph(p.c, page, head);
  uint8_t* const codes = p.c.c8[kv] + ph * kKvqPageBytes + (int64_t)r0 * kKvqHd;
  int8_t* const ex = p.c.ex[kv] + ph * kKvqSubs + r0 / kKvqSub;
  const int half = lane >> 4, col = (lane & 15) * 8;
  const int n_old = (int)min(16LL, max(0LL, s0 - slot0));
  const int n_live = (int)min(16LL, end - slot0);
  const int e_old = n_old > 0 ? *ex : 0;
  uint4 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 2 * i + half;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < n_old) {
      const uint2 c = *reinterpret_cast<const uint2*>(codes + r * kKvqHd + col);
      raw[i].x = c.x;
      raw[i].y = c.y;
    } else if (r < n_live) {
      const long long row = (long long)b * p.rows + (slot0 + r - s0);
      raw[i] = *reinterpret_cast<const uint4*>(p.in[kv] + row * p.stride[kv] + head * kKvqHd + col);
    }
  }
  KvqRows v;
  const float old_scale = pow2i(e_old);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i + half < n_old) {
      kvq_decode8(make_uint2(raw[i].x, raw[i].y), v.x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v.x[i][j] *= old_scale;
    } else {
      bf16x8_to_f(raw[i], v.x[i]);
    }
  }
  const int e = block_exponent(v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 2 * i + half;
    if (r < n_live && (r >= n_old || e != e_old))
      *reinterpret_cast<uint2*>(codes + r * kKvqHd + col) = code_row(v.x[i], e);
  }
  if (lane == 0) *ex = (int8_t)e;
}

// ---------------------------------------------------------------------------
// read: one thread per eight values of K and of V
// ---------------------------------------------------------------------------
struct ReadK {
  KvqK c;
  const int32_t *seq_ids, *start, *counts;
  bf16* out[2];
  int batch, rows;
};

__global__ void __launch_bounds__(256) kvq_read_kernel(const ReadK p) {
  pdl_trigger();
  pdl_wait();
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  const int col = (int)(t & 15) * 8;
  const long long u = t >> 4;
  const int head = (int)(u % p.c.Hkv);
  const long long row = u / p.c.Hkv;
  const int b = (int)(row / p.rows), j = (int)(row % p.rows);
  if (b >= p.batch) return;
  const int seq = kvq_seq(p.c, p.seq_ids, b);
  const int s0 = p.start ? p.start[b] : 0, cnt = p.counts ? p.counts[b] : p.rows;
  if (seq < 0) return;
  if (s0 < 0 || cnt < 0 || cnt > p.rows) {
    set_dev_status(p.c.status, kDevCheck);
    return;
  }
  if (j >= cnt) return;
  const long long slot = (long long)s0 + j;
  const int page = slot < (1LL << 31) ? kvq_page(p.c, seq, (int)(slot / kPageSlots)) : -1;
  if (page < 0) set_dev_status(p.c.status, kDevCapacity);
  const int r = (int)(slot % kPageSlots);
  const int64_t ph = kvq_ph(p.c, max(page, 0), head);
  uint2 c[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
  int e[2] = {0, 0};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    if (p.out[kv] && page >= 0) {
      c[kv] = *reinterpret_cast<const uint2*>(p.c.c8[kv] + ph * kKvqPageBytes + r * kKvqHd + col);
      e[kv] = p.c.ex[kv][ph * kKvqSubs + r / kKvqSub];
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    if (p.out[kv]) {
      float x[8];
      kvq_decode8(c[kv], x);
      const float s = pow2i(e[kv]);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] *= s;
      *reinterpret_cast<uint4*>(p.out[kv] + (row * p.c.Hkv + head) * kKvqHd + col) = f_to_bf16x8(x);
    }
}

// ---------------------------------------------------------------------------
// eviction.  Select: per (batch entry, head), the K-th largest score of the
// slots before the window by a radix search over the scores mapped to unsigned
// integers of the same order, then the kept slots in order by prefix sums.
// Move: one warp per destination block of 16 gathers its rows and codes them
// under the block's own exponent.
// ---------------------------------------------------------------------------
struct EvictK {
  KvqK c;
  const int32_t *src, *dst, *kv_lens;
  float* score;
  int32_t *kept, *new_lens;
  int batch, budget, window;
};

// order-preserving map of a score: NaN lowest, -0 equal to +0
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// lengths and ids of entry b; false: skip it
__device__ __forceinline__ bool evict_entry(const EvictK& p, int b, int& src, int& dst, int& n) {
  src = kvq_seq(p.c, p.src, b);
  dst = kvq_seq(p.c, p.dst, b);
  n = p.kv_lens[b];
  if (src < 0 || dst < 0) return false;
  if (src == dst || n < 0) {
    set_dev_status(p.c.status, kDevCheck);
    return false;
  }
  if (n > p.c.pps * kPageSlots) {
    set_dev_status(p.c.status, kDevCapacity);
    n = p.c.pps * kPageSlots;
  }
  return true;
}

constexpr int kSelThreads = 512;

__global__ void __launch_bounds__(kSelThreads) kvq_evict_select_kernel(const EvictK p) {
  pdl_trigger();
  pdl_wait();
  const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  int src, dst, n;
  if (!evict_entry(p, b, src, dst, n)) return;
  const int cap = p.c.pps * kPageSlots;
  const float* const sc = p.score + ((int64_t)src * p.c.Hkv + head) * cap;
  float* const dsc = p.score + ((int64_t)dst * p.c.Hkv + head) * cap;
  int32_t* const kept = p.kept + ((int64_t)b * p.c.Hkv + head) * p.budget;
  const int m = min(n, p.budget);
  const int w0 = n <= p.budget ? 0 : n - p.window;  // slots from here on are kept
  const int K = m - (n - w0);                       // kept slots before w0
  if (head == 0 && tid == 0) p.new_lens[b] = m;

  __shared__ int hist[256];
  __shared__ int s_digit, s_left;
  __shared__ int s_warp[2][kSelThreads / 32];
  // threshold: the K-th largest key T, and how many keys equal to T are kept
  uint32_t T = 0xffffffffu;
  int ties = 0;
  if (K > 0) {
    uint32_t prefix = 0;
    int left = K;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < w0; i += kSelThreads) {
        const uint32_t k = score_key(sc[i]);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_digit = d;
        s_left = left;
      }
      __syncthreads();
      prefix = (prefix << 8) | (uint32_t)s_digit;
      left = s_left;
      __syncthreads();
    }
    T = prefix;
    ties = left;
  }
  // kept slots in order: above T, or one of the first `ties` equal to T
  int above0 = 0, equal0 = 0;
  for (int i0 = 0; i0 < w0; i0 += kSelThreads) {
    const int i = i0 + tid;
    const float f = i < w0 ? sc[i] : 0.f;
    const uint32_t k = score_key(f);
    const bool gt = K > 0 && i < w0 && k > T, eq = K > 0 && i < w0 && k == T;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      s_warp[0][warp] = __popc(bg);
      s_warp[1][warp] = __popc(be);
    }
    __syncthreads();
    int above = above0, equal = equal0, ta = 0, te = 0;
    for (int x = 0; x < kSelThreads / 32; ++x) {
      if (x < warp) {
        above += s_warp[0][x];
        equal += s_warp[1][x];
      }
      ta += s_warp[0][x];
      te += s_warp[1][x];
    }
    const uint32_t lt = (1u << lane) - 1u;
    above += __popc(bg & lt);
    equal += __popc(be & lt);
    if (gt || (eq && equal < ties)) {
      const int at = above + min(equal, ties);
      kept[at] = i;
      dsc[at] = f;
    }
    above0 += ta;
    equal0 += te;
    __syncthreads();
  }
  for (int i = w0 + tid; i < n; i += kSelThreads) {
    kept[K + i - w0] = i;
    dsc[K + i - w0] = sc[i];
  }
  for (int i = m + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
  for (int i = m + tid; i < cap; i += kSelThreads) dsc[i] = 0.f;
}

__global__ void __launch_bounds__(128) kvq_evict_move_kernel(const EvictK p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int n_blk = (p.budget + kKvqSub - 1) / kKvqSub;
  long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int kv = (int)(w & 1);
  w >>= 1;
  const int blk = (int)(w % n_blk);
  w /= n_blk;
  const int head = (int)(w % p.c.Hkv);
  w /= p.c.Hkv;
  if (w >= p.batch) return;
  const int b = (int)w;
  int src, dst, n;
  if (!evict_entry(p, b, src, dst, n)) return;
  const int m = min(n, p.budget), d0 = blk * kKvqSub;
  if (d0 >= m) return;
  const int n_live = min(kKvqSub, m - d0);
  const int dpage = kvq_page(p.c, dst, d0 / kPageSlots);
  if (dpage < 0) {
    set_dev_status(p.c.status, kDevCapacity);
    return;
  }
  // lane r < 16: where row r comes from, and its exponent
  int64_t at = -1;
  int e_src = 0;
  if (lane < n_live) {
    const int s = p.kept[((int64_t)b * p.c.Hkv + head) * p.budget + d0 + lane];
    const int page = kvq_page(p.c, src, s / kPageSlots);
    if (page >= 0) {
      const int64_t ph = kvq_ph(p.c, page, head);
      const int r = s % kPageSlots;
      at = ph * kKvqPageBytes + (int64_t)r * kKvqHd;
      e_src = p.c.ex[kv][ph * kKvqSubs + r / kKvqSub];
    } else {
      set_dev_status(p.c.status, kDevCapacity);
    }
  }
  const int half = lane >> 4, col = (lane & 15) * 8;
  uint2 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t a = __shfl_sync(0xffffffffu, at, 2 * i + half);
    raw[i] = a >= 0 ? *reinterpret_cast<const uint2*>(p.c.c8[kv] + a + col) : make_uint2(0u, 0u);
  }
  KvqRows v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = pow2i(__shfl_sync(0xffffffffu, e_src, 2 * i + half));
    kvq_decode8(raw[i], v.x[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v.x[i][j] *= s;
  }
  const int e = block_exponent(v);
  const int r0 = d0 % kPageSlots;
  const int64_t ph = kvq_ph(p.c, dpage, head);
  uint8_t* const codes = p.c.c8[kv] + ph * kKvqPageBytes + (int64_t)r0 * kKvqHd;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 2 * i + half;
    if (r < n_live) *reinterpret_cast<uint2*>(codes + r * kKvqHd + col) = code_row(v.x[i], e);
  }
  if (lane == 0) p.c.ex[kv][ph * kKvqSubs + r0 / kKvqSub] = (int8_t)e;
}

// ---------------------------------------------------------------------------
// host checks
// ---------------------------------------------------------------------------
bool kvq_cache_ok(const dflash_kvq_cache* c) {
  return c && c->k8_dev && c->v8_dev && c->k_exp_dev && c->v_exp_dev && c->page_table_dev &&
         c->status_dev && c->n_pages >= 1 && c->n_kv_heads >= 1 && c->n_seqs >= 1 &&
         c->pages_per_seq >= 1 && c->pages_per_seq <= (1 << 22) && c->n_kv_heads <= 65535 &&
         (int64_t)c->n_pages * c->n_kv_heads * kPageSlots < ((int64_t)1 << 31) &&
         kvq_aligned(c->k8_dev, 16) && kvq_aligned(c->v8_dev, 16) && kvq_aligned(c->k_exp_dev, 8) &&
         kvq_aligned(c->v_exp_dev, 8) && kvq_aligned(c->page_table_dev, 4) &&
         kvq_aligned(c->status_dev, 4);
}

// A kernel that was handed host memory or another GPU's would fault, so the
// pointers are looked up (about 0.1 us each) before anything is launched.
dflash_status kvq_ptrs_ok(const void* const* ptrs, int n) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return DFLASH_E_CUDA;
  for (int i = 0; i < n; ++i) {
    if (!ptrs[i]) continue;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, ptrs[i]) != cudaSuccess) {
      cudaGetLastError();
      return DFLASH_E_CUDA;
    }
    if (a.type == cudaMemoryTypeManaged) continue;
    if (a.type != cudaMemoryTypeDevice || a.device != dev) return DFLASH_E_INVALID_ARG;
  }
  return DFLASH_OK;
}

dflash_status kvq_cache_ptrs_ok(const dflash_kvq_cache* c) {
  const void* const p[] = {c->k8_dev,    c->v8_dev,         c->k_exp_dev,
                           c->v_exp_dev, c->page_table_dev, c->status_dev};
  return kvq_ptrs_ok(p, 6);
}

KvqK kvq_device_view(const dflash_kvq_cache* c) {
  KvqK k;
  k.c8[0] = static_cast<uint8_t*>(c->k8_dev);
  k.c8[1] = static_cast<uint8_t*>(c->v8_dev);
  k.ex[0] = c->k_exp_dev;
  k.ex[1] = c->v_exp_dev;
  k.tab = c->page_table_dev;
  k.status = c->status_dev;
  k.n_pages = c->n_pages;
  k.Hkv = c->n_kv_heads;
  k.n_seqs = c->n_seqs;
  k.pps = c->pages_per_seq;
  return k;
}

static bool row_stride_ok(int64_t stride, int heads) {
  return stride >= (int64_t)heads * kKvqHd && stride % 8 == 0 && stride < ((int64_t)1 << 31);
}

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_kvq_append(const dflash_kvq_cache* cache, int32_t batch, int32_t rows,
                                const int32_t* seq_ids, const int32_t* start,
                                const int32_t* counts, const void* k, const void* v,
                                int64_t k_row_stride, int64_t v_row_stride,
                                dflash_stream_t stream) {
  if (!kvq_cache_ok(cache) || batch < 1 || rows < 1 || !start || !k || !v || !kvq_aligned(k, 16) ||
      !kvq_aligned(v, 16) || !row_stride_ok(k_row_stride, cache->n_kv_heads) ||
      !row_stride_ok(v_row_stride, cache->n_kv_heads) || rows >= (1 << 30))
    return DFLASH_E_INVALID_ARG;
  AppendK p;
  p.n_blk = (rows + 2 * kKvqSub - 2) / kKvqSub;  // blocks that `rows` slots can touch
  const int64_t warps = (int64_t)batch * p.n_blk * cache->n_kv_heads * 2;
  if (warps >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {seq_ids, start, counts, k, v};
  DF_TRY(kvq_cache_ptrs_ok(cache));
  DF_TRY(kvq_ptrs_ok(ptrs, 5));
  p.c = kvq_device_view(cache);
  p.seq_ids = seq_ids;
  p.start = start;
  p.counts = counts;
  p.in[0] = static_cast<const bf16*>(k);
  p.in[1] = static_cast<const bf16*>(v);
  p.stride[0] = k_row_stride;
  p.stride[1] = v_row_stride;
  p.batch = batch;
  p.rows = rows;
  if (launch_k(true, kvq_append_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0,
               (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_kvq_read(const dflash_kvq_cache* cache, int32_t batch, int32_t rows,
                              const int32_t* seq_ids, const int32_t* start, const int32_t* counts,
                              void* k_out, void* v_out, dflash_stream_t stream) {
  if (!kvq_cache_ok(cache) || batch < 1 || rows < 1 || (!k_out && !v_out) ||
      !kvq_aligned(k_out, 16) || !kvq_aligned(v_out, 16))
    return DFLASH_E_INVALID_ARG;
  if ((int64_t)batch * rows >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  const int64_t threads = (int64_t)batch * rows * cache->n_kv_heads * 16;
  if ((threads + 255) / 256 >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {seq_ids, start, counts, k_out, v_out};
  DF_TRY(kvq_cache_ptrs_ok(cache));
  DF_TRY(kvq_ptrs_ok(ptrs, 5));
  ReadK p;
  p.c = kvq_device_view(cache);
  p.seq_ids = seq_ids;
  p.start = start;
  p.counts = counts;
  p.out[0] = static_cast<bf16*>(k_out);
  p.out[1] = static_cast<bf16*>(v_out);
  p.batch = batch;
  p.rows = rows;
  if (launch_k(true, kvq_read_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0,
               (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_kvq_evict(const dflash_kvq_cache* cache, int32_t batch, const int32_t* src_ids,
                               const int32_t* dst_ids, const int32_t* kv_lens, int32_t max_keys,
                               int32_t budget, int32_t window, float* score, int32_t* kept,
                               int32_t* new_lens, dflash_stream_t stream) {
  if (!kvq_cache_ok(cache) || batch < 1 || batch > 65535 || !src_ids || !dst_ids || !kv_lens ||
      max_keys < 1 || max_keys > (1 << 29) || budget < 1 ||
      budget > cache->pages_per_seq * kPageSlots || window < 0 || window > budget || !score ||
      !kept || !new_lens || !kvq_aligned(score, 4) || !kvq_aligned(kept, 4))
    return DFLASH_E_INVALID_ARG;
  const int64_t warps =
      (int64_t)batch * cache->n_kv_heads * ((budget + kKvqSub - 1) / kKvqSub) * 2;
  if (warps >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {src_ids, dst_ids, kv_lens, score, kept, new_lens};
  DF_TRY(kvq_cache_ptrs_ok(cache));
  DF_TRY(kvq_ptrs_ok(ptrs, 6));
  EvictK p;
  p.c = kvq_device_view(cache);
  p.src = src_ids;
  p.dst = dst_ids;
  p.kv_lens = kv_lens;
  p.score = score;
  p.kept = kept;
  p.new_lens = new_lens;
  p.batch = batch;
  p.budget = budget;
  p.window = window;
  cudaStream_t st = (cudaStream_t)stream;
  if (launch_k(true, kvq_evict_select_kernel, dim3(cache->n_kv_heads, batch), dim3(kSelThreads), 0,
               st, p) != cudaSuccess ||
      launch_k(true, kvq_evict_move_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st,
               p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_kvq_check(const dflash_kvq_cache* cache, dflash_stream_t stream) {
  if (!kvq_cache_ok(cache)) return DFLASH_E_INVALID_ARG;
  DF_TRY(kvq_cache_ptrs_ok(cache));
  cudaStream_t st = (cudaStream_t)stream;
  int32_t s = 0;
  if (cudaMemcpyAsync(&s, cache->status_dev, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (s != 0 && (cudaMemsetAsync(cache->status_dev, 0, 4, st) != cudaSuccess ||
                 cudaStreamSynchronize(st) != cudaSuccess))
    return DFLASH_E_CUDA;
  switch (s) {
    case kDevOk: return DFLASH_OK;
    case kDevCapacity: return DFLASH_E_CAPACITY;
    case kDevTimeout: return DFLASH_E_TIMEOUT;
    default: return DFLASH_E_DEVICE_CHECK;
  }
}

}  // extern "C"
