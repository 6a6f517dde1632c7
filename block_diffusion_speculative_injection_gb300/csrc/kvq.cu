// The 8-bit KV cache: writing rows, reading them back, eviction by accumulated
// attention weight, and the host checks that all dflash_kvq_* calls share.
//
// Format: e4m3 codes in pages of 128 slots, one power-of-two exponent per 16
// slots of a head.  With a power of two, x -> x * 2^-e is exact, so the only
// rounding is the one to e4m3, recoding a block under another exponent moves
// codes by whole binades (lossless above the subnormal codes), and attention can
// fold the exponents into its scores.
#include "kvq.cuh"
#include "packed.cuh"

namespace dflash {

// A warp's block is 16 rows of 128 values: eight consecutive values (columns
// 8 (lane % 16) ..) of the rows 2 i + lane / 16, i < 8, in each lane.  The raw rows are kept
// and decoded twice, for the maximum and for the codes: 32 registers instead of the 64 of
// the values, so that twice as many blocks are in flight.

// running maximum of the finite magnitudes
__device__ __forceinline__ float finite_max(float a, const float* x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = fabsf(x[j]);
    a = m < INFINITY ? fmaxf(a, m) : a;
  }
  return a;
}
__device__ __forceinline__ float warp_max(float a) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  return a;
}
// codes of eight values times s (a power of two); a non-finite value becomes NaN
__device__ __forceinline__ uint2 code_row(const float* x, float s) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = fabsf(x[j]) < INFINITY ? x[j] * s : __int_as_float(0x7fffffff);
  return kvq_encode8(y);
}

// ---------------------------------------------------------------------------
// append: one warp per (batch entry, block of 16 slots, head, K or V).  It reads
// its block's committed codes and new rows whole before it writes, so a block
// has one writer.  Bound by memory: 2 B in and 1 B out per new element; 15,000 rows of
// 8 heads (92 MB) take 21 us, 4.3 TB/s.
//
// Packed rows: `rows` in all, and n_blk units of 16 of them; the r rows of a sequence touch up
// to floor(r / 16) + 2 blocks.  79,838 rows of 8 heads in 32 sequences (491 MB) take 80 us,
// 6.1 TB/s (91 % of a plain copy's rate).
// ---------------------------------------------------------------------------
struct AppendK {
  KvqK c;
  const int32_t *seq_ids, *start, *counts, *offsets;
  const bf16* in[2];
  long long stride[2];  // elements between rows
  int batch, rows;
  long long n_blk;
  PackedUnits units;
};

template <bool kPacked>
__global__ void __launch_bounds__(128, 7) kvq_append_kernel(const AppendK p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int kv = (int)(w & 1);
  int b, blk, cnt, head;
  int first = 0;  // the sequence's first row, packed
  if (kPacked) {
    packed_check(p.offsets, p.batch, p.rows, (long long)blockIdx.x * 128 + threadIdx.x,
                 (long long)gridDim.x * 128, p.c.status);
    w >>= 1;
    head = (int)(w % p.c.Hkv);
    w /= p.c.Hkv;
    if (w >= p.n_blk) return;
    b = packed_find(p.offsets, p.batch, p.units, w);
    if (b < 0 || !packed_rows(p.offsets, b, p.rows, first, cnt)) return;
    blk = (int)(w - packed_base(p.offsets, b, p.units));
  } else {
    w >>= 1;
    head = (int)(w % p.c.Hkv);
    w /= p.c.Hkv;
    blk = (int)(w % p.n_blk);
    w /= p.n_blk;
    if (w >= p.batch) return;
    b = (int)w;
    cnt = p.counts ? p.counts[b] : p.rows;
  }
  const int seq = kvq_seq(p.c, p.seq_ids, b);
  const int s0 = p.start[b];
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
  uint8_t* const codes = (kv ? p.c.c8[1] : p.c.c8[0]) + ph * kKvqPageBytes + (int64_t)r0 * kKvqHd;
  int8_t* const ex = (kv ? p.c.ex[1] : p.c.ex[0]) + ph * kKvqSubs + r0 / kKvqSub;
  const bf16* const in = kv ? p.in[1] : p.in[0];
  const long long stride = kv ? p.stride[1] : p.stride[0];
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
      const long long row = (kPacked ? first : (long long)b * p.rows) + (slot0 + r - s0);
      raw[i] = *reinterpret_cast<const uint4*>(in + row * stride + head * kKvqHd + col);
    }
  }
  const float old_scale = pow2i(e_old);
  auto values = [&](int i, float* x) {
    if (2 * i + half < n_old) {
      kvq_decode8(make_uint2(raw[i].x, raw[i].y), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= old_scale;
    } else {
      bf16x8_to_f(raw[i], x);
    }
  };
  // the largest magnitude: of new rows alone, from the bf16 pairs as integers (where
  // a NaN or an infinity would come out on top: then, and with committed rows
  // in the block, value by value)
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    constexpr uint32_t abs2 = 0x7fff7fffu;
    top = __vimax3_u16x2(top, raw[i].x & abs2, raw[i].y & abs2);
    top = __vimax3_u16x2(top, raw[i].z & abs2, raw[i].w & abs2);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, off));
  const uint32_t top1 = max(top & 0xffffu, top >> 16);
  float a = __uint_as_float(top1 << 16);
  const bool plain = n_old == 0 && top1 < 0x7f80u;
  if (!plain) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      values(i, x);
      a = finite_max(a, x);
    }
    a = warp_max(a);
  }
  const int e = kvq_exponent(a);
  if (plain) {
    const float s = pow2i(-e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      bf16x8_to_f(raw[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= s;
      if (2 * i + half < n_live)
        *reinterpret_cast<uint2*>(codes + (2 * i + half) * kKvqHd + col) = kvq_encode8(x);
    }
    if (lane == 0) *ex = (int8_t)e;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 2 * i + half;
    float x[8];
    values(i, x);
    if (r < n_live && (r >= n_old || e != e_old))
      *reinterpret_cast<uint2*>(codes + r * kKvqHd + col) = code_row(x, pow2i(-e));
  }
  if (lane == 0) *ex = (int8_t)e;
}

// ---------------------------------------------------------------------------
// read: one thread per eight values of K and of V (15,000 rows of 8 heads, 92 MB: 20 us;
// 64,000 rows, 393 MB: 74 us, 5.3 TB/s)
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
// Move: each destination block of 16 gathers its rows and codes them under the
// block's own exponent.
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

// and back
__device__ __forceinline__ float key_score(uint32_t k) {
  return k == 0u ? __int_as_float(0x7fffffff)
                 : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
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

// Select: a cluster of C CTAs per (entry, head), CTA c on the slots [c, c + 1) * chunk of
// the w0 slots before the window.  Three passes find the K-th largest key T eleven bits
// at a time (the last one ten): a histogram of the candidates' next bits in each
// CTA, whose bins that are not empty are added to the cluster's totals (a quarter of
// the bins in each of four CTAs, say) through distributed shared memory.  The keys are held in shared memory after the first pass (what does
// not fit is read again).  Then the kept slots (above T, and the first of those
// equal to T) are counted per warp and written in order.  Bound by latency (loads,
// barriers, shared-memory atomics): 8 lists of 32,768 in clusters of eight 21 us (a first
// form with one CTA a list: 78 us), 256 lists of up to 8192 25 us.
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 8192;  // keys a CTA holds
constexpr int kSelCluster = 8;  // most CTAs of a cluster
// [3][bins] histograms, [3][bins] totals, keys; the dynamic part of the shared memory
constexpr int kSelSmem = (6 * kSelBins + kSelKeys) * 4;

__global__ void __launch_bounds__(kSelThreads) kvq_evict_select_kernel(const EvictK p, const int C) {
  pdl_trigger();
  pdl_wait();
  const int head = blockIdx.x / C, rank = blockIdx.x % C, b = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  int src, dst, n;
  if (!evict_entry(p, b, src, dst, n)) return;  // the whole cluster
  const int64_t cap = (int64_t)p.c.pps * kPageSlots;
  const float* const sc = p.score + ((int64_t)src * p.c.Hkv + head) * cap;
  float* const dsc = p.score + ((int64_t)dst * p.c.Hkv + head) * cap;
  int32_t* const kept = p.kept + ((int64_t)b * p.c.Hkv + head) * p.budget;
  const int m = min(n, p.budget);
  const int w0 = n <= p.budget ? 0 : n - p.window;  // slots from here on are kept
  const int K = m - (n - w0);                       // kept slots before w0
  const int all = C * kSelThreads, gid = rank * kSelThreads + tid;
  // what needs no selection: the window, and the ends of the lists
  auto rest = [&]() {
    for (int i = w0 + gid; i < n; i += all) {
      kept[K + i - w0] = i;
      dsc[K + i - w0] = sc[i];
    }
    for (int i = m + gid; i < p.budget; i += all) kept[i] = -1;
    for (int64_t i = m + gid; i < cap; i += all) dsc[i] = 0.f;
  };
  if (K == 0) {
    rest();
    return;
  }

  extern __shared__ uint32_t sel_smem[];
  uint32_t* const hist = sel_smem;
  uint32_t* const total = C > 1 ? sel_smem + 3 * kSelBins : hist;
  uint32_t* const held = sel_smem + 6 * kSelBins;
  __shared__ uint32_t s_digit, s_left;
  __shared__ uint32_t s_cnt[2];               // this CTA's keys above and equal to T
  __shared__ uint32_t s_warp[2][kSelWarps];
  // whole warps' worth of slots per CTA, so that every warp's share is 32 x something
  const int chunk = (w0 + C * kSelThreads - 1) / (C * kSelThreads) * kSelThreads;
  const int i0 = rank * chunk, i1 = min(w0, i0 + chunk);
  auto key_at = [&](int i) -> uint32_t {
    return i - i0 < kSelKeys ? held[i - i0] : score_key(sc[i]);
  };
  for (int i = tid; i < (C > 1 ? 6 : 3) * kSelBins; i += kSelThreads) sel_smem[i] = 0;
  // (before another CTA adds to the totals)
  auto sync_all = [&]() {
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  sync_all();
  // T's known high bits, and the rank of T among the keys that share them
  uint32_t prefix = 0, left = (uint32_t)K;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    uint32_t* const h = hist + pass * kSelBins;
    constexpr int kU = 8;  // loads in flight
#pragma unroll 1
    for (int i8 = i0 + tid; i8 - tid < i1; i8 += kU * kSelThreads) {
      uint32_t k[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i8 + u * kSelThreads;
        k[u] = i >= i1 ? 0u : pass > 0 && i - i0 < kSelKeys ? held[i - i0] : __float_as_uint(sc[i]);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i8 + u * kSelThreads;
        if (i - tid >= i1) break;
        bool in = i < i1;
        if (pass == 0 || i - i0 >= kSelKeys) k[u] = score_key(__uint_as_float(k[u]));
        if (pass == 0) {
          if (in && i - i0 < kSelKeys) held[i - i0] = k[u];
        } else {
          in = in && (pass == 1 ? (k[u] >> 21) == prefix : (k[u] >> 10) == prefix);
        }
        // (a warp of one bin, as untouched scores of zero make it, adds once)
        const uint32_t bin = (k[u] >> shift) & mask;
        const uint32_t bin0 = __shfl_sync(0xffffffffu, bin, 0);
        if (__all_sync(0xffffffffu, in && bin == bin0)) {
          if (lane == 0) atomicAdd(&h[bin], 32u);
        } else if (in) {
          atomicAdd(&h[bin], 1u);
        }
      }
    }
    // the cluster's histogram, four bins a thread from the top down: thread t has
    // bins 2047 - 4 t - {0, 1, 2, 3}, whose totals are kept by CTA t % C
    uint32_t cnt[4], mine = 0;
    const int base = kSelBins - 4 - 4 * tid;
    uint32_t* const sum = total + pass * kSelBins + base;
    if (C > 1) {
      __syncthreads();
      const uint32_t owner = map_peer(smem_u32(sum), tid % C);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (h[base + j]) red_peer_u32(owner + 4 * j, h[base + j]);
      cluster_sync();
      const float4 v = ld_peer_f32x4(owner);
      cnt[0] = __float_as_uint(v.w);
      cnt[1] = __float_as_uint(v.z);
      cnt[2] = __float_as_uint(v.y);
      cnt[3] = __float_as_uint(v.x);
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) cnt[j] = sum[3 - j];
    }
    mine = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    uint32_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) s_warp[0][warp] = incl;
    __syncthreads();
    // keys in higher bins
    uint32_t before =
        incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[0][lane] : 0u);
    if (before < left && before + mine >= left) {
      int k = 0;
      while (before + cnt[k] < left) before += cnt[k++];
      s_digit = (uint32_t)(base + 3 - k);
      s_left = left - before;
    }
    __syncthreads();
    prefix = pass == 0 ? s_digit : pass == 1 ? (prefix << 11) | s_digit : (prefix << 10) | s_digit;
    left = s_left;
  }
  const uint32_t T = prefix, ties = left;
  // each warp's contiguous share of the chunk: counts, then the kept slots in order
  const int share = chunk / kSelWarps, j0 = i0 + warp * share, j1 = min(i1, j0 + share);
  uint32_t gt = 0, eq = 0;
#pragma unroll 1
  for (int j = j0; j < j1; j += 32) {
    const int i = j + lane;
    const uint32_t k = i < j1 ? key_at(i) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < j1 && k > T));
    eq += __popc(__ballot_sync(0xffffffffu, i < j1 && k == T));
  }
  __syncthreads();  // s_warp is read above
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (warp < 2) {
    const uint32_t sum =
        __reduce_add_sync(0xffffffffu, lane < kSelWarps ? s_warp[warp][lane] : 0u);
    if (lane == 0) s_cnt[warp] = sum;
  }
  sync_all();
  // before this warp: the lower CTAs' (one a lane) and the lower warps' counts
  uint32_t above = lane < warp ? s_warp[0][lane] : 0u, equal = lane < warp ? s_warp[1][lane] : 0u;
  if (lane < rank) {
    above += __float_as_uint(ld_peer_f32(map_peer(smem_u32(&s_cnt[0]), lane)));
    equal += __float_as_uint(ld_peer_f32(map_peer(smem_u32(&s_cnt[1]), lane)));
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 1
  for (int j = j0; j < j1; j += 32) {
    const int i = j + lane;
    const uint32_t k = i < j1 ? key_at(i) : 0u;
    const uint32_t bg = __ballot_sync(0xffffffffu, i < j1 && k > T);
    const uint32_t be = __ballot_sync(0xffffffffu, i < j1 && k == T);
    const uint32_t a = above + __popc(bg & lt), e = equal + __popc(be & lt);
    // (at < K unless the scores changed meanwhile: then no count is to be relied on)
    const uint32_t at = a + min(e, ties);
    if ((((bg >> lane) & 1u) || (((be >> lane) & 1u) && e < ties)) && at < (uint32_t)K) {
      kept[at] = i;
      dsc[at] = key_score(k);
    }
    above += __popc(bg);
    equal += __popc(be);
  }
  rest();
  if (C > 1) cluster_sync();  // no CTA leaves while its counts may be read
}

// Move: one warp per block of 16 destination rows of a head, of K or of V.  Bound by
// the scattered 128-byte reads and, after them, by issue: 64,000 rows of 8 heads (131 MB
// read, as much written) in 62 us, 4.2 TB/s (69 us before the recoding by pairs).
__global__ void __launch_bounds__(128, 10) kvq_evict_move_kernel(const EvictK p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int n_blk = (p.budget + kKvqSub - 1) / kKvqSub;
  uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int kv = (int)(w & 1);
  w >>= 1;
  const int blk = (int)(w % (uint32_t)n_blk);
  w /= (uint32_t)n_blk;
  const int head = (int)(w % (uint32_t)p.c.Hkv), b = (int)(w / (uint32_t)p.c.Hkv);
  if (b >= p.batch) return;
  const int d0 = blk * kKvqSub;
  // lane r < 16: row r's source slot (in bounds of the list; used once it is known
  // how many rows there are)
  int from = -1;
  if (lane < kKvqSub && d0 + lane < p.budget)
    from = p.kept[((int64_t)b * p.c.Hkv + head) * p.budget + d0 + lane];
  int src, dst, n;
  if (!evict_entry(p, b, src, dst, n)) return;
  const int m = min(n, p.budget);
  // Not earlier: new_lens may be kv_lens, which the selection reads everywhere.  Here m is
  // the same from the old length and from the new one.
  if (blk == 0 && head == 0 && kv == 0 && lane == 0) p.new_lens[b] = m;
  if (d0 >= m) return;
  const int n_live = min(kKvqSub, m - d0);
  const int dpage = kvq_page(p.c, dst, d0 / kPageSlots);
  if (dpage < 0) {
    set_dev_status(p.c.status, kDevCapacity);
    return;
  }
  uint8_t* const c8 = kv ? p.c.c8[1] : p.c.c8[0];
  int8_t* const ex = kv ? p.c.ex[1] : p.c.ex[0];
  // its row in the pool (pages * heads * 128 < 2^31) and its exponent
  int at = -1, e_src = 0;
  // (an entry of the list that the selection left open, because scores changed under it, is
  // whatever the caller's memory held: a negative one is no slot, and reads as zero)
  if (lane < n_live && from >= 0) {
    const int page = kvq_page(p.c, src, from / kPageSlots);
    if (page >= 0) {
      at = (int)kvq_ph(p.c, page, head) * kPageSlots + from % kPageSlots;
      e_src = ex[at / kKvqSub];
    } else {
      set_dev_status(p.c.status, kDevCapacity);
    }
  }
  const int half = lane >> 4, col = (lane & 15) * 8;
  uint2 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = __shfl_sync(0xffffffffu, at, 2 * i + half);
    raw[i] = a >= 0 ? *reinterpret_cast<const uint2*>(c8 + (int64_t)a * kKvqHd + col)
                    : make_uint2(0u, 0u);
  }
  // the largest magnitude: of a row's codes as integers (they order like their
  // values, NaN on top: then value by value)
  float a = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    constexpr uint32_t abs2 = 0x007f007fu;
    uint32_t t = __vimax3_u16x2(raw[i].x & abs2, (raw[i].x >> 8) & abs2, raw[i].y & abs2);
    t = __vmaxu2(t, (raw[i].y >> 8) & abs2);
    const uint32_t top = max(t & 0xffffu, t >> 16);
    nan = nan || top == 0x7fu;
    const __half_raw hv = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)top, __NV_E4M3);
    a = fmaxf(a, __half2float(*reinterpret_cast<const __half*>(&hv)) *
                     pow2i(__shfl_sync(0xffffffffu, e_src, 2 * i + half)));
  }
  if (__any_sync(0xffffffffu, nan)) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = pow2i(__shfl_sync(0xffffffffu, e_src, 2 * i + half));
      float x[8];
      kvq_decode8(raw[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= s;
      a = finite_max(a, x);
    }
  }
  const int e = kvq_exponent(warp_max(a));
  const int drow = (int)kvq_ph(p.c, dpage, head) * kPageSlots + d0 % kPageSlots;
  uint8_t* const codes = c8 + (int64_t)(drow + half) * kKvqHd + col;
  // Rows move by k binades, k = their exponent minus the block's.  Within an fp16's range of
  // k the values go by pairs: a code times 2^k is exact in fp16, but for bits far
  // below half a step of the smallest code, so it is rounded once.
  const bool far = lane < n_live && abs(e_src - e) > 14;
  if (!__any_sync(0xffffffffu, far || nan)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = __shfl_sync(0xffffffffu, e_src, 2 * i + half) - e;
      const uint32_t sb = (uint32_t)(k + 15) << 10;  // 2^k in fp16
      const uint32_t s2 = sb | (sb << 16);
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? raw[i].x : raw[i].y;
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h),
                                  *reinterpret_cast<const __half2*>(&s2));
        c[j] = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&y), __NV_SATFINITE,
                                          __NV_E4M3);
      }
      if (2 * i + half < n_live)
        *reinterpret_cast<uint2*>(codes + 2 * i * kKvqHd) =
            make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = pow2i(__shfl_sync(0xffffffffu, e_src, 2 * i + half) - e);
      float x[8];
      kvq_decode8(raw[i], x);
      if (2 * i + half < n_live) *reinterpret_cast<uint2*>(codes + 2 * i * kKvqHd) = code_row(x, s);
    }
  }
  if (lane == 0) ex[drow / kKvqSub] = (int8_t)e;
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

int kvq_sms() {
  static std::atomic<int> sms[kMaxDevices];
  const int dev = current_device_slot();
  if (dev < 0) return 1;
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 1;
    sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

static bool ranges_overlap(const MemRange& a, const MemRange& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < (uint64_t)a.bytes : x - y < (uint64_t)b.bytes;
}
bool ranges_apart(const MemRange* out, int n_out, const MemRange* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(out[i], out[j])) return false;
    for (int j = 0; j < n_in; ++j)
      if (ranges_overlap(out[i], in[j])) return false;
  }
  return true;
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

// n 32-bit words from p on
struct KvqRange {
  const void* p;
  int64_t n;
};
static bool kvq_overlap(const KvqRange& a, const KvqRange& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < (uint64_t)a.n * 4 : x - y < (uint64_t)b.n * 4;
}

static void append_fill(AppendK* p, const dflash_kvq_cache* cache, int batch, int rows,
                        const int32_t* seq_ids, const int32_t* start, const void* k, const void* v,
                        int64_t k_stride, int64_t v_stride) {
  p->c = kvq_device_view(cache);
  p->seq_ids = seq_ids;
  p->start = start;
  p->in[0] = static_cast<const bf16*>(k);
  p->in[1] = static_cast<const bf16*>(v);
  p->stride[0] = k_stride;
  p->stride[1] = v_stride;
  p->batch = batch;
  p->rows = rows;
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
      !row_stride_ok(v_row_stride, cache->n_kv_heads) || rows >= (1 << 30) ||
      !kvq_ints_aligned({seq_ids, start, counts}))
    return DFLASH_E_INVALID_ARG;
  AppendK p;
  p.n_blk = (rows + 2 * kKvqSub - 2) / kKvqSub;  // blocks that `rows` slots can touch
  const int64_t warps = (int64_t)batch * p.n_blk * cache->n_kv_heads * 2;
  if (warps >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {seq_ids, start, counts, k, v};
  DF_TRY(kvq_cache_ptrs_ok(cache));
  DF_TRY(kvq_ptrs_ok(ptrs, 5));
  append_fill(&p, cache, batch, rows, seq_ids, start, k, v, k_row_stride, v_row_stride);
  p.counts = counts;
  p.offsets = nullptr;
  if (launch_k(true, kvq_append_kernel<false>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0,
               (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_kvq_append_packed(const dflash_kvq_cache* cache, int32_t batch, int32_t n_rows,
                                       const int32_t* seq_ids, const int32_t* start,
                                       const int32_t* offsets, const void* k, const void* v,
                                       int64_t k_row_stride, int64_t v_row_stride,
                                       dflash_stream_t stream) {
  if (!kvq_cache_ok(cache) || batch < 1 || n_rows < 1 || !start || !offsets || !k || !v ||
      !kvq_aligned(k, 16) || !kvq_aligned(v, 16) || !row_stride_ok(k_row_stride, cache->n_kv_heads) ||
      !row_stride_ok(v_row_stride, cache->n_kv_heads) || n_rows >= (1 << 30) || batch >= (1 << 26) ||
      !kvq_ints_aligned({seq_ids, start, offsets}))
    return DFLASH_E_INVALID_ARG;
  AppendK p;
  p.n_blk = packed_units(n_rows, batch, kKvqSub, 2);
  p.units = packed_units_of(kKvqSub, 2);
  const int64_t warps = p.n_blk * cache->n_kv_heads * 2;
  if (warps >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {seq_ids, start, offsets, k, v};
  DF_TRY(kvq_cache_ptrs_ok(cache));
  DF_TRY(kvq_ptrs_ok(ptrs, 5));
  append_fill(&p, cache, batch, n_rows, seq_ids, start, k, v, k_row_stride, v_row_stride);
  p.counts = nullptr;
  p.offsets = offsets;
  if (launch_k(true, kvq_append_kernel<true>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0,
               (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_kvq_read(const dflash_kvq_cache* cache, int32_t batch, int32_t rows,
                              const int32_t* seq_ids, const int32_t* start, const int32_t* counts,
                              void* k_out, void* v_out, dflash_stream_t stream) {
  if (!kvq_cache_ok(cache) || batch < 1 || rows < 1 || (!k_out && !v_out) ||
      !kvq_aligned(k_out, 16) || !kvq_aligned(v_out, 16) ||
      !kvq_ints_aligned({seq_ids, start, counts}))
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
      !kept || !new_lens || !kvq_aligned(score, 4) ||
      !kvq_ints_aligned({src_ids, dst_ids, kv_lens, kept, new_lens}))
    return DFLASH_E_INVALID_ARG;
  const int64_t warps = (int64_t)batch * cache->n_kv_heads * ((budget + kKvqSub - 1) / kKvqSub) * 2;
  if (warps >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  // What is written must not be what other CTAs still read; only the lengths may be updated in
  // place (the move kernel writes them).
  const int64_t rows = (int64_t)cache->n_seqs * cache->n_kv_heads;
  const int64_t cap = (int64_t)cache->pages_per_seq * kPageSlots;
  const KvqRange in[] = {{kv_lens, batch},
                         {src_ids, batch},
                         {dst_ids, batch},
                         {cache->page_table_dev, (int64_t)cache->n_seqs * cache->pages_per_seq}};
  const KvqRange out[] = {{new_lens, batch},
                          {kept, (int64_t)batch * cache->n_kv_heads * budget},
                          {score, rows > (INT64_MAX >> 3) / cap ? INT64_MAX >> 3 : rows * cap}};
  for (int i = 0; i < 3; ++i) {
    for (int j = new_lens == kv_lens && i == 0 ? 1 : 0; j < 4; ++j)
      if (kvq_overlap(out[i], in[j])) return DFLASH_E_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (kvq_overlap(out[i], out[j])) return DFLASH_E_INVALID_ARG;
  }
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
  // a CTA for every 4096 slots, up to a cluster of eight, but no more than the two CTAs
  // per SM that fit at once
  int C = 1;
  while (C < kSelCluster && (int64_t)C * 4096 < max_keys &&
         (int64_t)C * 2 * cache->n_kv_heads * batch <= 2 * kvq_sms())
    C *= 2;
  static std::atomic<bool> smem_done[kMaxDevices];
  if (ensure_smem_attr(smem_done, kvq_evict_select_kernel, kSelSmem) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (launch_k_cluster(true, dim3(C, 1, 1), kvq_evict_select_kernel, dim3(cache->n_kv_heads * C, batch),
                       dim3(kSelThreads), kSelSmem, st, p, C) != cudaSuccess ||
      launch_k(true, kvq_evict_move_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st,
               p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_status_check(int32_t* status_dev, dflash_stream_t stream) {
  if (!status_dev || !kvq_aligned(status_dev, 4)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {status_dev};
  DF_TRY(kvq_ptrs_ok(ptrs, 1));
  cudaStream_t st = (cudaStream_t)stream;
  int32_t s = 0;
  if (cudaMemcpyAsync(&s, status_dev, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (s != 0 && (cudaMemsetAsync(status_dev, 0, 4, st) != cudaSuccess ||
                 cudaStreamSynchronize(st) != cudaSuccess))
    return DFLASH_E_CUDA;
  switch (s) {
    case kDevOk: return DFLASH_OK;
    case kDevCapacity: return DFLASH_E_CAPACITY;
    case kDevTimeout: return DFLASH_E_TIMEOUT;
    default: return DFLASH_E_DEVICE_CHECK;
  }
}

dflash_status dflash_kvq_check(const dflash_kvq_cache* cache, dflash_stream_t stream) {
  if (!kvq_cache_ok(cache)) return DFLASH_E_INVALID_ARG;
  DF_TRY(kvq_cache_ptrs_ok(cache));
  return dflash_status_check(cache->status_dev, stream);
}

}  // extern "C"
