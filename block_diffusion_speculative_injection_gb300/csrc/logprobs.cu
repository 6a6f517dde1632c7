// Log probabilities of given tokens, with the entropy of their distributions and the best
// alternatives (dflash_token_logprobs), from one read of the logits.
//
// With m the row's maximum and d_i = x_i - m,
//   S = sum e^d_i,  T = sum d_i e^d_i,
//   log p_t = d_t - log S,  entropy = -sum p_i log p_i = log S - T / S.
// S and T of parts of a row with maxima m1 <= m join as
//   S += f S1,  T += f (T1 + (m1 - m) S1),  f = e^(m1 - m).
//
// Bound by memory where rows fill the GPU: 2048 rows of 128,256 in bf16 take 84 us, 6.3 TB/s (92 % of
// a plain copy's rate).  With 20 alternatives 512 rows of 151,936 in fp32, 384 of them in use, take
// 40.6 us, 5.7 TB/s: the rest is the selection, whose barriers all CTAs reach at about the same
// time, so that the memory idles meanwhile.  Few rows are bound by latency: 16 such rows with 5
// alternatives take 9.1 us, where their bytes take 1.4.  (Times in this file are from memory: calls in
// a graph whose inputs rotate through 1.2 GB.)
#include <cmath>

#include "attn_util.cuh"
#include "kvq.cuh"

namespace dflash {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpStep = kLpThreads * 16;          // ids of an iteration of a CTA
constexpr int kLpTop = 32;                        // most alternatives
constexpr int kLpKeys = 768;                      // candidates a CTA holds
constexpr int kLpCluster = 8;                     // most CTAs a row
constexpr float kLpLog2e = 1.4426950408889634f;
// d_i are cut off here, where e^d_i is zero in fp32, so that a logit of -inf adds 0 and not
// 0 * inf to T
constexpr float kLpFloor = -200.f;

struct LogpK {
  const void* logits;
  long long stride;  // elements between rows
  const int32_t* tokens;
  float *logp, *entropy, *top_logp;
  int32_t* top_ids;
  int vocab, top;
};

// Sums of a part of a row: maximum, S, T.
struct RowSum {
  float m, s, t;
};
// max that passes NaN on
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lp_exp(float d) { return ex2(d * kLpLog2e); }
__device__ __forceinline__ void raise(RowSum& a, float m) {
  // (from -inf nothing has been added yet; the floor also keeps inf - inf out)
  const float d = fmaxf(a.m - m, kLpFloor), f = lp_exp(d);
  a.t = f * (a.t + d * a.s);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ RowSum join(RowSum a, RowSum b) {
  const float m = max_nan(a.m, b.m);
  raise(a, m);
  raise(b, m);
  a.s += b.s;
  a.t += b.t;
  return a;
}

// Candidates as numbers that order like them: the larger value first, then the lower id.  0 is
// below every logit but -inf and NaN, which are no alternatives.
__device__ __forceinline__ uint64_t lp_key(float x, int id) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 equals 0
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return ((uint64_t)o << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float lp_key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// 16 bytes of logits: the values, the largest (NaN passes), and a word of -inf.
// kAtOnce vectors a thread and iteration, kStages iterations' places in shared memory, kCtas CTAs an
// SM.  152 rows of 151,936 in fp32: 16.6 us with 4 x 3 at 4 CTAs, 22.4 with 2 x 4 at 5, 20.7 with 4 x 2 at 5
// (what is in L2 already: 10.3, 12, 20.2; 512 rows: 48.8, 50.4, 48.7).  With alternatives fp32 needs the
// registers of 3 CTAs (20 of them, 384 of 512 rows in use: 40.6 us, with 4 CTAs of 4 x 2 48.5; but all
// 512 rows 62.3 and 52.7), and in bf16 the lists leave room for 4, and 63 registers (lists short enough
// for 5: 512 rows of 128,256 42.8 -> 51.3 us, 2000 rows 131.2 -> 130.2).
template <typename T>
struct LpVec;
template <>
struct LpVec<float> {
  static constexpr int kN = 4, kAtOnce = 4, kStages = 3, kCtas = 4;  // values; vectors a thread reads at once
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ void get(uint4 r, float* x) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float top(uint4 r) {
    return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)),
                   max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
};
template <>
struct LpVec<bf16> {
  static constexpr int kN = 8, kAtOnce = 2, kStages = 4, kCtas = 5;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ void get(uint4 r, float* x) { bf16x8_to_f(r, x); }
  static __device__ __forceinline__ __nv_bfloat162 pair(const uint32_t& w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ float top(uint4 r) {
    const __nv_bfloat162 m =
        __hmax2_nan(__hmax2_nan(pair(r.x), pair(r.y)), __hmax2_nan(pair(r.z), pair(r.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
};

// (The ring behind these starts at a 128-byte line: without that a loop of loads takes 10 % longer.)
struct alignas(128) LpSums {
  RowSum part[kLpWarps];
  RowSum sums[kLpCluster];   // of all parts, in the first CTA
};
struct alignas(128) LpLists {
  uint64_t keys[kLpKeys];
  uint64_t shorter[kLpKeys];
  uint64_t group_key[kLpThreads / 8];
  uint64_t best[kLpTop];     // the part's alternatives in order, 0 behind the last
  uint64_t all[kLpCluster * kLpTop];
  uint64_t warp_best[2][kLpWarps];
  float group[kLpThreads / 8];
  int count, n_short;
  float floor;
};

__host__ __device__ constexpr int lp_lists_size(bool top) {
  return (int)(sizeof(LpSums) + (top ? sizeof(LpLists) : 0));
}

// Fewer keys than c with the n best among them, to sh.shorter; whole CTA.  The maxima of 32 groups
// are 32 different keys (or zeros), and the n-th largest of them leaves a short list: of 768
// random keys 31 for n = 20.
__device__ __forceinline__ int lp_shorten(const uint64_t* keys, int c, int n, LpLists& sh) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint64_t g = 0;
  for (int i = tid; i < c; i += kLpThreads) g = max(g, keys[i]);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
  if ((lane & 7) == 0) sh.group_key[tid >> 3] = g;
  if (tid == 0) sh.n_short = 0;
  __syncthreads();
  g = sh.group_key[lane];
  int above = 0;
#pragma unroll 1
  for (int j = 0; j < 32; ++j) {
    const uint64_t o = __shfl_sync(0xffffffffu, g, j);
    above += o > g || (o == g && j < lane);
  }
  const int nth = __ffs(__ballot_sync(0xffffffffu, above == n - 1)) - 1;
  const uint64_t least = max(__shfl_sync(0xffffffffu, g, nth), (uint64_t)1);
  for (int i = tid; i < c; i += kLpThreads)
    if (keys[i] >= least) sh.shorter[atomicAdd(&sh.n_short, 1)] = keys[i];
  __syncthreads();
  return sh.n_short;
}

// The n best of c keys (all different but for zeros), in order, to out[0 .. n), zeros behind the
// last; whole CTA.  Each is ranked by counting.
__device__ __forceinline__ void lp_select(const uint64_t* keys, int c, int n, uint64_t* out,
                                          LpLists& sh) {
  const int tid = threadIdx.x;
  if (tid < n) out[tid] = 0;
  if (c > kLpThreads) {
    c = lp_shorten(keys, c, n, sh);
    keys = sh.shorter;
  } else {
    __syncthreads();
  }
  for (int i = tid; i < c; i += kLpThreads) {
    const uint64_t k = keys[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < c; ++j) rank += keys[j] > k;
    if (k != 0 && rank < n) out[rank] = k;
  }
  __syncthreads();
}

// join of the first n (a power of two, up to 32) sums, by a whole warp; in every lane
__device__ __forceinline__ RowSum lp_join(const RowSum* sums, int n) {
  RowSum a = sums[threadIdx.x & (n - 1)];
#pragma unroll 1
  for (int o = n >> 1; o > 0; o >>= 1) {
    RowSum b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
    // (in the order of the lanes, so that all have the same)
    a = (threadIdx.x & o) ? join(b, a) : join(a, b);
  }
  return a;
}

// largest of the threads' keys, in every thread; two calls in a row use different buffers
__device__ __forceinline__ uint64_t lp_block_max(uint64_t b, uint64_t* buffer) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
  if ((threadIdx.x & 31) == 0) buffer[threadIdx.x >> 5] = b;
  __syncthreads();
  b = buffer[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) b = max(b, buffer[w]);
  return b;
}

// The n best of ids f0 .. f1 - 1 in order, one after the other, to out; whole CTA.
template <typename T>
__device__ __noinline__ void lp_rounds(const T* x, int f0, int f1, int n, uint64_t* out, LpLists& sh) {
  uint64_t last = ~0ull;
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    uint64_t b = 0;
#pragma unroll 4
    for (int i = f0 + (int)threadIdx.x; i < f1; i += kLpThreads) {
      const float v = ld_f(x + i);
      const uint64_t key = v > -INFINITY ? lp_key(v, i) : 0;
      if (key < last && key > b) b = key;
    }
    last = lp_block_max(b, sh.warp_best[k & 1]);
    if (threadIdx.x == 0) out[k] = last;
  }
}

// the next fp32 below x (not NaN; -inf stays)
__device__ __forceinline__ float just_below(float x) {
  const int b = __float_as_int(x);
  if (x == -INFINITY) return x;
  return x == 0.f ? __int_as_float((int)0x80000001u) : __int_as_float(b > 0 ? b - 1 : b + 1);
}

// The n-th largest of 32 groups' maxima of the threads' values (NaN counts as +inf), -inf for a +inf
// (a row with a +inf or NaN has no alternatives' values anyway); whole CTA, one warp ranks.  The
// maxima are 32 different values, so it is no more than the n-th best of all.
__device__ __forceinline__ float lp_group_floor(float mx, int n, LpLists& sh) {
  const int tid = threadIdx.x, lane = tid & 31;
  float g = mx != mx ? INFINITY : mx;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  if ((lane & 7) == 0) sh.group[tid >> 3] = g;
  __syncthreads();
  if (tid < 32) {
    g = sh.group[lane];
    int above = 0;  // groups before this one
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(0xffffffffu, g, j);
      above += o > g || (o == g && j < lane);
    }
    if (above == n - 1) sh.floor = g == INFINITY ? -INFINITY : g;
  }
  __syncthreads();
  return sh.floor;
}

// The n best of what the list holds become the list, and sh.best; whole CTA.
__device__ __forceinline__ void lp_cut(int n, LpLists& sh) {
  lp_select(sh.keys, min(sh.count, kLpKeys), n, sh.best, sh);
  if (threadIdx.x < n) sh.keys[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) sh.count = n;  // (zeros among them are no candidates)
  __syncthreads();
}

// The list had no room for all candidates of ids f0 .. f1 - 1 (logits that rise with the id): these
// ids anew, above the n-th best of the ids before them and above their own groups' floor; if that
// is too many as well (many equal ones), one after the other.  Whole CTA; then as lp_cut.  (512 rows
// of 151,936 in fp32, 20 alternatives: 62 us; with logits that are three standard deviations higher
// from id 9000 on 87, with ascending ones 308.)
template <typename T>
__device__ __noinline__ void lp_overflow(const T* x, int f0, int f1, int n, LpLists& sh) {
  const int tid = threadIdx.x;
  for (int i = tid; i < min(sh.count, kLpKeys); i += kLpThreads)
    if ((int)~(uint32_t)sh.keys[i] >= f0) sh.keys[i] = 0;
  __syncthreads();
  lp_cut(n, sh);
  const float before = sh.best[n - 1] != 0 ? lp_key_value(sh.best[n - 1]) : -INFINITY;
  float mx = -INFINITY;
#pragma unroll 16
  for (int i = f0 + tid; i < f1; i += kLpThreads) mx = max_nan(mx, ld_f(x + i));
  const float least = fmaxf(before, just_below(lp_group_floor(mx, n, sh)));
#pragma unroll 16
  for (int i = f0 + tid; i < f1; i += kLpThreads) {
    const float v = ld_f(x + i);
    if (v > least) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kLpKeys) sh.keys[at] = lp_key(v, i);
    }
  }
  __syncthreads();
  if (sh.count > kLpKeys) {
    lp_rounds(x, f0, f1, n, sh.keys + n, sh);
    __syncthreads();
    if (tid == 0) sh.count = 2 * n;
    __syncthreads();
  }
  lp_cut(n, sh);
}

// A row's part of a CTA: the cluster of C CTAs shares the row out.  Each thread has the next
// iterations' loads under way while it works on this one's.  (What it takes: fp32 15 and bf16 9
// instructions a logit with the shares of everything else.)
template <typename T, bool kTopIds>
__global__ void __launch_bounds__(kLpThreads, LpVec<T>::kCtas - (kTopIds ? 1 : 0))
    token_logprobs_kernel(const LogpK p, const int C) {
  pdl_trigger();
  pdl_wait();
  constexpr int E = LpVec<T>::kN, U = LpVec<T>::kAtOnce;
  extern __shared__ __align__(16) uint8_t lp_smem[];
  LpSums& sums = *reinterpret_cast<LpSums*>(lp_smem);
  LpLists& sh = *reinterpret_cast<LpLists*>(lp_smem + sizeof(LpSums));  // (with alternatives only)
  const int row = blockIdx.x / C, rank = blockIdx.x % C, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int n_top = kTopIds ? p.top : 0;
  const int tok = p.tokens ? p.tokens[row] : 0;
  const T* const x = static_cast<const T*>(p.logits) + (long long)row * p.stride;
  // the row: up to E - 1 ids before the first 16-byte boundary, whole vectors, up to E - 1 behind
  const int head = min(p.vocab, (int)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
  const int vecs = (p.vocab - head) / E, tail0 = head + vecs * E;
  const int v0 = (int)((long long)vecs * rank / C), v1 = (int)((long long)vecs * (rank + 1) / C);
  const uint4* const vec = reinterpret_cast<const uint4*>(x + head) + tid;
  // A thread's vectors of the next iterations are on their way into its own places of shared
  // memory (nobody else touches them, so there is nothing to synchronise).
  constexpr int kStages = LpVec<T>::kStages;
  uint4* const ring = reinterpret_cast<uint4*>(lp_smem + lp_lists_size(kTopIds)) + tid;
  int fetched = 0;
  auto fetch = [&](int i0) {
    const uint32_t dst = smem_u32(ring + fetched * (U * kLpThreads));
    fetched = fetched + 1 == kStages ? 0 : fetched + 1;
    if (i0 + kLpThreads * U <= v1) {
#pragma unroll
      for (int u = 0; u < U; ++u) cp_async16(dst + u * kLpThreads * 16, vec + i0 + u * kLpThreads, 16);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * kLpThreads + tid < v1)
          cp_async16(dst + u * kLpThreads * 16, vec + i0 + u * kLpThreads, 16);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(v0 + k * kLpThreads * U);  // (before the token is there)
  if (tok < 0) {  // (the whole cluster) a row that is not in use
    cp_async_wait<0>();
    return;
  }
  if (C > 1) cluster_started_arrive();
  float x_tok = 0.f;
  if (rank == 0 && tid == 0 && p.tokens && tok < p.vocab) x_tok = ld_f(x + tok);
  if (kTopIds && tid == 0) sh.count = 0;
  float m = -INFINITY;  // this thread's maximum, and its sums in two parts each
  float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
  auto raise_to = [&](float top) {
    const float d = fmaxf(m - top, kLpFloor), f = lp_exp(d);
    t2 = mul2(fma2(s2, make_float2(d, d), t2), f);
    s2 = mul2(s2, f);
    m = top;
  };
  auto add = [&](float v) {
    if (v == -INFINITY) return;
    const float top = max_nan(m, v);
    if (!(top == m)) raise_to(top);
    const float d = fmaxf(v - m, kLpFloor), e = lp_exp(d);
    s2.x += e;
    t2.x += e * d;
  };
  auto keep = [&](float v, int id) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kLpKeys) sh.keys[at] = lp_key(v, id);
  };
  // the n best of the ids up to `end` become the list, those from `begun` on having been added to it
  int begun = head + v0 * E;
  auto cut = [&](int end) {
    if (sh.count > kLpKeys)
      lp_overflow(x, begun, end, n_top, sh);
    else
      lp_cut(n_top, sh);
    begun = end;
  };
  if (kTopIds) __syncthreads();
  // the ids before the vectors: candidates with the first ones
  if (rank == 0 && tid < head) {
    const float v = ld_f(x + tid);
    add(v);
    if (kTopIds && v > -INFINITY) keep(v, tid);
  }
  bool open = true;         // not known yet to have `top` candidates
  float floor = -INFINITY;  // values up to here are no candidates any more
  // The floor rises with what has been seen after iteration next_cut, then 4 times as many.  The
  // n-th largest of 32 groups' maxima leaves 32 (H(32) - H(32 - n)) candidates an iteration on
  // average (H: harmonic numbers): 22 for n = 16, but 130 for 32, whose four iterations would often
  // overflow the list.  A cut too many costs 0.3 us of 10.
  int next_cut = n_top > kLpTop / 2 ? 0 : 3;
  int it = 0, at = 0;
#pragma unroll 1
  for (int i0 = v0; i0 < v1; i0 += kLpThreads * U, ++it) {
    uint4 now[U];
    cp_async_wait<kStages - 2>();
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = ring[(at * U + u) * kLpThreads];
    const T* const here = reinterpret_cast<const T*>(ring + at * (U * kLpThreads));
    at = at + 1 == kStages ? 0 : at + 1;
    if (i0 + kLpThreads * U > v1) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * kLpThreads + tid >= v1)
          now[u] = make_uint4(LpVec<T>::kNone, LpVec<T>::kNone, LpVec<T>::kNone, LpVec<T>::kNone);
    }
    fetch(i0 + (kStages - 1) * kLpThreads * U);
    float mx = LpVec<T>::top(now[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) mx = max_nan(mx, LpVec<T>::top(now[u]));
    const float top = max_nan(m, mx);
    if (!(top == m)) raise_to(top);
    if (m != -INFINITY) {
      const float2 minus_m = make_float2(-m, -m);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[E];
        LpVec<T>::get(now[u], v);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          float2 d = add2(make_float2(v[e], v[e + 1]), minus_m);
          d.x = fmaxf(d.x, kLpFloor);
          d.y = fmaxf(d.y, kLpFloor);
          float2 w = mul2(d, kLpLog2e);
          w.x = ex2(w.x);
          w.y = ex2(w.y);
          s2 = add2(s2, w);
          t2 = fma2(w, d, t2);
        }
      }
    }
    if (!kTopIds) continue;
    const bool opened = open;
    float low = 0.f;
    if (opened) {
      low = lp_group_floor(mx, n_top, sh);
      floor = just_below(low);
      open = low == -INFINITY;
    }
    if (mx > floor) {
      float v[U * E];  // (unpacked anew, not held in registers)
      uint32_t some = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        asm volatile("" : "+r"(now[u].x), "+r"(now[u].y), "+r"(now[u].z), "+r"(now[u].w));
        LpVec<T>::get(now[u], v + u * E);
      }
#pragma unroll
      for (int i = 0; i < U * E; ++i) some |= v[i] > floor ? 1u << i : 0u;
#pragma unroll 1
      for (; some; some &= some - 1) {
        const int k = __ffs(some) - 1;
        keep(ld_f(here + k / E * (kLpThreads * E) + k % E), head + (i0 + k / E * kLpThreads + tid) * E + k % E);
      }
    }
    // ids rise with the iterations: what only equals the floor comes behind those that made it
    if (opened) floor = low;
    if (it >= next_cut && i0 + 3 * kLpThreads * U < v1) {
      next_cut = 4 * it + 3;
      __syncthreads();
      cut(head + min(v1, i0 + kLpThreads * U) * E);
      open = sh.best[n_top - 1] == 0;
      if (!open) floor = lp_key_value(sh.best[n_top - 1]);
    }
  }
  cp_async_wait<0>();
  // the ids behind the vectors
  if (rank == C - 1 && tail0 + tid < p.vocab) {
    const float v = ld_f(x + tail0 + tid);
    add(v);
    if (kTopIds && v > floor) keep(v, tail0 + tid);
  }
  RowSum a = {m, s2.x + s2.y, t2.x + t2.y};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    RowSum b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
    a = join(a, b);
  }
  if (lane == 0) sums.part[warp] = a;
  __syncthreads();
  if (kTopIds) cut(rank == C - 1 ? p.vocab : head + v1 * E);
  const uint64_t* best = sh.best;
  RowSum r;
  if (warp == 0) r = lp_join(sums.part, kLpWarps);
  if (C > 1) {
    // every part goes to the first CTA's shared memory
    cluster_started_wait();
    if (kTopIds && tid < n_top)
      st_peer_u64(map_peer(smem_u32(&sh.all[rank * n_top + tid]), 0), sh.best[tid]);
    if (tid == 0) {
      const uint32_t to = map_peer(smem_u32(&sums.sums[rank]), 0);
      st_peer_f32(to, r.m);
      st_peer_f32(to + 4, r.s);
      st_peer_f32(to + 8, r.t);
    }
    cluster_sync();
    if (rank != 0) return;
    if (kTopIds) {
      lp_select(sh.all, C * n_top, n_top, sh.keys, sh);
      best = sh.keys;
    }
    if (warp == 0) r = lp_join(sums.sums, C);
  }
  if (warp != 0) return;  // (up to 32 alternatives)
  const bool mass = r.m != -INFINITY;
  const float log_s = logf(r.s);
  // what has no probability; a NaN (never a candidate) or +inf leaves the row without any numbers
  const float none = r.m < INFINITY ? -INFINITY : NAN;
  if (tid == 0) {
    if (p.logp && p.tokens)
      p.logp[row] = tok >= p.vocab || !mass ? none : (x_tok - r.m) - log_s;
    if (p.entropy) p.entropy[row] = mass ? log_s - r.t / r.s : 0.f;
  }
  if (tid < n_top) {
    const uint64_t k = best[tid];
    const long long at = (long long)row * n_top + tid;
    p.top_ids[at] = k ? (int)~(uint32_t)k : -1;
    p.top_logp[at] = k ? (lp_key_value(k) - r.m) - log_s : none;
  }
}

template <typename T>
constexpr int lp_smem_size(bool top) {
  return lp_lists_size(top) + LpVec<T>::kStages * LpVec<T>::kAtOnce * kLpThreads * 16;
}
static_assert(DFLASH_F32 == 0 && DFLASH_BF16 == 1, "an index of smem_done");

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_token_logprobs(int32_t rows, int32_t vocab, int32_t dtype, const void* logits,
                                    int64_t row_stride, const int32_t* tokens, int32_t top,
                                    float* logp, float* entropy, int32_t* top_ids, float* top_logp,
                                    dflash_stream_t stream) {
  if (rows < 1 || rows >= (1 << 27) || vocab < 1 || vocab >= (1 << 30) ||
      (dtype != DFLASH_F32 && dtype != DFLASH_BF16) || !logits || row_stride < vocab ||
      row_stride >= ((int64_t)1 << 40) || top < 0 || top > kLpTop || (logp && !tokens) ||
      (top > 0 && (!top_ids || !top_logp)) || (!logp && !entropy && top == 0) ||
      !kvq_aligned(logits, dtype == DFLASH_F32 ? 4 : 2) || !kvq_aligned(logp, 4) ||
      !kvq_aligned(entropy, 4) || !kvq_aligned(top_logp, 4) || !kvq_ints_aligned({tokens, top_ids}))
    return DFLASH_E_INVALID_ARG;
  // (rows that would lie past any memory: their addresses would not fit 64 bits either)
  if (rows - 1 >= ((int64_t)1 << 48) / row_stride) return DFLASH_E_INVALID_ARG;
  // What is written must be nothing that other CTAs still read, nor another output.
  const int64_t words = 4 * (int64_t)rows;
  const MemRange out[] = {{logp, words}, {entropy, words}, {top_ids, words * top}, {top_logp, words * top}};
  const MemRange in[] = {{logits, ((rows - 1) * row_stride + vocab) * (dtype == DFLASH_F32 ? 4 : 2)},
                         {tokens, words}};
  if (!ranges_apart(out, 4, in, 2)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {logits, tokens, logp, entropy, top_ids, top_logp};
  DF_TRY(kvq_ptrs_ok(ptrs, 6));
  LogpK p;
  p.logits = logits;
  p.stride = row_stride;
  p.tokens = tokens;
  p.logp = logp;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logp = top_logp;
  p.vocab = vocab;
  p.top = top;
  // A row to several CTAs while there are no more than two an SM, and each has more than an
  // iteration: 16 rows of 151,936 with 5 alternatives take 9.1 us by 8 CTAs each, 10.9 by four and 19 by
  // one; 100 rows with 20 take 24.5 by two and 30 by one (and 19 by four: the rule is not the best there;
  // without alternatives two and four are equal, and 152 rows take 16.6 and 20.5).  Beyond that it gains
  // little (256 rows: 39 us by two, 37 by one, without alternatives 27 and 30) and soon costs, since every
  // CTA makes a selection of its own (512 rows: 62 by one or two, 77 by four).
  int C = 1;
  while (C < kLpCluster && (int64_t)rows * C * 2 <= 2 * kvq_sms() && vocab > C * kLpStep) C *= 2;
  const auto kernel = dtype == DFLASH_F32
                          ? (top ? token_logprobs_kernel<float, true> : token_logprobs_kernel<float, false>)
                          : (top ? token_logprobs_kernel<bf16, true> : token_logprobs_kernel<bf16, false>);
  static std::atomic<bool> smem_done[4][kMaxDevices];
  const int lp_smem_bytes = dtype == DFLASH_F32 ? lp_smem_size<float>(top > 0) : lp_smem_size<bf16>(top > 0);
  if (ensure_smem_attr(smem_done[2 * dtype + (top > 0)], kernel, lp_smem_bytes) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (launch_k_cluster(true, dim3(C, 1, 1), kernel, dim3((unsigned)(rows * C)), dim3(kLpThreads),
                       lp_smem_bytes, (cudaStream_t)stream, p, C) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
