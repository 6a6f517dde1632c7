// Attention over the 8-bit KV cache and the accumulation of its weights
// (dflash_kvq_attention, dflash_kvq_score).
//
// For a query row q that sees the slots S of a sequence,
//   s_k = q . K_k / sqrt(128),  out = sum_k exp(s_k - lse) V_k,
//   lse = log sum_k exp(s_k),   score_k += exp(s_k - lse),
// with K_k, V_k the cache's values (code times power of two).
#include <cfloat>
#include <cmath>

#include "kvq.cuh"

namespace dflash {

struct KvqAttnK {
  KvqK c;
  const int32_t *seq_ids, *kv_lens, *q_lens;
  const uint64_t* anc;
  int anc_words, mask;
  int batch, block, H, G;
  const bf16* q;
  long long q_stride;
  bf16* out;
  float* lse;            // attention: out (may be null); score: in
  const float* score_in;
  float* score_out;
  float decay;
};

constexpr float kScaleLog2 = 0.12751743f;  // log2(e) / sqrt(128)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Entry b: sequence, slots n, rows r, and the first slot the cache cannot hold
// or the sequence does not have (key_end); false: skip it.
__device__ __forceinline__ bool kvq_entry(const KvqAttnK& p, int b, int& seq, int& n, int& r,
                                          int& key_end) {
  seq = kvq_seq(p.c, p.seq_ids, b);
  n = p.kv_lens[b];
  r = p.q_lens ? p.q_lens[b] : p.block;
  if (seq < 0) return false;
  if (n < 0 || r < 0 || r > p.block) {
    set_dev_status(p.c.status, kDevCheck);
    return false;
  }
  key_end = min(n, p.c.pps * kPageSlots);
  if (key_end < n) set_dev_status(p.c.status, kDevCapacity);
  return true;
}

// does row j of a sequence (n slots, r rows) see slot k < n?
__device__ __forceinline__ bool kvq_sees(const KvqAttnK& p, int k, int n, int r, int j,
                                         const uint64_t* anc_row) {
  const int i = k - (n - r);
  if (p.mask == DFLASH_MASK_NONE || i < 0) return true;
  if (p.mask == DFLASH_MASK_CAUSAL) return i <= j;
  return (i >> 6) < p.anc_words && ((anc_row[i >> 6] >> (i & 63)) & 1ull);
}

// four codes of a lane as floats, without the exponent
__device__ __forceinline__ float4 decode4(uint32_t w) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 load_q4(const bf16* q) {
  const uint2 w = *reinterpret_cast<const uint2*>(q);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  float d = a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
  return d;
}

// one warp per (row, query head), slots in order, lane l holding dims 4l..4l+3
__global__ void __launch_bounds__(128) kvq_attn_kernel(const KvqAttnK p) {
  pdl_trigger();
  pdl_wait();
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int h = (int)(w % p.H);
  const long long row = w / p.H;
  const int b = (int)(row / p.block), j = (int)(row % p.block);
  if (b >= p.batch) return;
  int seq, n, r, key_end;
  if (!kvq_entry(p, b, seq, n, r, key_end) || j >= r) return;
  const int kvh = h / p.G;
  const uint64_t* anc = p.mask == DFLASH_MASK_TREE ? p.anc + row * p.anc_words : nullptr;
  const float4 q = load_q4(p.q + row * p.q_stride + h * kKvqHd + lane * 4);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < key_end; k0 += kPageSlots) {
    const int page = kvq_page(p.c, seq, k0 / kPageSlots);
    if (page < 0) {
      set_dev_status(p.c.status, kDevCapacity);
      continue;
    }
    const int64_t ph = kvq_ph(p.c, page, kvh);
    for (int i = 0; i < min(kPageSlots, key_end - k0); ++i) {
      if (!kvq_sees(p, k0 + i, n, r, j, anc)) continue;
      const int64_t at = ph * kKvqPageBytes + i * kKvqHd + lane * 4;
      const int64_t sub = ph * kKvqSubs + i / kKvqSub;
      const float4 k = decode4(*reinterpret_cast<const uint32_t*>(p.c.c8[0] + at));
      const float s = dot4(q, k) * (pow2i(p.c.ex[0][sub]) * kScaleLog2);
      const float mn = fmaxf(m, s);
      const float corr = exp2f(m - mn), pk = exp2f(s - mn);
      const float4 v = decode4(*reinterpret_cast<const uint32_t*>(p.c.c8[1] + at));
      const float pv = pk * pow2i(p.c.ex[1][sub]);
      l = l * corr + pk;
      o.x = o.x * corr + pv * v.x;
      o.y = o.y * corr + pv * v.y;
      o.z = o.z * corr + pv * v.z;
      o.w = o.w * corr + pv * v.w;
      m = mn;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  const __nv_bfloat162 c = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 pk;
  pk.x = *reinterpret_cast<const uint32_t*>(&a);
  pk.y = *reinterpret_cast<const uint32_t*>(&c);
  *reinterpret_cast<uint2*>(p.out + (row * p.H + h) * kKvqHd + lane * 4) = pk;
  if (p.lse && lane == 0)
    p.lse[row * p.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// one warp per (sequence, KV head, slot): the rows in order
__global__ void __launch_bounds__(128) kvq_score_kernel(const KvqAttnK p) {
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.x * 4 + (threadIdx.x >> 5), kvh = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31;
  int seq, n, r, key_end;
  if (!kvq_entry(p, b, seq, n, r, key_end)) return;
  for (int s0 = k; s0 < key_end; s0 += gridDim.x * 4) {
    const int page = kvq_page(p.c, seq, s0 / kPageSlots);
    float w = 0.f;
    if (page < 0) {
      set_dev_status(p.c.status, kDevCapacity);
    } else {
      const int64_t ph = kvq_ph(p.c, page, kvh);
      const int i = s0 % kPageSlots;
      const float4 kk =
          decode4(*reinterpret_cast<const uint32_t*>(p.c.c8[0] + ph * kKvqPageBytes + i * kKvqHd +
                                                     lane * 4));
      const float sc = pow2i(p.c.ex[0][ph * kKvqSubs + i / kKvqSub]) * kScaleLog2;
      for (int j = 0; j < r; ++j) {
        const long long row = (long long)b * p.block + j;
        if (!kvq_sees(p, s0, n, r, j, p.mask == DFLASH_MASK_TREE ? p.anc + row * p.anc_words : nullptr))
          continue;
        for (int g = 0; g < p.G; ++g) {
          const int h = kvh * p.G + g;
          const float lse = p.lse[row * p.H + h];
          if (lse == -INFINITY) continue;
          const float4 q = load_q4(p.q + row * p.q_stride + h * kKvqHd + lane * 4);
          w += exp2f(dot4(q, kk) * sc - lse * kLog2e);
        }
      }
    }
    if (lane == 0) {
      const int64_t at = ((int64_t)seq * p.c.Hkv + kvh) * ((int64_t)p.c.pps * kPageSlots) + s0;
      p.score_out[at] = (p.score_in ? p.decay * p.score_in[at] : 0.f) + w;
    }
  }
}

static bool kvq_attn_shape_ok(int batch, int H, int Hkv, int block, int max_keys) {
  return batch >= 1 && batch <= 65535 && H >= 1 && Hkv >= 1 && Hkv <= 65535 && H % Hkv == 0 &&
         H / Hkv <= 64 && block >= 1 && max_keys >= 1 && max_keys <= (1 << 29) &&
         (int64_t)batch * block < ((int64_t)1 << 31) &&
         (int64_t)batch * block * H < ((int64_t)1 << 31);
}

// what the attention and the score take alike
static dflash_status kvq_attn_args(KvqAttnK* p, const dflash_kvq_cache* cache, int batch, int H,
                                   int block, int mask, const int32_t* seq_ids,
                                   const int32_t* kv_lens, const int32_t* q_lens,
                                   const uint64_t* anc, int anc_words, int max_keys, const void* q,
                                   int64_t q_row_stride) {
  if (!kvq_cache_ok(cache) || !kvq_attn_shape_ok(batch, H, cache->n_kv_heads, block, max_keys) ||
      mask < DFLASH_MASK_NONE || mask > DFLASH_MASK_TREE || !kv_lens || !q || !kvq_aligned(q, 16) ||
      q_row_stride < (int64_t)H * kKvqHd || q_row_stride % 8 != 0 ||
      q_row_stride >= ((int64_t)1 << 31))
    return DFLASH_E_INVALID_ARG;
  if (mask == DFLASH_MASK_TREE && (!anc || !kvq_aligned(anc, 8) || anc_words < 1))
    return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {seq_ids, kv_lens, q_lens, mask == DFLASH_MASK_TREE ? anc : nullptr, q};
  DF_TRY(kvq_cache_ptrs_ok(cache));
  DF_TRY(kvq_ptrs_ok(ptrs, 5));
  memset(p, 0, sizeof(*p));
  p->c = kvq_device_view(cache);
  p->seq_ids = seq_ids;
  p->kv_lens = kv_lens;
  p->q_lens = q_lens;
  p->anc = anc;
  p->anc_words = anc_words;
  p->mask = mask;
  p->batch = batch;
  p->block = block;
  p->H = H;
  p->G = H / cache->n_kv_heads;
  p->q = static_cast<const bf16*>(q);
  p->q_stride = q_row_stride;
  return DFLASH_OK;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

int64_t dflash_kvq_attention_workspace(int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                       int32_t block, int32_t max_keys) {
  if (!kvq_attn_shape_ok(batch, n_heads, n_kv_heads, block, max_keys)) return -1;
  return 0;
}

dflash_status dflash_kvq_attention(const dflash_kvq_cache* cache, int32_t batch, int32_t n_heads,
                                   int32_t block, int32_t mask, const int32_t* seq_ids,
                                   const int32_t* kv_lens, const int32_t* q_lens,
                                   const uint64_t* anc, int32_t anc_words, int32_t max_keys,
                                   const void* q, int64_t q_row_stride, void* out, float* lse,
                                   void* workspace, int64_t workspace_bytes,
                                   dflash_stream_t stream) {
  if (!out || !kvq_aligned(out, 16) || !kvq_aligned(lse, 4) || !kvq_aligned(workspace, 16) ||
      workspace_bytes < 0)
    return DFLASH_E_INVALID_ARG;
  KvqAttnK p;
  DF_TRY(kvq_attn_args(&p, cache, batch, n_heads, block, mask, seq_ids, kv_lens, q_lens, anc,
                       anc_words, max_keys, q, q_row_stride));
  const void* const ptrs[] = {out, lse, workspace};
  DF_TRY(kvq_ptrs_ok(ptrs, 3));
  p.out = static_cast<bf16*>(out);
  p.lse = lse;
  const int64_t warps = (int64_t)batch * block * n_heads;
  if (launch_k(true, kvq_attn_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0,
               (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_kvq_score(const dflash_kvq_cache* cache, int32_t batch, int32_t n_heads,
                               int32_t block, int32_t mask, const int32_t* seq_ids,
                               const int32_t* kv_lens, const int32_t* q_lens, const uint64_t* anc,
                               int32_t anc_words, int32_t max_keys, const void* q,
                               int64_t q_row_stride, const float* lse, float decay,
                               const float* score_in, float* score_out, dflash_stream_t stream) {
  if (!lse || !score_out || !kvq_aligned(lse, 4) || !kvq_aligned(score_in, 4) ||
      !kvq_aligned(score_out, 4))
    return DFLASH_E_INVALID_ARG;
  KvqAttnK p;
  DF_TRY(kvq_attn_args(&p, cache, batch, n_heads, block, mask, seq_ids, kv_lens, q_lens, anc,
                       anc_words, max_keys, q, q_row_stride));
  const void* const ptrs[] = {lse, score_in, score_out};
  DF_TRY(kvq_ptrs_ok(ptrs, 3));
  p.lse = const_cast<float*>(lse);
  p.decay = decay;
  p.score_in = score_in;
  p.score_out = score_out;
  const dim3 grid((unsigned)((max_keys + 3) / 4), cache->n_kv_heads, batch);
  if (launch_k(true, kvq_score_kernel, grid, dim3(128), 0, (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
