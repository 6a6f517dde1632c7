// Attention of a packed batch of prompts over themselves (dflash_prompt_attention).
//
// For row i of a prompt of n rows, head h and its KV head,
//   s_k = q_i . k_k / sqrt(128),  lse = log sum_k exp(s_k),  out = sum_k exp(s_k - lse) v_k
// over the keys k <= i (causal) or k < n.
#include <cmath>

#include "kvq.cuh"
#include "packed.cuh"

namespace dflash {

constexpr int kPromptHd = 128;

struct PromptK {
  const int32_t* offsets;
  const bf16 *q, *k, *v;
  long long qs, ks, vs;  // elements between rows
  bf16* out;
  float* lse;
  int32_t* status;
  int batch, n_rows, H, Hkv, causal;
};

// One warp for a row and head, four dims a lane.
__global__ void __launch_bounds__(128) prompt_attn_kernel(const PromptK p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  packed_check(p.offsets, p.batch, p.n_rows, (long long)blockIdx.x * 128 + threadIdx.x,
               (long long)gridDim.x * 128, p.status);
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(w % p.H);
  const long long u = w / p.H;
  const int b = packed_find(p.offsets, p.batch, 1, 0, u);
  int first = 0, n = 0;
  if (b < 0 || !packed_rows(p.offsets, b, p.n_rows, first, n)) return;
  const long long i = u - first;
  if (i >= n) return;
  const int kvh = h / (p.H / p.Hkv);
  const int end = p.causal ? (int)i + 1 : n;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int e = 0; e < 4; ++e) q[e] = ld_f(p.q + u * p.qs + h * kPromptHd + 4 * lane + e);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    const bf16* k = p.k + (first + j) * p.ks + kvh * kPromptHd + 4 * lane;
    const bf16* v = p.v + (first + j) * p.vs + kvh * kPromptHd + 4 * lane;
    float s = 0.f;
    for (int e = 0; e < 4; ++e) s += q[e] * ld_f(k + e);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= 0.08838834764831845f;
    const float m2 = fmaxf(m, s), base = m2 == -INFINITY ? 0.f : m2;
    const float f = expf(m - base), e1 = expf(s - base);
    l = l * f + e1;
    for (int e = 0; e < 4; ++e) o[e] = o[e] * f + e1 * ld_f(v + e);
    m = m2;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int e = 0; e < 4; ++e) st_f(p.out + (u * p.H + h) * kPromptHd + 4 * lane + e, o[e] * inv);
  if (p.lse && lane == 0) p.lse[u * p.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

static bool prompt_stride_ok(int64_t stride, int heads) {
  return stride >= (int64_t)heads * kPromptHd && stride % 8 == 0 && stride < ((int64_t)1 << 31);
}
// bytes [p, p + n)
static bool prompt_overlap(const void* p, int64_t n, const void* q, int64_t m) {
  if (!p || !q) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  return x < y ? y - x < (uint64_t)n : x - y < (uint64_t)m;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_prompt_attention(int32_t batch, int32_t n_rows, int32_t n_heads,
                                      int32_t n_kv_heads, int32_t causal, const int32_t* offsets,
                                      const void* q, int64_t q_row_stride, const void* k,
                                      int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                      void* out, float* lse, int32_t* status,
                                      dflash_stream_t stream) {
  if (batch < 1 || batch >= (1 << 26) || n_rows < 1 || n_rows >= (1 << 30) || n_heads < 1 ||
      n_heads > 65535 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 64 ||
      (causal != 0 && causal != 1) || !offsets || !q || !k || !v || !out || !status ||
      !prompt_stride_ok(q_row_stride, n_heads) || !prompt_stride_ok(k_row_stride, n_kv_heads) ||
      !prompt_stride_ok(v_row_stride, n_kv_heads) || !kvq_aligned(q, 16) || !kvq_aligned(k, 16) ||
      !kvq_aligned(v, 16) || !kvq_aligned(out, 16) || !kvq_aligned(lse, 4) ||
      !kvq_ints_aligned({offsets, status}))
    return DFLASH_E_INVALID_ARG;
  // What is written must be nothing that other CTAs still read, nor the other output.
  struct Range {
    const void* p;
    int64_t n;
  };
  auto bytes = [&](int64_t stride, int heads) {
    return ((n_rows - 1) * stride + (int64_t)heads * kPromptHd) * 2;
  };
  const Range in[] = {{q, bytes(q_row_stride, n_heads)},
                      {k, bytes(k_row_stride, n_kv_heads)},
                      {v, bytes(v_row_stride, n_kv_heads)},
                      {offsets, ((int64_t)batch + 1) * 4},
                      {status, 4}};
  const Range o[] = {{out, (int64_t)n_rows * n_heads * kPromptHd * 2},
                     {lse, (int64_t)n_rows * n_heads * 4}};
  for (const Range& w : o)
    for (const Range& r : in)
      if (prompt_overlap(w.p, w.n, r.p, r.n)) return DFLASH_E_INVALID_ARG;
  if (prompt_overlap(o[0].p, o[0].n, o[1].p, o[1].n)) return DFLASH_E_INVALID_ARG;
  const void* const ptrs[] = {offsets, q, k, v, out, lse, status};
  DF_TRY(kvq_ptrs_ok(ptrs, 7));
  PromptK p;
  p.offsets = offsets;
  p.q = static_cast<const bf16*>(q);
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.qs = q_row_stride;
  p.ks = k_row_stride;
  p.vs = v_row_stride;
  p.out = static_cast<bf16*>(out);
  p.lse = lse;
  p.status = status;
  p.batch = batch;
  p.n_rows = n_rows;
  p.H = n_heads;
  p.Hkv = n_kv_heads;
  p.causal = causal;
  const int64_t warps = (int64_t)n_rows * n_heads;
  if (warps >= ((int64_t)1 << 32)) return DFLASH_E_INVALID_ARG;
  if (launch_k(true, prompt_attn_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0,
               (cudaStream_t)stream, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
