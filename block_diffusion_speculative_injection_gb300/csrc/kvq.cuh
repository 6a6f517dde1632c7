// Shared pieces of the 8-bit KV cache operators (dflash_kvq_*): the device view
// of a cache, its addressing, the e4m3 block format and the host checks.
#pragma once

#include <cuda_fp8.h>

#include <initializer_list>

#include "internal.cuh"

namespace dflash {

constexpr int kKvqHd = 128;                          // head_dim
constexpr int kKvqSub = 16;                          // slots that share an exponent
constexpr int kKvqSubs = kPageSlots / kKvqSub;       // exponents per page and head
constexpr int kKvqExpMin = -40, kKvqExpMax = 40;     // range of an exponent
constexpr int64_t kKvqPageBytes = (int64_t)kPageSlots * kKvqHd;  // codes of a page, one head

struct KvqK {
  uint8_t* c8[2];   // K, V codes
  int8_t* ex[2];    // K, V exponents
  const int32_t* tab;
  int32_t* status;
  int n_pages, Hkv, n_seqs, pps;
};

// sequence of batch entry b, or -1 (bad id: status set)
__device__ __forceinline__ int kvq_seq(const KvqK& c, const int32_t* ids, int b) {
  const int q = ids ? ids[b] : b;
  if (q < 0 || q >= c.n_seqs) {
    set_dev_status(c.status, kDevCheck);
    return -1;
  }
  return q;
}
// Page of table entry i of a sequence, or -1 (past the table, unmapped or out of the
// pool): in two steps, so that a loop can read an entry some iterations before
// anything waits for it.
__device__ __forceinline__ int kvq_page_load(const KvqK& c, int seq, int i) {
  return i >= 0 && i < c.pps ? c.tab[(int64_t)seq * c.pps + i] : -1;
}
__device__ __forceinline__ int kvq_page_check(const KvqK& c, int raw) {
  return raw >= 0 && raw < c.n_pages ? raw : -1;
}
__device__ __forceinline__ int kvq_page(const KvqK& c, int seq, int i) {
  return kvq_page_check(c, kvq_page_load(c, seq, i));
}
// (page, head) index: times kKvqPageBytes the codes, times kKvqSubs the exponents
__device__ __forceinline__ int64_t kvq_ph(const KvqK& c, int page, int head) {
  return (int64_t)page * c.Hkv + head;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// exponent of a block whose largest finite magnitude is a: the smallest e with
// a <= 448 * 2^e = 1.75 * 2^(e + 8)
__device__ __forceinline__ int kvq_exponent(float a) {
  const int bits = __float_as_int(a);
  const int e = (bits >> 23) - 127 - ((bits & 0x7fffff) > 0x600000 ? 7 : 8);
  return min(kKvqExpMax, max(kKvqExpMin, e));
}

// eight codes <-> eight floats (code values, without the exponent)
__device__ __forceinline__ void kvq_decode8(uint2 c, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? c.x : c.y;
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint2 kvq_encode8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// eight bf16 <-> eight floats
__device__ __forceinline__ void bf16x8_to_f(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 f_to_bf16x8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// host checks (kvq.cu)
// ---------------------------------------------------------------------------
// every field of the cache, without a CUDA call
bool kvq_cache_ok(const dflash_kvq_cache* c);
// device memory of the current device, or NULL where `optional`
dflash_status kvq_ptrs_ok(const void* const* ptrs, int n);
dflash_status kvq_cache_ptrs_ok(const dflash_kvq_cache* c);
KvqK kvq_device_view(const dflash_kvq_cache* c);
int kvq_sms();  // SM count of the current device (cached per device)
inline bool kvq_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool kvq_ints_aligned(std::initializer_list<const int32_t*> ptrs) {
  for (const int32_t* p : ptrs)
    if (!kvq_aligned(p, 4)) return false;
  return true;
}

// `bytes` bytes from p on (p NULL: none)
struct MemRange {
  const void* p;
  int64_t bytes;
};
// whether nothing of out[0 .. n_out) overlaps another of them or an input
bool ranges_apart(const MemRange* out, int n_out, const MemRange* in, int n_in);

}  // namespace dflash
