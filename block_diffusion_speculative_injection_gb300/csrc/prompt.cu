// Attention of a packed batch of prompts over themselves (dflash_prompt_attention).
//
// For row i of a prompt of n rows, head h and its KV head,
//   s_k = q_i . k_k / sqrt(128),  lse = log sum_k exp(s_k),  out = sum_k exp(s_k - lse) v_k
// over the keys k <= i (causal) or k < n.
#include <cmath>

#include "attn_util.cuh"
#include "kvq.cuh"
#include "packed.cuh"

namespace dflash {

constexpr int kPromptHd = 128;

struct PromptK {
  const int32_t* offsets;
  const bf16* v;
  long long vs;  // elements between V's rows
  bf16* out;
  float* lse;
  int32_t* status;
  int batch, n_rows, H, Hkv, G, causal;
  int pos, g_inv;  // positions of a tile's 128 rows; row / G = row * g_inv >> 16 (row < 128)
  int tiles;       // query tiles of a CTA: 1 or 2
  int units;       // of tiles * pos positions, over all sequences
};

struct PromptMaps {
  CUtensorMap q, k, v;
};

// ---------------------------------------------------------------------------
// One CTA: two tiles of 128 query rows (128 / G positions x the G query heads of a KV head)
// against the prompt's keys, 128 a step.  While the tensor cores work on one tile's products, a
// warpgroup of softmax threads, one a row, works on the other's scores:
//
//   S = Q K^T (tensor memory, fp32); each row's maximum m; P = exp2((S - m) log2(e) / sqrt(128))
//   to bf16, over S in tensor memory; O += P V with A = P from there.
//
// m is the largest score when it was taken and is raised only when a tile's largest exceeds it
// by more than 2^8 in the weights: then the row of O in tensor memory and the sum l are rescaled.  Any
// consistent m gives the same O / l.  A weight is rounded to bf16 (half a step: 2^-9) because V is
// bf16 and both operands of a product have one type; the sum l takes it unrounded.
//
// Keys behind a row's own position, or the prompt's end, have weight 0, which keeps finite values
// of V out, not NaN or infinities (0 * NaN): in the tiles that not every row of the CTA sees
// whole, a warp replaces those by zeros in shared memory.  If there were any, the rows that do see
// them add them to their results at the end.
//
// Shared memory (1024-aligned, rows of 128 B, 128-byte swizzle): Q 2 x 32 KB, a ring of five
// stages of 32 KB for K and V in the order K0 K1 V0 K2 V1 ..  Tensor memory: S and O of both tiles, all
// 512 columns.
// Warps 0-3, 4-7: softmax of tile 0 and 1.  Warp 8: TMA.  Warps 9, 10: the tiles' MMAs, O(j) and
// then S(j + 1), so that S(j + 1) follows the last read of P(j), which it overwrites.  Warp 11: V.
// ---------------------------------------------------------------------------
constexpr int kPT = 128;                       // rows of a query tile, keys of a step
constexpr uint32_t kPBox = kPT * 128;          // 128 rows of 64 dims
constexpr uint32_t kPStage = 2 * kPBox;        // a K, V or Q tile
constexpr int kPStages = 5;
constexpr uint32_t kPOffKV = 2 * kPStage;
constexpr uint32_t kPOffBar = kPOffKV + kPStages * kPStage;
constexpr int kPromptSmem = (int)kPOffBar + 256 + 1024;  // barriers, alignment slack
static_assert(kPromptSmem <= 227 * 1024, "shared memory of a CTA");
constexpr int kPromptThreads = 384;
constexpr int kPromptRegs = 168, kPSoftRegs = 216, kPIssueRegs = 72;
static_assert(kPromptThreads * kPromptRegs <= 65536, "registers of an SM");
static_assert(2 * kPSoftRegs + kPIssueRegs <= 3 * kPromptRegs, "what one takes the others leave");
constexpr uint32_t kPTmemS = 0, kPTmemO = 2 * kPT;
constexpr float kPScaleLog2 = 0.12751743f;  // log2(e) / sqrt(128)
constexpr float kPLn2 = 0.6931471805599453f;
// growth of a maximum that is not yet rescaled: weights up to 2^8
constexpr float kPLazy = 8.f / kPScaleLog2;
// Scores from here on are taken relative to the maximum before they are scaled: the rounding of
// the product with log2(e) / sqrt(128) would be a factor in the weights, 2^-4 binades here.
constexpr float kPFar = 1048576.f / kPScaleLog2;

struct PromptItem {
  int first, n;     // the prompt's rows
  int p0a, p0b;     // first position of each query tile
  int steps_a, steps_b;  // key tiles each sees (0: no row)
  int clean;        // first key tile that not every row sees whole
  int kvh;
};

__device__ __forceinline__ bool prompt_item(const PromptK& p, PromptItem& it) {
  it.kvh = blockIdx.x % p.Hkv;
  // the last positions first: their CTAs take longest
  const long long u = p.units - 1 - (long long)(blockIdx.x / p.Hkv);
  const int per = p.tiles * p.pos;
  const int b = packed_find(p.offsets, p.batch, per, 1, u);
  if (b < 0 || !packed_rows(p.offsets, b, p.n_rows, it.first, it.n)) return false;
  const long long at = (u - packed_base(p.offsets, b, per, 1)) * per;
  if (at >= it.n) return false;
  const int mask_from = p.causal ? (int)at + 1 : it.n;
  it.p0a = (int)at;
  it.p0b = (int)at + p.pos;
  auto steps = [&](int p0) {
    return ((p.causal ? min(it.n, p0 + p.pos) : it.n) + kPT - 1) / kPT;
  };
  it.steps_a = steps(it.p0a);
  it.steps_b = p.tiles > 1 && it.p0b < it.n ? steps(it.p0b) : 0;
  it.clean = mask_from / kPT;
  return true;
}
// (at most 2 * 128 positions a CTA: their own keys lie in three tiles at most)
constexpr int kPClean = 3;

// which of the loads in ring order is K or V of step j of n
__device__ __forceinline__ int prompt_load_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int prompt_load_v(int j, int n) { return min(2 * j + 2, 2 * n - 1); }

__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptMaps maps, const PromptK p) {
  pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  packed_check(p.offsets, p.batch, p.n_rows, (long long)blockIdx.x * kPromptThreads + threadIdx.x,
               (long long)gridDim.x * kPromptThreads, p.status);
  PromptItem it;
  if (!prompt_item(p, it)) {  // the whole CTA
    pdl_trigger();
    return;
  }
  int32_t* const status = p.status;
  const int n_steps = max(it.steps_a, it.steps_b);

  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + kPOffBar);
  uint64_t* const q_full = bars;        // [2]
  uint64_t* const s_full = bars + 2;    // [2]
  uint64_t* const p_full = bars + 4;    // [2][2] halves of P
  uint64_t* const o_full = bars + 8;    // [2]
  uint64_t* const drained = bars + 10;  // [2]
  uint64_t* const clean = bars + 12;    // [kPClean] tiles it.clean ..
  uint64_t* const raw_full = clean + kPClean;  // [kPClean] the same before they are cleaned
  uint64_t* const kv_full = raw_full + kPClean;  // [stages]
  uint64_t* const kv_empty = kv_full + kPStages;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(kv_empty + kPStages);
  volatile int* const v_bad = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((12 + 2 * kPClean + 2 * kPStages) * 8 + 8 <= 256, "barriers fit");

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[2 * x], 4);
      mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&drained[x], 1);
    }
    for (int i = 0; i < kPClean; ++i) {
      mbar_init(&clean[i], 1);
      mbar_init(&raw_full[i], 1);
    }
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], it.steps_b > 0 ? 2 : 1);
    }
    *v_bad = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tslot;

  if (warp >= 8) {
    regs_dec<kPIssueRegs>();
    const bool leader = elect_one();
    if (warp == 8) {
      // ---- producer
      if (leader) {
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
      }
      int issued = 0, v_issued = 0;
      auto load = [&](bool is_v, int j) -> bool {
        const int st = issued % kPStages, round = issued / kPStages;
        if (round > 0 && !__all_sync(0xffffffffu, warp_wait(&kv_empty[st], (round - 1) & 1, status)))
          return false;
        if (leader) {
          uint8_t* const dst = sm + kPOffKV + st * kPStage;
          const CUtensorMap* const map = is_v ? &maps.v : &maps.k;
          // The tiles of V that are cleaned have barriers of their own: those warps do not
          // follow the ring, whose barriers have one bit for the round.
          uint64_t* full = &kv_full[st];
          if (is_v && j >= it.clean) {
            mbar_arrive(full);
            full = &raw_full[j - it.clean];
          }
          mbar_arrive_expect_tx(full, kPStage);
          tma_load_3d(dst, map, 0, it.kvh, it.first + j * kPT, full);
          tma_load_3d(dst + kPBox, map, 64, it.kvh, it.first + j * kPT, full);
        }
        __syncwarp();
        ++issued;
        if (is_v) v_issued = j + 1;
        return true;
      };
      auto load_q = [&](int x, int p0, int steps) {
        if (leader && steps > 0) {
          uint8_t* const dst = sm + x * kPStage;
          mbar_arrive_expect_tx(&q_full[x], (uint32_t)(2 * 128 * p.G * p.pos));
          tma_load_3d(dst, &maps.q, 0, it.kvh * p.G, it.first + p0, &q_full[x]);
          tma_load_3d(dst + kPBox, &maps.q, 64, it.kvh * p.G, it.first + p0, &q_full[x]);
        }
        __syncwarp();
      };
      load_q(0, it.p0a, it.steps_a);
      load(false, 0);
      load_q(1, it.p0b, it.steps_b);
#pragma unroll 1
      for (int j = 0; j < n_steps; ++j) {
        if (j + 1 < n_steps && !load(false, j + 1)) break;
        if (!load(true, j)) break;
      }
      // every issued copy has landed before this warp leaves
      warp_wait(&q_full[0], 0, status);
      if (it.steps_b > 0) warp_wait(&q_full[1], 0, status);
#pragma unroll 1
      for (int i = max(0, issued - kPStages); i < issued; ++i)
        warp_wait(&kv_full[i % kPStages], (i / kPStages) & 1, status);
#pragma unroll 1
      for (int j = it.clean; j < v_issued; ++j) warp_wait(&raw_full[j - it.clean], 0, status);
      __syncwarp();
    } else if (warp <= 10) {
      // ---- MMA issuers, one for each query tile, so that one's waits pass beside the other's
      // products.  Whole warps wait, one lane issues: the descriptors stay in uniform registers.
      const int x = warp - 9, steps = x == 0 ? it.steps_a : it.steps_b;
      constexpr uint32_t id_s = idesc_bf16_f32(kPT, kPT);
      constexpr uint32_t id_o = idesc_bf16_f32(kPT, kPromptHd) | kIdescBMajorMN;
      const uint64_t q_desc = sw128_desc(smem_u32(sm + x * kPStage));
      const uint64_t k_desc = sw128_desc(smem_u32(sm + kPOffKV));
      const uint64_t v_desc = sw128_desc_mn(smem_u32(sm + kPOffKV), kPBox);
      const uint32_t t_s = tmem + kPTmemS + x * kPT, t_o = tmem + kPTmemO + x * kPromptHd;
      bool ok = true;
      auto wait_for = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, warp_wait(bar, parity, status));
        return ok;
      };
      auto wait_kv = [&](int at) { wait_for(&kv_full[at % kPStages], (at / kPStages) & 1); };
      auto scores = [&](int j) {  // and K is free when they are done
        const int st = prompt_load_k(j) % kPStages;
        tc_fence_after();
        if (leader) {
          const uint64_t kd = k_desc + st * (kPStage >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * kPBox + (kk & 3) * 32) >> 4;
            tc_mma_bf16(t_s, q_desc + off, kd + off, id_s, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[x]);
          tc_commit(&kv_empty[st]);
        }
        __syncwarp();
      };
      if (steps > 0) {
        wait_kv(0);
        if (wait_for(&q_full[x], 0)) scores(0);
      }
#pragma unroll 1
      for (int j = 0; ok && j < steps; ++j) {
        const int at = prompt_load_v(j, n_steps), st = at % kPStages;
        // the step's loads first (they are early), then only the softmax is waited for
        if (j + 1 < steps) wait_kv(prompt_load_k(j + 1));
        if (j >= it.clean)
          wait_for(&clean[j - it.clean], 0);
        else
          wait_kv(at);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait_for(&p_full[2 * x + half], j & 1)) break;
          tc_fence_after();
          if (leader) {
            const uint64_t vd = v_desc + st * (kPStage >> 4);
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              tc_mma_f16_ta(t_o, t_s + 8 * kk, vd + kk * (16 * 128 >> 4), id_o, j + kk > 0 ? 1u : 0u);
            if (half == 1) tc_commit(&kv_empty[st]);
            if (half == 1 && j + 1 == steps) tc_commit(&o_full[x]);
          }
          __syncwarp();
        }
        if (ok && j + 1 < steps) scores(j + 1);
      }
      // What this tile does not use is free as far as it is concerned, once it is loaded: an
      // arrival before that would count for the stage's load before.
#pragma unroll 1
      for (int i = 2 * steps; ok && steps > 0 && i < 2 * n_steps; ++i) {
        const int at = i & 1 ? prompt_load_v(i >> 1, n_steps) : prompt_load_k(i >> 1);
        wait_kv(at);
        if (ok && leader) mbar_arrive(&kv_empty[at % kPStages]);
        __syncwarp();
      }
      // nothing of this warp is in flight when it leaves
      if (leader) tc_commit(&drained[x]);
      __syncwarp();
      warp_wait(&drained[x], 0, status);
      __syncwarp();
    } else {
      // ---- V without NaN and infinities where not every row sees all keys
            bool bad = false;
#pragma unroll 1
      for (int j = it.clean; j < n_steps; ++j) {
        const int at = prompt_load_v(j, n_steps), st = at % kPStages;
        if (!__all_sync(0xffffffffu, warp_wait(&raw_full[j - it.clean], 0, status))) break;
        uint4* const tile = reinterpret_cast<uint4*>(sm + kPOffKV + st * kPStage);
#pragma unroll 4
        for (int i = lane; i < (int)(kPStage / 16); i += 32) {
          const uint4 v = tile[i];
          uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // a half whose exponent is all ones carries into its top bit
            const uint32_t b = ((w[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
            any |= b;
            w[e] &= ~((b - (b >> 15)) | b);
          }
          if (any) {
            tile[i] = make_uint4(w[0], w[1], w[2], w[3]);
            bad = true;
          }
        }
        if (bad) *v_bad = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&clean[j - it.clean]);
      }
      __syncwarp();
    }
  } else {
    regs_inc<kPSoftRegs>();
    // ---- softmax: this thread's row of tile x
    const int x = warp >> 2, row = threadIdx.x & 127;
    const int g_pos = row * p.g_inv >> 16;
    const int p0 = x == 0 ? it.p0a : it.p0b, pos = p0 + g_pos;
    const int n_mine = x == 0 ? it.steps_a : it.steps_b;
    const int limit = p.causal ? min(pos + 1, it.n) : it.n;  // its keys
    const int mask_from = p.causal ? p0 + 1 : it.n;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + kPTmemS + x * kPT, t_o = lanes + kPTmemO + x * kPromptHd;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n_mine; ++j) {
      if (!(ok = __all_sync(0xffffffffu, warp_wait(&s_full[x], j & 1, status)))) break;
      tc_fence_after();
      uint32_t s[kPT];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_nowait(t_s + 32 * c, s + 32 * c);
      tmem_wait_ld();
      if ((j + 1) * kPT > mask_from) {
        const int end = limit - j * kPT;
#pragma unroll
        for (int i = 0; i < kPT; ++i)
          if (i >= end) s[i] = __float_as_uint(-INFINITY);
      }
      float mx = -INFINITY, mx2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPT; i += 4) {
        mx = max3(mx, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        mx2 = max3(mx2, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
      }
      mx = fmaxf(mx, mx2);
      const bool grown = mx > m + kPLazy || (m == -INFINITY && mx > m);
      if (__any_sync(0xffffffffu, grown)) {
        const float alpha = grown ? ex2((m - mx) * kPScaleLog2) : 1.f;
        if (j > 0) {  // O holds the steps before: S(j) is complete, so they are
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32_nowait(t_o + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(t_o + 32 * c, o);
          }
        }
        if (grown) {
          l *= alpha;
          m = mx;
        }
      }
      float base = m == -INFINITY ? 0.f : -m * kPScaleLog2;
      if (__any_sync(0xffffffffu, fabsf(m) > kPFar && m != -INFINITY)) {
        if (m != -INFINITY) {
#pragma unroll
          for (int i = 0; i < kPT; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) - m);
          base = 0.f;
        }
      }
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int e = 64 * half + 2 * i;
          float2 z = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), kPScaleLog2,
                          base);
          z.x = ex2(z.x);
          z.y = ex2(z.y);
          sum[i & 1] = add2(sum[i & 1], z);
          const __nv_bfloat162 h = __floats2bfloat162_rn(z.x, z.y);
          pk[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tmem_st32(t_s + 32 * half, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
    }
    // ---- the rows' results
    if (n_mine > 0 && ok) ok = __all_sync(0xffffffffu, warp_wait(&o_full[x], 0, status));
    if (n_mine > 0 && ok) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int head0 = it.kvh * p.G;
      const bool live = g_pos < p.pos && pos < it.n;
      if (live && p.lse)
        p.lse[(long long)(it.first + pos) * p.H + head0 + row - g_pos * p.G] =
            l == 0.f ? -INFINITY : (m * kPScaleLog2 + log2f(l)) * kPLn2;
      const bool bad = *v_bad != 0;
      // through shared memory (this warp's rows of Q, which is used up), 16 bytes at chunk c ^ row
      uint8_t* const stage = sm + x * kPStage + (warp & 3) * (32 * 256);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32_nowait(t_o + 32 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
        if (bad && live) {
#pragma unroll 1
          for (int key = it.clean * kPT; key < limit; ++key) {
            const bf16* const v = p.v + (long long)(it.first + key) * p.vs + it.kvh * kPromptHd + 32 * c;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float f = ld_f(v + i);
              if (!(fabsf(f) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + f);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]),
                                                           __uint_as_float(o[8 * k + 2 * e + 1]));
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(stage + lane * 256 + (((4 * c + k) ^ (lane & 15)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4), chunk = lane & 15;
        const int rr = (warp & 3) * 32 + r, g = rr * p.g_inv >> 16;
        if (g < p.pos && p0 + g < it.n) {
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 256 + ((chunk ^ (r & 15)) << 4));
          *reinterpret_cast<uint4*>(p.out +
                                    ((long long)(it.first + p0 + g) * p.H + head0 + rr - g * p.G) *
                                        kPromptHd +
                                    8 * chunk) = v;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
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

// bf16 rows [n_rows] of `heads` heads, boxes of 64 dims, box_heads heads and box_rows rows
static bool prompt_map(CUtensorMap* m, const void* ptr, int heads, int n_rows, int64_t row_stride,
                       int box_heads, int box_rows) {
  const uint64_t dims[3] = {(uint64_t)kPromptHd, (uint64_t)heads, (uint64_t)n_rows};
  const uint64_t strides[2] = {kPromptHd * 2, (uint64_t)row_stride * 2};
  const uint32_t box[3] = {64u, (uint32_t)box_heads, (uint32_t)box_rows};
  return encode_tmap_bf16(m, ptr, 3, dims, strides, box);
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
  p.v = static_cast<const bf16*>(v);
  p.vs = v_row_stride;
  p.out = static_cast<bf16*>(out);
  p.lse = lse;
  p.status = status;
  p.batch = batch;
  p.n_rows = n_rows;
  p.H = n_heads;
  p.Hkv = n_kv_heads;
  p.G = n_heads / n_kv_heads;
  p.causal = causal;
  p.pos = kPT / p.G;
  p.g_inv = 65536 / p.G + 1;
  // two query tiles a CTA, but one where the CTAs would be fewer than the SMs
  p.tiles = packed_units(n_rows, batch, 2 * p.pos, 1) * n_kv_heads < kvq_sms() ? 1 : 2;
  const int64_t units = packed_units(n_rows, batch, p.tiles * p.pos, 1);
  if (units * n_kv_heads >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  p.units = (int)units;
  PromptMaps maps;
  if (!prompt_map(&maps.q, q, n_heads, n_rows, q_row_stride, p.G, p.pos) ||
      !prompt_map(&maps.k, k, n_kv_heads, n_rows, k_row_stride, 1, kPT) ||
      !prompt_map(&maps.v, v, n_kv_heads, n_rows, v_row_stride, 1, kPT))
    return DFLASH_E_CUDA;
  static std::atomic<bool> smem_done[kMaxDevices];
  if (ensure_smem_attr(smem_done, prompt_attn_kernel, kPromptSmem) != cudaSuccess)
    return DFLASH_E_CUDA;
  if (launch_k(true, prompt_attn_kernel, dim3((unsigned)(units * n_kv_heads)), dim3(kPromptThreads),
               kPromptSmem, (cudaStream_t)stream, maps, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
