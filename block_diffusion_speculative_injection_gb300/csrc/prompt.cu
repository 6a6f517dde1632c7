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
  int box_out;     // 32 rows are whole positions: maps.out has boxes of them
  int n_units;     // of tiles * pos positions, over all sequences
  PackedUnits units;
};

struct PromptMaps {
  CUtensorMap q, k, v, out;
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
// consistent m gives the same O / l.  A weight is rounded to bf16 (by up to 2^-8 of it) because V is
// bf16 and both operands of a product have one type; the sum l takes it unrounded.
//
// Keys behind a row's own position, or the prompt's end, have weight 0, which keeps finite values
// of V out, not NaN or infinities (0 * NaN): in the tiles that not every row of the CTA sees
// whole, a warp replaces those by zeros in shared memory.  If there were any, the rows that do see
// them add them to their results at the end.
//
// Shared memory (1024-aligned, rows of 128 B, 128-byte swizzle): Q 2 x 32 KB, a ring of four
// stages of 32 KB for K and V in the order K0 K1 V0 K2 V1 .., 32 KB for results on their way out.
// Tensor memory: S and O of both tiles, all 512 columns.
// Warps 0-3, 4-7: softmax of tile 0 and 1.  Warp 8: TMA.  Warps 9, 10: the tiles' MMAs, O(j) and
// then S(j + 1), so that S(j + 1) follows the last read of P(j), which it overwrites.  Warp 11: V.
//
// A CTA that is done with its two tiles takes on those of one that has not started, so that loads and
// scores of the next item begin under the results of the last, and SMs that had short items take more
// (32 ragged prompts: 1.68 -> 1.38 ms).  Items go from the last rows of the packed batch to the first: the
// long ones of a causal prompt before its short ones, but the prompts just as the caller has them, the last
// one first.  A batch of 8192 tokens and 64 times 256 takes 387 us with the longest prompt first or last,
// bidirectional (equally long items) 668 with it first and 651 with it last; 4096 and 200 times 128 take
// 183, and 260 and 236.
//
// What bounds it: a step of both tiles is four products of 4.2 MFLOP, 1.35 us at 1.89 PFLOP/s over
// 152 SMs.  Long prompts reach that (four of 8192, bidirectional, 32 heads: 2.33 ms); one of 16,384
// causal tokens takes 1.2 ms, 1.8 PFLOP/s (1.34 ms under the power cap, 96 % of the rate that a large
// library matrix product sustains there).  Shorter prompts pay 2.6 us for each change of items (the
// last step's chain, the results, the first scores) and some 0.25 us more for a step with a mask: 32
// prompts of 512 to 4096 take 1.22 ms, 1.54 PFLOP/s.  One of 2048 is 28.5 us with its inputs in L2, as the
// projection before leaves them, and 31.2 from memory: 16 steps in a row and two more changes; three
// short ones 7.1 us, a launch and one step.
//
// Measured and left: three stages instead of four (with the room, five) and P in one or four parts
// (slower); results by separate warps (slower: registers), in four parts of 32 dims through two
// buffers in turn (no gain), their second half behind the next item's first weights (2 % slower);
// items known three ahead, and the next CTA asked for three steps early (2048 tokens: 34 us instead
// of 30); V cleaned by the softmax warps in front of their stores (2 % slower); half a step's
// products and weights left out where the last step has no more than 64 keys (0.4 us less for
// short prompts, 2 to 5 % more for long ones: the loop's code is scheduled less well).
// ---------------------------------------------------------------------------
constexpr int kPT = 128;                       // rows of a query tile, keys of a step
constexpr uint32_t kPBox = kPT * 128;          // 128 rows of 64 dims
constexpr uint32_t kPStage = 2 * kPBox;        // a K, V or Q tile
constexpr int kPStages = 4;
constexpr uint32_t kPOffKV = 2 * kPStage;
constexpr uint32_t kPOffOut = kPOffKV + kPStages * kPStage;
constexpr uint32_t kPOutBytes = 32 * 128;      // a softmax warp's 32 rows of 64 dims on their way out
constexpr uint32_t kPOffBar = kPOffOut + 8 * kPOutBytes;
constexpr int kPromptSmem = (int)kPOffBar + 768 + 1024;  // barriers, alignment slack
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

// An item: two query tiles of a prompt and KV head, `index` of units * Hkv.
struct PromptItem {
  int first, n;          // the prompt's rows
  int p0a, p0b;          // first position of each query tile
  int steps_a, steps_b;  // key tiles each sees (0: no row)
  int clean;             // first key tile that not every row sees whole
  int kvh;
};
constexpr int kPParts = 2;    // of P: a part's products begin while the next is computed
constexpr int kPSlots = 2;    // items known ahead
constexpr int kPAskLate = 1;  // steps
constexpr int kPClean = 4;    // barriers of the cleaned tiles, used in turn
constexpr int kPIdle = 1 << 16;  // empty items after which there is word of them (70 ms; a wait ends after 2 s)
struct PromptShared {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][kPParts], o_full[2], o_empty[2], issued[2], drained[2];
  uint64_t raw_full[kPClean], clean[kPClean];
  uint64_t kv_full[kPStages], kv_empty[kPStages];
  uint64_t item_full[kPSlots], item_empty[kPSlots], next_full;
  PromptItem item[kPSlots];  // n = 0: no more
  int bad[kPSlots];          // whether V held a NaN or infinity in the tiles cleaned
  uint32_t tmem;
  alignas(16) uint8_t next[2][16];  // what a request for the next item answered
};
static_assert(sizeof(PromptShared) <= 768, "barriers fit");

// whole warp
__device__ __forceinline__ bool prompt_item(const PromptK& p, int index, PromptItem& it) {
  const int from_end = (int)((uint32_t)index / (uint32_t)p.Hkv);
  it.kvh = index - from_end * p.Hkv;
  // the last rows first: in a causal prompt they take longest
  const int u = p.n_units - 1 - from_end;
  const int b = packed_find(p.offsets, p.batch, p.units, u);
  if (b < 0 || !packed_rows(p.offsets, b, p.n_rows, it.first, it.n)) return false;
  const long long at = (u - packed_base(p.offsets, b, p.units)) * (p.tiles * p.pos);
  if (at >= it.n) return false;
  const int mask_from = p.causal ? (int)at + 1 : it.n;
  it.p0a = (int)at;
  it.p0b = (int)at + p.pos;
  auto steps = [&](int p0) {
    return ((p.causal ? min(it.n, p0 + p.pos) : it.n) + kPT - 1) / kPT;
  };
  it.steps_a = steps(it.p0a);
  it.steps_b = p.tiles > 1 && it.p0b < it.n ? steps(it.p0b) : 0;
  it.clean = min(mask_from / kPT, max(it.steps_a, it.steps_b));
  return true;
}

// which of an item's loads in ring order is K or V of step j of n
__device__ __forceinline__ int prompt_load_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int prompt_load_v(int j, int n) { return min(2 * j + 2, 2 * n - 1); }

// Asks for a CTA of this launch that has not started, to do its work here; the answer (16
// bytes) arrives on the barrier.
__device__ __forceinline__ void request_cta(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// its blockIdx.x, or -1: none is left (or the GPU wants them to start by themselves)
__device__ __forceinline__ int requested_cta(const void* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (int)x : -1;
}

// What every role but the producer keeps of the items it has passed.
struct PromptPast {
  int items;    // so far
  int loads;    // of the ring
  int cleaned;  // tiles of V
  __device__ __forceinline__ void pass(const PromptItem& it) {
    const int n = max(it.steps_a, it.steps_b);
    ++items;
    loads += 2 * n;
    cleaned += n - it.clean;
  }
};

__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptMaps maps, const PromptK p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  PromptShared& sh = *reinterpret_cast<PromptShared*>(sm + kPOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* const status = p.status;
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.q_full[x], 1);
      mbar_init(&sh.q_empty[x], 1);
      mbar_init(&sh.s_full[x], 1);
      for (int i = 0; i < kPParts; ++i) mbar_init(&sh.p_full[x][i], 4);
      mbar_init(&sh.o_full[x], 1);
      mbar_init(&sh.o_empty[x], 4);
      mbar_init(&sh.issued[x], 1);
      mbar_init(&sh.drained[x], 1);
    }
    for (int i = 0; i < kPClean; ++i) {
      mbar_init(&sh.clean[i], 1);
      mbar_init(&sh.raw_full[i], 1);
    }
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 2);
    }
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], 11);  // every warp but the producer
    }
    mbar_init(&sh.next_full, 1);
    mbar_fence_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  // (before there is tensor memory: the kernel before may not hold all of its own yet)
  pdl_wait();
  if (warp == 8) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = sh.tmem;
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    return __all_sync(0xffffffffu, warp_wait(bar, phase & 1, status));
  };
  // the next item (false: none, or a wait that ran out), and that this warp is done with it
  auto next_item = [&](const PromptPast& past, PromptItem& it) -> bool {
    const int slot = past.items % kPSlots;
    if (!wait(&sh.item_full[slot], past.items / kPSlots)) return false;
    it = sh.item[slot];
    return it.n > 0;
  };
  auto item_done = [&](const PromptPast& past) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_empty[past.items % kPSlots]);
  };

  if (warp >= 8) {
    regs_dec<kPIssueRegs>();
    const bool leader = elect_one();
    if (warp == 8) {
      // ---- producer: finds the items and loads them
      int issued = 0, cleaned = 0, items = 0, q_loads[2] = {0, 0};
      bool ok = true;
      auto load = [&](const PromptItem& it, bool is_v, int j) -> bool {
        const int st = issued % kPStages, round = issued / kPStages;
        if (round > 0 && !wait(&sh.kv_empty[st], round - 1)) return ok = false;
        // The tiles of V that are cleaned have barriers of their own: that warp does not
        // follow the ring, whose barriers have one bit for the round.
        const bool raw = is_v && j >= it.clean;
        if (leader) {
          uint8_t* const dst = sm + kPOffKV + st * kPStage;
          const CUtensorMap* const map = is_v ? &maps.v : &maps.k;
          uint64_t* full = &sh.kv_full[st];
          if (raw) {
            mbar_arrive(full);
            full = &sh.raw_full[cleaned % kPClean];
          }
          mbar_arrive_expect_tx(full, kPStage);
          tma_load_3d(dst, map, 0, it.kvh, it.first + j * kPT, full);
          tma_load_3d(dst + kPBox, map, 64, it.kvh, it.first + j * kPT, full);
        }
        __syncwarp();
        ++issued;
        if (raw) ++cleaned;
        return true;
      };
      auto load_q = [&](const PromptItem& it, int x, int p0, int steps, int& loads) -> bool {
        if (steps == 0) return true;
        if (loads > 0 && !wait(&sh.q_empty[x], loads - 1)) return ok = false;
        if (leader) {
          uint8_t* const dst = sm + x * kPStage;
          mbar_arrive_expect_tx(&sh.q_full[x], (uint32_t)(2 * 128 * p.G * p.pos));
          tma_load_3d(dst, &maps.q, 0, it.kvh * p.G, it.first + p0, &sh.q_full[x]);
          tma_load_3d(dst + kPBox, &maps.q, 64, it.kvh * p.G, it.first + p0, &sh.q_full[x]);
        }
        __syncwarp();
        ++loads;
        return true;
      };
      // makes an item known (n = 0: there are no more)
      auto publish = [&](const PromptItem& it) -> bool {
        const int slot = items % kPSlots, round = items / kPSlots;
        if (round > 0 && !wait(&sh.item_empty[slot], round - 1)) return ok = false;
        if (lane == 0) {
          sh.item[slot] = it;
          sh.bad[slot] = 0;
          mbar_arrive(&sh.item_full[slot]);
        }
        __syncwarp();
        ++items;
        return true;
      };
      int index = blockIdx.x;
#pragma unroll 1
      for (int asked = 0; ok && index >= 0; ++asked) {
        auto ask = [&]() {
          if (leader) {  // (the answer before was read: order that before the next one's writing)
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&sh.next_full, 16);
            request_cta(sh.next[asked & 1], &sh.next_full);
          }
          __syncwarp();
        };
        packed_check(p.offsets, p.batch, p.n_rows, 32ll * index + lane, 1ll << 40, status);
        PromptItem it;
        bool any = prompt_item(p, index, it);
        if (!any && asked % kPIdle == kPIdle - 1) {  // so that the others' waits do not run out
          memset(&it, 0, sizeof(it));
          it.n = 1;  // (an item without steps)
          any = true;
        }
        any = any && publish(it);
        const int n = any ? max(it.steps_a, it.steps_b) : 0;
        // The next item is asked for while the last steps' loads are under way; with few steps
        // there is no time for that, and little to share out better.
        if (n <= kPAskLate) ask();
        if (n > 0) {
          load(it, false, 0) && load_q(it, 0, it.p0a, it.steps_a, q_loads[0]) &&
              load_q(it, 1, it.p0b, it.steps_b, q_loads[1]);
#pragma unroll 1
          for (int j = 0; ok && j < n; ++j)
            if (j + 1 == n || load(it, false, j + 1)) load(it, true, j);
        }
        if (n > kPAskLate) ask();
        // (also after a failure: nothing may arrive here later)
        if (!wait(&sh.next_full, asked)) ok = false;
        index = requested_cta(sh.next[asked & 1]);
      }
      PromptItem none;
      memset(&none, 0, sizeof(none));
      if (ok) publish(none);
      // every issued copy has landed before this warp leaves
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const int n = x == 0 ? q_loads[0] : q_loads[1];
        if (n > 0) wait(&sh.q_full[x], n - 1);
      }
#pragma unroll 1
      for (int i = max(0, issued - kPStages); i < issued; ++i) wait(&sh.kv_full[i % kPStages], i / kPStages);
#pragma unroll 1
      for (int i = max(0, cleaned - kPClean); i < cleaned; ++i) wait(&sh.raw_full[i % kPClean], i / kPClean);
    } else if (warp <= 10) {
      // ---- MMA issuers, one for each query tile, so that one's waits pass beside the other's
      // products.  Whole warps wait, one lane issues: the descriptors stay in uniform registers.
      const int x = warp - 9;
      constexpr uint32_t id_s = idesc_bf16_f32(kPT, kPT);
      constexpr uint32_t id_o = idesc_bf16_f32(kPT, kPromptHd) | kIdescBMajorMN;
      const uint64_t q_desc = sw128_desc(smem_u32(sm + x * kPStage));
      const uint64_t k_desc = sw128_desc(smem_u32(sm + kPOffKV));
      const uint64_t v_desc = sw128_desc_mn(smem_u32(sm + kPOffKV), kPBox);
      const uint32_t t_s = tmem + kPTmemS + x * kPT, t_o = tmem + kPTmemO + x * kPromptHd;
      bool ok = true;
      auto wait_for = [&](uint64_t* bar, int phase) {
        if (ok) ok = wait(bar, phase);
        return ok;
      };
      auto wait_kv = [&](int at) { wait_for(&sh.kv_full[at % kPStages], at / kPStages); };
      PromptPast past = {0, 0, 0};
      int mine = 0, done = 0;  // items with rows in this tile, and their steps
      int turns = 0;           // steps that both tiles had
      PromptItem it;
#pragma unroll 1
      for (; ok && next_item(past, it); item_done(past), past.pass(it)) {
        const int steps = x == 0 ? it.steps_a : it.steps_b;
        const int n_steps = max(it.steps_a, it.steps_b), n_both = min(it.steps_a, it.steps_b);
        auto scores = [&](int j) {  // and K, after the last step Q, is free when they are done
          const int st = (past.loads + prompt_load_k(j)) % kPStages;
          tc_fence_after();
          if (leader) {
            const uint64_t kd = k_desc + st * (kPStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = ((kk >> 2) * kPBox + (kk & 3) * 32) >> 4;
              tc_mma_bf16(t_s, q_desc + off, kd + off, id_s, kk > 0 ? 1u : 0u);
            }
            tc_commit(&sh.s_full[x]);
            tc_commit(&sh.kv_empty[st]);
            if (j + 1 == steps) tc_commit(&sh.q_empty[x]);
          }
          __syncwarp();
        };
        if (steps > 0) {
          wait_kv(past.loads);
          if (wait_for(&sh.q_full[x], mine)) scores(0);
        }
#pragma unroll 1
        for (int j = 0; ok && j < steps; ++j) {
          const int at = past.loads + prompt_load_v(j, n_steps), st = at % kPStages;
          // the step's loads first (they are early), then only the softmax is waited for
          if (j + 1 < steps) wait_kv(past.loads + prompt_load_k(j + 1));
          const int c = past.cleaned + j - it.clean;
          if (j >= it.clean)
            wait_for(&sh.clean[c % kPClean], c / kPClean);
          else
            wait_kv(at);
          // O of the item before has been read
          if (j == 0 && mine > 0) wait_for(&sh.o_empty[x], mine - 1);
          // The tiles take turns, the first before the second.  Left to themselves both come at
          // once, their products pass in alternation and end together, and so do the softmaxes:
          // in step for good, with the tensor cores idle meanwhile (2.0 us a step instead of 1.4).
          const int turn = turns + j - (x == 0 ? 1 : 0);
          if (j < n_both && turn >= 0) wait_for(&sh.issued[1 - x], turn);
#pragma unroll
          for (int part = 0; part < kPParts; ++part) {
            if (!wait_for(&sh.p_full[x][part], done + j)) break;
            tc_fence_after();
            if (leader) {
              const uint64_t vd = v_desc + st * (kPStage >> 4);
              constexpr int kSteps = kPT / 16 / kPParts;  // of 16 keys
#pragma unroll
              for (int kk = kSteps * part; kk < kSteps * (part + 1); ++kk)
                tc_mma_f16_ta(t_o, t_s + 8 * kk, vd + kk * (16 * 128 >> 4), id_o, j + kk > 0 ? 1u : 0u);
              if (part == kPParts - 1) tc_commit(&sh.kv_empty[st]);
              if (part == kPParts - 1 && j + 1 == steps) tc_commit(&sh.o_full[x]);
            }
            __syncwarp();
          }
          if (ok && leader && j < n_both) mbar_arrive(&sh.issued[x]);
          if (ok && j + 1 < steps) scores(j + 1);
        }
        turns += n_both;
        // What this tile does not use is free as far as it is concerned, once it is loaded: an
        // arrival before that would count for the stage's load before.
#pragma unroll 1
        for (int i = 2 * steps; ok && i < 2 * n_steps; ++i) {
          const int at = past.loads + (i & 1 ? prompt_load_v(i >> 1, n_steps) : prompt_load_k(i >> 1));
          wait_kv(at);
          if (ok && leader) mbar_arrive(&sh.kv_empty[at % kPStages]);
          __syncwarp();
        }
        if (steps > 0) ++mine;
        done += steps;
      }
      // nothing of this warp is in flight when it leaves
      if (leader) tc_commit(&sh.drained[x]);
      __syncwarp();
      wait(&sh.drained[x], 0);
    } else {
      // ---- V without NaN and infinities where not every row sees all keys
      bool ok = true;
      PromptPast past = {0, 0, 0};
      PromptItem it;
#pragma unroll 1
      for (; ok && next_item(past, it); item_done(past), past.pass(it)) {
        const int n_steps = max(it.steps_a, it.steps_b);
        bool bad = false;
#pragma unroll 1
        for (int j = it.clean; j < n_steps; ++j) {
          const int st = (past.loads + prompt_load_v(j, n_steps)) % kPStages;
          const int c = past.cleaned + j - it.clean;
          if (!(ok = wait(&sh.raw_full[c % kPClean], c / kPClean))) break;
          uint4* const tile = reinterpret_cast<uint4*>(sm + kPOffKV + st * kPStage);
          // the largest exponent first: all ones is rare
          uint32_t top = 0;
#pragma unroll 8
          for (int i = lane; i < (int)(kPStage / 16); i += 32) {
            const uint4 v = tile[i];
            constexpr uint32_t ones = 0x7f807f80u;
            top = __vimax3_u16x2(top, v.x & ones, v.y & ones);
            top = __vimax3_u16x2(top, v.z & ones, v.w & ones);
          }
          if ((top & 0xffffu) == 0x7f80u || (top >> 16) == 0x7f80u) {
            bad = true;
#pragma unroll 1
            for (int i = lane; i < (int)(kPStage / 16); i += 32) {
              const uint4 v = tile[i];
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // a half whose exponent is all ones carries into its top bit
                const uint32_t b = ((w[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                w[e] &= ~((b - (b >> 15)) | b);
              }
              tile[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (bad) *const_cast<volatile int*>(&sh.bad[past.items % kPSlots]) = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.clean[c % kPClean]);
        }
      }
    }
    __syncwarp();
  } else {
    regs_inc<kPSoftRegs>();
    // ---- softmax: this thread's row of tile x
    const int x = warp >> 2, row = threadIdx.x & 127;
    const int g_pos = row * p.g_inv >> 16;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + kPTmemS + x * kPT, t_o = lanes + kPTmemO + x * kPromptHd;
    bool ok = true;
    PromptPast past = {0, 0, 0};
    int mine = 0, done = 0;  // items with rows in this tile, and their steps
    PromptItem it;
#pragma unroll 1
    for (; ok && next_item(past, it); item_done(past), past.pass(it)) {
      const int n_mine = x == 0 ? it.steps_a : it.steps_b;
      if (n_mine == 0) continue;
      const int p0 = x == 0 ? it.p0a : it.p0b, pos = p0 + g_pos;
      const int limit = p.causal ? min(pos + 1, it.n) : it.n;  // its keys
      const int mask_from = p.causal ? p0 + 1 : it.n;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < n_mine; ++j) {
        if (!(ok = wait(&sh.s_full[x], done + j))) break;
        tc_fence_after();
        uint32_t s[kPT];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_nowait(t_s + 32 * c, s + 32 * c);
        tmem_wait_ld();
        if ((j + 1) * kPT > mask_from) {
          const int end = limit - j * kPT, all = __shfl_sync(0xffffffffu, end, 0);  // (rows see more and more)
#pragma unroll
          for (int c = 0; c < kPT; c += 32) {
            // (bits to predicates eight at a time: half the instructions of a comparison each)
            if (all >= c + 32) continue;
            const int n = end - c;
            const uint32_t seen = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((seen >> i) & 1u)) s[c + i] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mx[c] = max3(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]), -INFINITY);
#pragma unroll
        for (int i = 8; i < kPT; i += 2) {
          float& t = mx[(i >> 1) & 3];
          t = max3(t, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        }
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        const bool grown = top > m + kPLazy || (m == -INFINITY && top > m);
        const float m_next = grown ? top : m;
        float base = m_next == -INFINITY ? 0.f : -m_next * kPScaleLog2;
        const bool far = fabsf(m_next) > kPFar && m_next != -INFINITY;
        // (at the first step there is nothing to rescale, nor this code to be fetched)
        if (__any_sync(0xffffffffu, (grown && j > 0) || far)) {
          if (j > 0 && __any_sync(0xffffffffu, grown)) {
            // O holds the steps before: S(j) is complete, so they are
            const float alpha = grown ? ex2((m - top) * kPScaleLog2) : 1.f;
            l *= alpha;
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
          if (far) {
            const float2 minus_m = make_float2(-m_next, -m_next);
#pragma unroll
            for (int i = 0; i < kPT; i += 2) {
              const float2 y =
                  add2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), minus_m);
              s[i] = __float_as_uint(y.x);
              s[i + 1] = __float_as_uint(y.y);
            }
            base = 0.f;
          }
        }
        m = m_next;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto stored = [&](int part) {  // P of this part is in tensor memory
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[x][part]);
        };
        constexpr int kWords = kPT / 2 / kPParts;
#pragma unroll
        for (int part = 0; part < kPParts; ++part) {
          float pk[kWords];
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const int e = 2 * (kWords * part + i);
            float2 z = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), kPScaleLog2,
                            base);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            sum[i & 1] = add2(sum[i & 1], z);
            const __nv_bfloat162 h = __floats2bfloat162_rn(z.x, z.y);
            pk[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
          }
          if (part > 0) stored(part - 1);  // (the store passes while this part is computed)
#pragma unroll
          for (int i = 0; i < kWords; i += 16) tmem_st16(t_s + kWords * part + i, pk + i);
        }
        stored(kPParts - 1);
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      }
      // ---- the rows' results.  (Rolled, and as little as can be behind the wait: this code runs once
      // an item, and the instruction cache has forgotten it by then.)
      const float inv = l == 0.f ? 0.f : rcp(l);
      const int n_live = min(p.pos, it.n - p0) * p.G;  // rows of the prompt
      // first of the tile's rows: position p0, the first head of this KV head
      const long long row0 = (long long)(it.first + p0) * p.H + it.kvh * p.G;
      if (row < n_live && p.lse)
        p.lse[row0 + g_pos * (p.H - p.G) + row] =
            l == 0.f ? -INFINITY : (m * kPScaleLog2 + log2f(l)) * kPLn2;
      // Out through shared memory, 64 dims at a time (16 bytes at chunk c ^ row): a row a lane would
      // touch 32 lines an instruction, so 32 turns of the memory pipe instead of 4.  A warp whose 32
      // rows are all the prompt's, and whole positions, leaves them to one bulk copy.
      uint8_t* const out_rows = sm + kPOffOut + warp * kPOutBytes;
      const int rr0 = (warp & 3) * 32;
      const bool bulk = p.box_out && rr0 + 32 <= n_live;
      if (ok) ok = wait(&sh.o_full[x], mine);
      if (!ok) break;
      tc_fence_after();
      const bool bad = *const_cast<volatile int*>(&sh.bad[past.items % kPSlots]) != 0;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (lane == 0) bulk_wait_read();  // what was here before has left
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          tmem_ld32_nowait(t_o + 64 * half + 32 * c, o);
          tmem_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y = mul2(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), inv);
            const __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(out_rows + lane * 128 + (((4 * c + i) ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        if (half == 1) {  // O may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.o_empty[x]);
        }
        if (bad && row < n_live) {
          // what this row sees of the elements that were replaced by zeros
#pragma unroll 1
          for (int key = it.clean * kPT; key < limit; ++key) {
            const bf16* const v = p.v + (long long)(it.first + key) * p.vs + it.kvh * kPromptHd + 64 * half;
#pragma unroll 1
            for (int d = 0; d < 64; ++d) {
              const float f = ld_f(v + d);
              bf16* const y = reinterpret_cast<bf16*>(out_rows + lane * 128 + (((d >> 3) ^ (lane & 7)) << 4)) +
                              (d & 7);
              if (!(fabsf(f) < INFINITY)) st_f(y, ld_f(y) + f);
            }
          }
        }
        if (bulk) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&maps.out, out_rows, 64 * half, it.kvh * p.G,
                         it.first + p0 + (rr0 * p.g_inv >> 16));
            bulk_commit();
          }
        } else {
          __syncwarp();
#pragma unroll 2
          for (int i = lane; i < 32 * 8; i += 32) {
            const int r = i >> 3, c = i & 7, g = (rr0 + r) * p.g_inv >> 16;
            if (rr0 + r < n_live)
              *reinterpret_cast<uint4*>(p.out + (row0 + g * (p.H - p.G) + rr0 + r) * kPromptHd + 64 * half +
                                        8 * c) =
                  *reinterpret_cast<const uint4*>(out_rows + r * 128 + ((c ^ (r & 7)) << 4));
          }
        }
        __syncwarp();
      }
      ++mine;
      done += n_mine;
    }
    if (lane == 0) bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

static bool prompt_stride_ok(int64_t stride, int heads) {
  return stride >= (int64_t)heads * kPromptHd && stride % 8 == 0 && stride < ((int64_t)1 << 31);
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
  if (batch < 1 || batch >= (1 << 26) || n_rows < 1 || n_rows >= (1 << 26) || n_heads < 1 ||
      n_heads > 65535 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 64 ||
      (causal != 0 && causal != 1) || !offsets || !q || !k || !v || !out || !status ||
      !prompt_stride_ok(q_row_stride, n_heads) || !prompt_stride_ok(k_row_stride, n_kv_heads) ||
      !prompt_stride_ok(v_row_stride, n_kv_heads) || !kvq_aligned(q, 16) || !kvq_aligned(k, 16) ||
      !kvq_aligned(v, 16) || !kvq_aligned(out, 16) || !kvq_aligned(lse, 4) ||
      !kvq_ints_aligned({offsets, status}))
    return DFLASH_E_INVALID_ARG;
  // What is written must be nothing that other CTAs still read, nor the other output.
  auto bytes = [&](int64_t stride, int heads) {
    return ((n_rows - 1) * stride + (int64_t)heads * kPromptHd) * 2;
  };
  const MemRange in[] = {{q, bytes(q_row_stride, n_heads)},
                      {k, bytes(k_row_stride, n_kv_heads)},
                      {v, bytes(v_row_stride, n_kv_heads)},
                      {offsets, ((int64_t)batch + 1) * 4},
                      {status, 4}};
  const MemRange o[] = {{out, (int64_t)n_rows * n_heads * kPromptHd * 2},
                     {lse, (int64_t)n_rows * n_heads * 4}};
  if (!ranges_apart(o, 2, in, 5)) return DFLASH_E_INVALID_ARG;
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
  p.box_out = 32 % p.G == 0;
  // Two query tiles a CTA, each beside the other's softmax; one while that leaves no SM two CTAs.  32
  // and 8 heads, inputs in L2, one prompt of 256: 7.4 us by one tile, 8.3 by two; 512: 10.7 and 11.1;
  // 1024: 19.5 and 16.9, bidirectional 26.7 and 16.9.
  p.tiles = 2 * packed_units(n_rows, batch, 2 * p.pos, 1) * n_kv_heads <= kvq_sms() ? 1 : 2;
  const int64_t units = packed_units(n_rows, batch, p.tiles * p.pos, 1);
  if (units * n_kv_heads >= ((int64_t)1 << 31)) return DFLASH_E_INVALID_ARG;
  p.n_units = (int)units;
  p.units = packed_units_of(p.tiles * p.pos, 1);
  PromptMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!prompt_map(&maps.q, q, n_heads, n_rows, q_row_stride, p.G, p.pos) ||
      !prompt_map(&maps.k, k, n_kv_heads, n_rows, k_row_stride, 1, kPT) ||
      !prompt_map(&maps.v, v, n_kv_heads, n_rows, v_row_stride, 1, kPT) ||
      (p.box_out && !prompt_map(&maps.out, out, n_heads, n_rows, (int64_t)n_heads * kPromptHd, p.G, 32 / p.G)))
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
