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
  int pos, g_inv;  // block positions of a CTA's 64 rows; row / G = row * g_inv >> 16 (row < 64)
  int q_tiles, n_splits;
  float *part_o, *part_ml;  // [split][row][head][128], [split][row][head] (m, l)
};

constexpr float kScaleLog2 = 0.12751743f;  // log2(e) / sqrt(128)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Entry b: sequence, slots n, rows r, and the first slot the cache cannot hold
// or the sequence does not have (key_end); false: skip it.  In two steps, so that
// the loads can be under way while something else is done.
struct KvqEntry {
  int seq, n, r;
};
__device__ __forceinline__ KvqEntry kvq_entry_load(const KvqAttnK& p, int b) {
  KvqEntry e;
  e.seq = p.seq_ids ? p.seq_ids[b] : b;
  e.n = p.kv_lens[b];
  e.r = p.q_lens ? p.q_lens[b] : p.block;
  return e;
}
__device__ __forceinline__ bool kvq_entry_check(const KvqAttnK& p, const KvqEntry& e, int& key_end) {
  key_end = 0;
  if (e.seq < 0 || e.seq >= p.c.n_seqs || e.n < 0 || e.r < 0 || e.r > p.block) {
    set_dev_status(p.c.status, kDevCheck);
    return false;
  }
  key_end = min(e.n, p.c.pps * kPageSlots);
  if (key_end < e.n) set_dev_status(p.c.status, kDevCapacity);
  return true;
}
__device__ __forceinline__ bool kvq_entry(const KvqAttnK& p, int b, int& seq, int& n, int& r,
                                          int& key_end) {
  const KvqEntry e = kvq_entry_load(p, b);
  seq = e.seq;
  n = e.n;
  r = e.r;
  return kvq_entry_check(p, e, key_end);
}

// ---------------------------------------------------------------------------
// Attention on the 5th-generation tensor cores: q . K in 8 bits, the weights times V in 16.
//
// One CTA: 64 query rows (64 / G block positions x the G query heads of a KV
// head) against one split of the sequence's slots, a page (128 slots) a tile.
// K goes from the pages to the tensor cores as it is (e4m3, TMA); q, which is not 8-bit, in
// two e4m3 parts:
//
//   q = 2^a (q1 + q2): q1 = e4m3(q 2^-a), q2 = e4m3 of what q1 leaves.  The parts'
//   4 + 4 significand bits hold a bf16 (8 bits) exactly where the element is above
//   2^-10 of the row's largest, and to 2^-18 of that below.  S = Q1 K^T + Q2 K^T,
//   two MMAs (M = 64) into one accumulator.
//
//   The weights carry V's exponents: with u_k = log2(e) s_k + eV_k (eV_k the exponent of
//   slot k's block of V), z_k = 2^(u_k - m + 11) is the weight of the CODES of V, and the
//   softmax sum is sum z_k 2^-eV_k.  So neither K's exponents (a factor of S) nor V's (an
//   addend of the exponent) cost a multiplication an element.
//
//   z is held in fp16, with m (a maximum met so far) so that a row's largest is in
//   [2^11, 2^15]: off by at most 2^-11 of itself down to 2^-14, by 2^-25 below, which is 2^-36
//   of the largest.  So the thin tail beside a slot that draws nearly all of the weight
//   keeps its 11 bits, and 131,072 slots below that floor sum to less than 2^-18 of the
//   largest.  (Two e4m3 parts of z lose the tail: their codes end some 17 binades below the
//   largest.)
//   V's codes are exact in fp16.  Four warps convert each tile once, transposed, into tensor memory:
//   O^T = V^T Z^T is an M = 128 MMA (full rate) with A = V^T there and B = Z in shared memory.
//   Through shared memory the fp16 V would be written and read again at twice the bytes of its
//   codes, and shared memory would bound the loop (1800 of 2190 cycles a tile, measured so).
//
// Shared memory (1024-aligned, rows of 128 B, 128-byte swizzle):
//   Q1, Q2 [64][128] 8 KB each; Z fp16 [2][64 rows][64 slots] 16 KB, twice; two stages of K and
//   two of V [128 slots][128], 16 KB each.  112 KB, so two CTAs share an SM: one's softmax runs
//   beside the other's MMAs and loads.
// Tensor memory: 256 columns, S [64 rows][128] twice, V^T [128 dims][128 slots] in fp16 (64
// columns), O^T [128 dims][64 rows].  An M = 64 accumulator keeps row m in lane
// (m / 16) * 32 + m % 16, so a second one fits into the other 16 lanes of each quarter: S of
// odd tiles starts at lane 16.
//
// Warps 0-3 (softmax): two threads per row (lanes t, t + 16), 64 slots each, held in registers.
// Warps 4-7: V to fp16, and O's rescaling when a row's maximum has grown by more than a factor
// 16 (its columns are all four's).  Warp 8 (producer): TMA of K and V.  Warp 9: the MMAs, S two
// tiles ahead of O^T.  (Warps 10 and 11 only complete a warpgroup, whose registers the softmax takes
// over.)  A softmax warp none of whose rows is in use only takes part in the barriers.
//
// Measured: 32 sequences of one row over 24,000 to 32,769 slots (1.89 GB) 309 us, 6.1 TB/s; 8
// sequences of 16 rows over 16,400 slots (271 MB) 57 us, 4.8 TB/s; 1000 rows of 2 sequences
// over 2500 to 5097 slots 216 us.
// Tried and slower (8 sequences of 8 KV heads over 16,384 slots, 1 and 16 rows a sequence; kept form
// 50 and 56 us): the conversion in rolled loops (81, 85), on eight warps instead of four (66, 76),
// with the header's 16-bit operands instead of both halves of a register at once (56, 64); V in
// fp16 through shared memory, one buffer, a ring of quarters or Z in halves (32,769 slots a row: 388 to
// 407 us against 307); softmax warps without rows left out of the barriers (54, 62: spills).
// Earlier forms: S re-read from tensor memory instead of held in registers, eight softmax warps of 32
// slots a thread, the tile's maximum looked for only after a weight overflowed, shares of the longest
// sequence instead of each sequence's own: each 20 % and more slower.
// ---------------------------------------------------------------------------
constexpr int kTile = kPageSlots;
constexpr uint32_t kTileBytes = kTile * kKvqHd;  // one K or V tile in codes, and Z
constexpr uint32_t kQPart = 64 * kKvqHd;
constexpr uint32_t kZBlock = 64 * 128;       // Z of 64 slots
constexpr uint32_t kAOffZ = 2 * kQPart;
constexpr uint32_t kAOffK = kAOffZ + 2 * 2 * kZBlock;
constexpr int kAStages = 2;  // of K and of V
constexpr uint32_t kAOffV = kAOffK + kAStages * kTileBytes;
constexpr uint32_t kAOffQs = kAOffV + kAStages * kTileBytes;  // scale of each query row; later
constexpr uint32_t kAOffAlpha = kAOffQs;                      // [2][64] factors of rescaling
constexpr uint32_t kAOffGrown = kAOffAlpha + 2 * 64 * 4;      // [2][4] whether a warp has any
constexpr uint32_t kAOffBar = kAOffGrown + 2 * 4 * 4;
constexpr uint32_t kORow = kKvqHd * 4 + 16;  // an accumulator row staged over Q and Z, padded
static_assert(64 * kORow <= kAOffK, "accumulator rows fit");
constexpr int kAttnQSmem = (int)kAOffBar + 256;  // barriers
static_assert(2 * (kAttnQSmem + 1024) <= 228 * 1024, "two CTAs on an SM");
// Three warpgroups of 80 registers a thread: the softmax takes over what the others leave.
constexpr int kAttnQThreads = 384;
constexpr int kAttnRegs = 80, kSoftmaxRegs = 128, kConvertRegs = 56, kIssueRegs = 56;
static_assert(2 * kAttnQThreads * kAttnRegs <= 65536, "two CTAs on an SM");
static_assert(kSoftmaxRegs + kConvertRegs + kIssueRegs <= 3 * kAttnRegs,
              "what one takes the others leave");
constexpr uint32_t kAttnQTmem = 256, kTmemVCol = 128, kTmemOCol = 192;
constexpr uint32_t kSOdd = 16u << 16;  // lane offset of the S buffer of odd tiles
// z of the largest weight, when it is met, and its growth that is not yet rescaled: z <= 2^15.
// (Rescaling at a factor of 2, 58 % of the warps' tiles rescaled O on 33-page splits, at 16
// one in ten does.)
constexpr float kTopLog2 = 11.f, kLazyLog2 = 4.f;
// Maxima (in units of log2) up to which their own rounding, that of kTopLog2 - m and that of its
// sum with an exponent, 2^-4 each at most, keep z below 2^15.2.
constexpr float kFarLog2 = 1048576.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / l to one or two units in the last place (l is a sum of weights, or NaN), and
// log2 within 2^-22
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// log of a softmax sum l of z (l 2^-11 is at most the row's slots, and 1 where one has all the
// weight: log2 is most exact there)
__device__ __forceinline__ float lse_of(float m, float l) {
  return (m + __log2f(l * (1.f / 2048))) * kLn2;
}
static_assert(kTopLog2 == 11.f, "2^kTopLog2 = 2048");
// the values of four e4m3 codes, two a word
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// where the NaN bits of a slot of the tile in stage st lie, for the dims 32 cw .. + 31: in the
// codes they stand for
__device__ __forceinline__ uint8_t* nan_bits(uint8_t* sm, int st, int slot, int cw) {
  return sm + kAOffV + st * kTileBytes + slot * 128 + ((2 * cw ^ (slot & 7)) << 4);
}
// V's codes of 32 dims in shared memory: zeros from slot `end` on, and in place of NaN from slot
// `from` on, noted in a bit for each dim of the lane's slots lane + 32 k.
__device__ __forceinline__ void clean_v(uint8_t* sm, int st, int cw, int lane, int end, int from,
                                        uint32_t* found) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int slot = lane + 32 * k;
    found[k] = 0;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      uint4* const at = reinterpret_cast<uint4*>(sm + kAOffV + st * kTileBytes + slot * 128 +
                                                 (((2 * cw + hh) ^ (slot & 7)) << 4));
      if (slot >= end) {
        *at = make_uint4(0u, 0u, 0u, 0u);
      } else if (slot >= from) {
        const uint4 v = *at;
        uint32_t w[4] = {v.x, v.y, v.z, v.w}, bits = 0;  // a bit per byte
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t m = ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
          w[i] &= ~(m | (m - (m >> 7)));
          bits |= ((m >> 7) * 0x10204080u >> 28) << (4 * i);
        }
        if (bits) *at = make_uint4(w[0], w[1], w[2], w[3]);
        found[k] |= bits << (16 * hh);
      }
    }
  }
}
// Registers a thread of this warpgroup gives back or takes over (all its warps together).
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// bits below n set (n clamped to 0..32)
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : ((1u << n) - 1u));
}

// (a0, a1) * b + c and (a0, a1) + (b0, b1) in one instruction each
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// block position (within the CTA's) of one of its 64 rows
__device__ __forceinline__ int row_pos(const KvqAttnK& p, int row) { return row * p.g_inv >> 16; }

// Slots of a split: a sequence's are shared out over the launch's splits in whole pages;
// `used` splits are not empty.
struct KvqSpan {
  int key_end, per_split, used;
};
__device__ __forceinline__ KvqSpan kvq_span(const KvqAttnK& p, int n, int r, int key_end, int j1) {
  KvqSpan s;
  // rows j < j1 of a causal pass see slots below n - r + j1
  s.key_end = p.mask == DFLASH_MASK_CAUSAL ? min(key_end, n - r + j1) : key_end;
  s.key_end = max(s.key_end, 0);
  const int tiles = (s.key_end + kTile - 1) / kTile;
  const int per = max(1, (tiles + p.n_splits - 1) / p.n_splits);
  s.per_split = per * kTile;
  s.used = (tiles + per - 1) / per;
  return s;
}

// visibility of slots kb .. kb + 31 (all below `stop`) for row j
__device__ __forceinline__ uint32_t visible32(const KvqAttnK& p, int kb, int stop, int ctx, int j,
                                              const uint64_t* anc) {
  const uint32_t m = bits_below(stop - kb);
  if (p.mask == DFLASH_MASK_NONE) return m;
  if (p.mask == DFLASH_MASK_CAUSAL) return m & bits_below(ctx + j + 1 - kb);
  uint32_t t = 0;
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {  // the one or two words that 32 ancestor bits span
    const int i0 = kb - ctx;     // block index of bit 0
    const int word = (i0 >> 6) + w;
    if (word < 0 || word >= p.anc_words) continue;
    const int sh = word * 64 - i0;  // where the word's bit 0 lands
    if (sh >= 32 || sh <= -64) continue;
    t |= (uint32_t)(sh >= 0 ? anc[word] << sh : anc[word] >> -sh);
  }
  return m & (bits_below(ctx - kb) | t);
}

// The 16 query rows of a warp, from global memory: two rows a load, lane l holds dims
// 8 (l % 16) .. of row 2 i + l / 16 in raw[i].  Rows past a sequence's count are in
// bounds (j < block) and dropped later.
__device__ __forceinline__ void load_q(const KvqAttnK& p, int b, int kvh, int j0, int warp, int lane,
                                       uint4* raw) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = warp * 16 + 2 * i + (lane >> 4), g = row_pos(p, row), j = j0 + g;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < p.pos * p.G && j < p.block)
      raw[i] = *reinterpret_cast<const uint4*>(p.q + ((long long)b * p.block + j) * p.q_stride +
                                               (kvh * p.G + row - g * p.G) * kKvqHd +
                                               8 * (lane & 15));
  }
}

// Those rows in two e4m3 parts, to dst [64][128] and dst + kQPart (128-byte
// swizzle), and their scales 2^a log2(e) / sqrt(128) (minus that for a row with a
// NaN, an infinity or a magnitude above 448 * 2^118: such a row is NaN).
// y = q 2^-(a + 8) in fp16 is exact but for elements below 2^-15 of the largest; an
// fp16 below 2 is an e4m3 code times 2^8 with three more significand bits, so the
// parts come out of integer operations on its bits.
__device__ __forceinline__ void convert_q(uint4* q_raw, int warp, int lane, uint8_t* dst,
                                          float* q_scales) {
  const int t16 = lane & 15, h = lane >> 4;
  // largest magnitude of each row, on bf16 pairs (as integers, NaN above all)
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    constexpr uint32_t abs2 = 0x7fff7fffu;
    top[i] = __vimax3_u16x2(q_raw[i].x & abs2, q_raw[i].y & abs2, q_raw[i].z & abs2);
    top[i] = __vmaxu2(top[i], q_raw[i].w & abs2);
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], off));
#pragma unroll 1
  for (int i = 0; i < 8; i += 2) {  // two of the lane's eight rows, for overlap
    uint4 now[2];
    uint32_t bits[2], w1[2][4], w2[2][4];
    int e[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      now[r] = q_raw[r];
      bits[r] = max(top[r] & 0xffffu, top[r] >> 16) << 16;
      // the smallest e with a <= 448 * 2^e; a row with a NaN, an infinity or a
      // magnitude above 448 * 2^118 becomes NaN
      e[r] = max(-80, (int)(bits[r] >> 23) - 127 - ((bits[r] & 0x7fffff) > 0x600000 ? 7 : 8));
    }
#pragma unroll
    for (int k = 0; k < 6; ++k) {  // keeps the loop rolled
      q_raw[k] = q_raw[k + 2];
      top[k] = top[k + 2];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sc = pow2i(-min(e[r], 118) - 8);
        const uint32_t q2 = k == 0 ? now[r].x : k == 1 ? now[r].y : k == 2 ? now[r].z : now[r].w;
        const __half2 y = __floats2half2_rn(__uint_as_float(q2 << 16) * sc,
                                            __uint_as_float(q2 & 0xffff0000u) * sc);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&y) + 0x00400040u;
        const uint32_t d = u & 0xff80ff80u;
        const __half2 res = __hsub2(y, *reinterpret_cast<const __half2*>(&d));
        const uint32_t v = *reinterpret_cast<const uint32_t*>(&res) + 0x00400040u;
        w1[r][k] = ((u + u) & 0x7fff7fffu) | (u & 0x80008000u);
        w2[r][k] = ((v + v) & 0x7fff7fffu) | (v & 0x80008000u);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int qr = warp * 16 + 2 * (i + r) + h;
      const uint32_t off =
          (uint32_t)qr * 128 + ((uint32_t)((t16 >> 1) ^ (qr & 7)) << 4) + 8 * (t16 & 1);
      *reinterpret_cast<uint2*>(dst + off) = make_uint2(__byte_perm(w1[r][0], w1[r][1], 0x7531),
                                                       __byte_perm(w1[r][2], w1[r][3], 0x7531));
      *reinterpret_cast<uint2*>(dst + kQPart + off) = make_uint2(
          __byte_perm(w2[r][0], w2[r][1], 0x7531), __byte_perm(w2[r][2], w2[r][3], 0x7531));
      // a bad row: minus its scale
      if (t16 == 0)
        q_scales[2 * (i + r) + h] = e[r] > 118 ? -kScaleLog2 : pow2i(e[r]) * kScaleLog2;
    }
  }
}

__device__ __forceinline__ float2 mul2(float2 a, float b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b));
  return r;
}

// Rows of the q tile from block position j0 on that see block slot i (r rows in the
// sequence), a bit each.
__device__ __forceinline__ uint64_t score_rows_seeing(const KvqAttnK& p, int b, int i, int j0, int r) {
  if (p.mask == DFLASH_MASK_CAUSAL) {
    const int from = max(i - j0, 0);  // positions from here on
    return from >= p.pos ? 0ull : ~0ull << (from * p.G);
  }
  uint64_t v = 0;
  if ((i >> 6) >= p.anc_words) return 0;
  const uint64_t* const a = p.anc + (long long)b * p.block * p.anc_words + (i >> 6);
  const uint64_t head = p.G == 64 ? ~0ull : (1ull << p.G) - 1;
#pragma unroll 1
  for (int q = 0; q < p.pos && j0 + q < r; ++q)
    if ((a[(long long)(j0 + q) * p.anc_words] >> (i & 63)) & 1ull) v |= head << (q * p.G);
  return v;
}

struct KvqMaps {
  CUtensorMap k, v;
};

// Bounded wait of a whole warp (every lane polls, so every lane has the
// barrier's ordering): gives up after about 2 s, like mbar_wait.  A poll may suspend
// the warp for up to 20 us (a hint), so a waiting warp leaves its issue slots to
// the others, and the clock is read only after such a poll has failed.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int32_t* status) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; i < kSpinLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if ((i & 15u) == 0) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > 2000000000ull) break;
    }
  }
  set_dev_status(status, kDevTimeout);
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return warp_wait(smem_u32(bar), parity, status);
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// one lane of a converged warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__global__ void __launch_bounds__(kAttnQThreads, 2)
    kvq_attn_kernel(const __grid_constant__ KvqMaps maps, const KvqAttnK p) {
  pdl_wait();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (the swizzled tiles want 1024-byte alignment, and two CTAs' shared memory leaves
  // no slack for it)
  uint8_t* const sm = smem_raw;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int POS = p.pos;
  const int b = blockIdx.z / p.n_splits, split = blockIdx.z % p.n_splits;
  const int kvh = blockIdx.y, j0 = blockIdx.x * POS;
  int32_t* const status = p.c.status;
  const KvqEntry entry = kvq_entry_load(p, b);
  // the query rows' loads, under way during the set-up
  const int t16 = lane & 15, h = lane >> 4;
  uint4 q_raw[8];
  if (warp < 4) load_q(p, b, kvh, j0, warp, lane, q_raw);

  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + kAOffBar);
  uint64_t* const q_full = bars;
  uint64_t* const meet = bars + 1;  // the softmax warps among themselves
  uint64_t* const o_ready = bars + 2;   // O is rescaled for the tile
  uint64_t* const nan_full = bars + 3;  // NaN's places in a tile, see below
  uint64_t* const nan_read = bars + 4;
  uint64_t* const s_full = bars + 5;  // two S buffers
  uint64_t* const a_full = bars + 7;  // two buffers of the rows' rescaling factors
  uint64_t* const z_full = bars + 9;  // two Z buffers; S of the tile is read
  uint64_t* const vt_full = bars + 11;  // the two halves of V^T
  uint64_t* const vt_empty = bars + 13;
  uint64_t* const o_done = bars + 15;  // all of O
  uint64_t* const k_full = bars + 16;
  uint64_t* const k_empty = k_full + kAStages;
  uint64_t* const v_full = k_empty + kAStages;
  uint64_t* const v_empty = v_full + kAStages;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(v_empty + kAStages);
  volatile int* const nan_any = reinterpret_cast<volatile int*>(tslot + 1);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 4);
    mbar_init(meet, 4);
    mbar_init(o_ready, 4);
    mbar_init(o_done, 1);
    mbar_init(nan_full, 4);
    mbar_init(nan_read, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&a_full[i], 4);
      mbar_init(&z_full[i], 4);
      mbar_init(&vt_full[i], 4);
      mbar_init(&vt_empty[i], 1);
    }
    for (int i = 0; i < kAStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 4);
    }
    nan_any[0] = nan_any[1] = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    tmem_alloc(tslot, kAttnQTmem);
    tmem_relinquish();
  }
  int key_end;
  bool work = kvq_entry_check(p, entry, key_end) && j0 < entry.r;
  if ((smem_u32(sm) & 1023u) != 0) {
    set_dev_status(status, kDevCheck);
    work = false;
  }
  const int seq = entry.seq, n = entry.n, r = entry.r;
  const int j1 = min(j0 + POS, r), ctx = n - r;
  const KvqSpan span = kvq_span(p, n, r, key_end, j1);
  const int k_begin = split * span.per_split;
  const int k_stop = min(span.key_end, k_begin + span.per_split);
  const int n_tiles = work && k_stop > k_begin ? (k_stop - k_begin + kTile - 1) / kTile : 0;

  // the row of a softmax thread
  const int row = warp * 16 + t16;
  const int jg = row_pos(p, row);
  const int jr = j0 + jg, hr = kvh * p.G + row - jg * p.G;
  const bool live = work && warp < 4 && row < POS * p.G && jr < j1;
  const long long grow = (long long)b * p.block + jr;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // dependents start once every CTA holds its tensor memory: one that allocates
  // earlier could keep this kernel waiting for columns while it waits for us
  pdl_trigger();
  const uint32_t tmem = *tslot;
  const int first_page = k_begin / kPageSlots;
  // rows of the CTA that a launch can use, in the granularity of an MMA's N
  const int rows16 = (min(p.block, POS) * p.G + 15) & ~15;
  // slots from here on are not seen by every row of the CTA
  const int mask_from = p.mask == DFLASH_MASK_NONE     ? k_stop
                        : p.mask == DFLASH_MASK_CAUSAL ? min(k_stop, ctx + j0 + 1)
                                                       : min(k_stop, ctx);

  if (n_tiles == 0) {
    // no slot at all: rows without anything seen get zeros (an unused split of a
    // longer sequence has nothing to do: the merge knows the used ones)
    if (split == 0 && live) {
      uint4* o = reinterpret_cast<uint4*>(p.out + (grow * p.H + hr) * kKvqHd + 64 * h);
      for (int i = 0; i < 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse && h == 0) p.lse[grow * p.H + hr] = -INFINITY;
    }
  } else if (warp >= 8) {
    regs_dec<kIssueRegs>();
    if (warp == 8) {
      // ---- producer: K one tile ahead of V; an unmapped page loads page 0 (the
      // softmax does not see its slots).  Whole warps wait, one lane issues: the
      // addresses and descriptors stay in uniform registers.
      const bool leader = elect_one();
      if (leader) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
      }
      int k_issued = 0, v_issued = 0;
      auto load = [&](int t, bool is_v, int pg) -> bool {
        const int st = t % kAStages, ph = (t / kAStages) & 1;
        uint64_t* empty = is_v ? &v_empty[st] : &k_empty[st];
        uint64_t* full = is_v ? &v_full[st] : &k_full[st];
        if (t >= kAStages && !__all_sync(0xffffffffu, warp_wait(empty, ph ^ 1, status))) return false;
        if (leader) {
          mbar_arrive_expect_tx(full, kTileBytes);
          tma_load_2d(sm + (is_v ? kAOffV : kAOffK) + st * kTileBytes, is_v ? &maps.v : &maps.k, 0,
                      (max(pg, 0) * p.c.Hkv + kvh) * kPageSlots, full);
        }
        __syncwarp();
        return true;
      };
      int raw_k = kvq_page_load(p.c, seq, first_page), pg_v = 0;
#pragma unroll 1
      for (int t = 0; t <= n_tiles; ++t) {
        const int pg_k = kvq_page_check(p.c, raw_k);
        raw_k = t + 1 < n_tiles ? kvq_page_load(p.c, seq, first_page + t + 1) : 0;
        if (t < n_tiles) {
          if (pg_k < 0) set_dev_status(status, kDevCapacity);
          if (!load(t, false, pg_k)) break;
          k_issued = t + 1;
        }
        if (t >= 1) {
          if (!load(t - 1, true, pg_v)) break;
          v_issued = t;
        }
        pg_v = pg_k;
      }
      // every issued copy has landed before this warp leaves
#pragma unroll 1
      for (int t = max(0, k_issued - kAStages); t < k_issued; ++t)
        warp_wait(&k_full[t % kAStages], (t / kAStages) & 1, status);
#pragma unroll 1
      for (int t = max(0, v_issued - kAStages); t < v_issued; ++t)
        warp_wait(&v_full[t % kAStages], (t / kAStages) & 1, status);
      __syncwarp();
    } else if (warp == 9) {
      // ---- MMA issuer: S two tiles ahead of O^T.  A commit covers all that was issued before: that
      // S(t) is done says that O^T(t - 2) is, and that Z(t) is full that S(t) is read.
      constexpr uint32_t id_s = idesc_e4m3_f32(64, kTile);
      const uint32_t id_o = idesc_f16_f32(128, 0) | ((uint32_t)(rows16 >> 3) << 17);
      const uint64_t q_desc = sw128_desc(smem_u32(sm)), z_desc = sw128_desc(smem_u32(sm + kAOffZ));
      const uint64_t k_desc = sw128_desc(smem_u32(sm + kAOffK));
      // (a descriptor's address field counts 16 bytes)
      const bool leader = elect_one();
      bool ok = __all_sync(0xffffffffu, warp_wait(q_full, 0, status));
      auto scores = [&](int t) {
        const int st = t % kAStages;
        ok = warp_wait(&k_full[st], (t / kAStages) & 1, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          const uint64_t kd = k_desc + st * (kTileBytes >> 4);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f8(tmem + (t & 1) * kSOdd, q_desc + part * (kQPart >> 4) + kk * 2, kd + kk * 2,
                        id_s, part + kk > 0 ? 1u : 0u);
          tc_commit(&s_full[t & 1]);
          tc_commit(&k_empty[st]);
        }
        __syncwarp();
      };
      if (ok) scores(0);
      if (ok && n_tiles > 1) scores(1);
#pragma unroll 1
      for (int t = 0; ok && t < n_tiles; ++t) {
        ok = warp_wait(o_ready, t & 1, status);
        if (ok) ok = warp_wait(&z_full[t & 1], (t >> 1) & 1, status);
        const uint64_t zd = z_desc + (t & 1) * (2 * kZBlock >> 4);
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // 64 slots each
          if (ok) ok = warp_wait(&vt_full[u], t & 1, status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 16 slots
              tc_mma_f16_ta(tmem + kTmemOCol, tmem + kTmemVCol + 32 * u + 8 * kk,
                            zd + u * (kZBlock >> 4) + kk * 2, id_o, t + u + kk > 0 ? 1u : 0u);
            tc_commit(&vt_empty[u]);
            if (u == 1 && t + 1 == n_tiles) tc_commit(o_done);
          }
          __syncwarp();
        }
        if (ok && t + 2 < n_tiles) scores(t + 2);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    regs_dec<kConvertRegs>();
    // ---- V to fp16 in tensor memory, exactly (NaN stays NaN), and O's rescaling.  This warp has
    // the dims 32 cw .. + 31, its lane quarter.  A transposing load gives a lane four
    // slots 4 (lane % 4) .. of dim lane / 4 (and + 8) of 16 x 16 codes; in fp16 they are
    // the two words that the 16x256b store takes from it.
    // V rows that are not seen must not hold NaN (0 * NaN): those behind the split's slots, or
    // on no page, are zeroed first; in rows that some query rows see and others do not,
    // NaN codes are zeroed and noted for the rows that see them: a bit for each of the warp's dims,
    // left over the slot's own codes, which are used by then.
    const int cw = warp - 4;
    const uint32_t lane_base = tmem + ((uint32_t)(cw * 32) << 16);
    // this lane's rows of the transposing loads: slots lane + 32 g, 16 dims
    const uint32_t v_at0 = smem_u32(sm + kAOffV) + lane * 128 + ((2 * cw ^ (lane & 7)) << 4);
    const uint32_t v_at1 = smem_u32(sm + kAOffV) + lane * 128 + (((2 * cw + 1) ^ (lane & 7)) << 4);
    bool ok = true;
    int marked = 0;  // tiles so far that not every row sees whole
    int raw = kvq_page_load(p.c, seq, first_page);
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      const int tile0 = k_begin + t * kTile, st = t % kAStages;
      const int stop = kvq_page_check(p.c, raw) < 0 ? tile0 : k_stop;
      if (t + 1 < n_tiles) raw = kvq_page_load(p.c, seq, first_page + t + 1);
      const bool partly = tile0 + kTile > min(stop, mask_from);
      ok = __all_sync(0xffffffffu, warp_wait(&v_full[st], (t / kAStages) & 1, status));
      if (!ok) break;
      uint32_t found[4] = {0u, 0u, 0u, 0u};
      if (partly) {
        clean_v(sm, st, cw, lane, stop - tile0, mask_from - tile0, found);
        if (found[0] | found[1] | found[2] | found[3]) nan_any[marked & 1] = 1;
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // 64 slots each
        // this half of O^T(t - 1) is done: its place is free
        if (ok && t > 0) ok = warp_wait(&vt_empty[u], (t - 1) & 1, status);
        if (u == 1) {
          // O holds tiles 0 .. t - 1 now: its columns (rows of q) times the factors by which the
          // maximum of this tile shrinks them, 16 columns for each softmax warp that has any
          if (ok) ok = warp_wait(&a_full[t & 1], (t >> 1) & 1, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          const float* const factor = reinterpret_cast<const float*>(sm + kAOffAlpha) + (t & 1) * 64;
          const int* const any = reinterpret_cast<const int*>(sm + kAOffGrown) + (t & 1) * 4;
          if (t > 0) {
            tc_fence_after();
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
              if (!any[w]) continue;
              float o[16];
              tmem_ld16(lane_base + kTmemOCol + 16 * w, o);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(factor + 16 * w + i);
                o[i] *= f.x;
                o[i + 1] *= f.y;
                o[i + 2] *= f.z;
                o[i + 3] *= f.w;
              }
              tmem_st16(lane_base + kTmemOCol + 16 * w, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(o_ready);
        }
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        uint32_t w[2][8];  // 16 dims each
        const uint32_t off = st * kTileBytes + u * (64 * 128);
        ldmatrix_b8_trans(v_at0 + off, &w[0][0]);
        ldmatrix_b8_trans(v_at0 + off + 32 * 128, &w[0][4]);
        ldmatrix_b8_trans(v_at1 + off, &w[1][0]);
        ldmatrix_b8_trans(v_at1 + off + 32 * 128, &w[1][4]);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t vt[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) codes_to_half(w[hh][i], vt[2 * i], vt[2 * i + 1]);
          tmem_st_16x256b_x4(lane_base + ((uint32_t)(16 * hh) << 16) + kTmemVCol + 32 * u, vt);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vt_full[u]);
      }
      if (!ok) break;
      if (partly) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint32_t*>(nan_bits(sm, st, lane + 32 * k, cw)) = found[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(nan_full);
        ok = __all_sync(0xffffffffu, warp_wait(nan_read, marked & 1, status));
        if (!ok) break;
        // (two flags, in turn: another of these warps may be a tile ahead, but not two)
        if (threadIdx.x == 128) nan_any[marked & 1] = 0;
        ++marked;
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&v_empty[st]);
    }
    __syncwarp();
  } else {
    regs_inc<kSoftmaxRegs>();
    // ---- softmax warps: half h of row t16's thread pair holds slots
    // 64 h .. 64 h + 63 of every tile (blocks 4 h .. 4 h + 3)
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint64_t* const anc =
        p.mask == DFLASH_MASK_TREE ? p.anc + (live ? grow : (long long)b * p.block + j0) * p.anc_words
                                   : nullptr;
    float* const q_scales = reinterpret_cast<float*>(sm + kAOffQs) + warp * 16;
    if (warp_live) convert_q(q_raw, warp, lane, sm, q_scales);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    const float q_signed = warp_live ? q_scales[t16] : 0.f;
    const float q_scale = fabsf(q_signed);
    __syncwarp();  // (the scales' place takes the factors of even tiles)
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    float m_used = -INFINITY, l = 0.f;
    uint32_t bad[4] = {0u, 0u, 0u, 0u};  // dims in which the row saw a NaN of V
    bool ok = true;
    // Page ids are read two tiles ahead, exponents one: from running pointers, few
    // instructions each (a warp spends about four cycles on every one of them).
    const int32_t* next_id = p.c.tab + (int64_t)seq * p.c.pps + first_page;
    const int8_t* const k_ex = p.c.ex[0] + kvh * kKvqSubs + 4 * h;
    const int8_t* const v_ex = p.c.ex[1] + kvh * kKvqSubs + 4 * h;
    const int page_ex = p.c.Hkv * kKvqSubs;  // exponents of a page
    auto exps_of = [&](int pg) -> uint2 {    // (of page 0 in place of an unmapped one)
      const int64_t at = (int64_t)max(pg, 0) * page_ex;
      return make_uint2(*reinterpret_cast<const uint32_t*>(k_ex + at),
                        *reinterpret_cast<const uint32_t*>(v_ex + at));
    };
    const uint32_t b_s_full = smem_u32(s_full), b_z_full = smem_u32(z_full);
    auto wait_for = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, warp_wait(bar, parity, status));
    };
    // this lane's 64 weights of a tile: a row of its block of Z
    uint8_t* const z_row = sm + kAOffZ + h * kZBlock + row * 128;
    int marked = 0;  // tiles so far that not every row sees whole
    int pg = kvq_page_check(p.c, *next_id++);
    int raw_next = n_tiles > 1 ? *next_id++ : -1;
    uint2 ex = exps_of(pg);
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      const int tile0 = k_begin + t * kTile;
      const int pg_now = pg;
      uint2 ex_now = ex;
      const uint32_t odd8 = (t & 1) * 8, phase = (t >> 1) & 1;
      if (t + 1 < n_tiles) {
        pg = kvq_page_check(p.c, raw_next);
        ex = exps_of(pg);
        if (t + 2 < n_tiles) raw_next = *next_id++;
      }
      const int stop = pg_now < 0 ? tile0 : k_stop;  // slots from here on are not seen
      const bool masked = tile0 + kTile > min(stop, mask_from);
      if (!(ok = wait_for(b_s_full + odd8, phase))) break;
      float s[64];
      if (warp_live) {
        tc_fence_after();
        const uint32_t s_base = lane_base + (t & 1) * kSOdd;
        tmem_ld_half32_nowait<64>(s_base, reinterpret_cast<uint32_t*>(s));
        tmem_ld_half32_nowait<64>(s_base + 32, reinterpret_cast<uint32_t*>(s) + 32);
        tmem_wait_ld();
        tc_fence_before();
      }
      float ck[4], ev[4], mx = -INFINITY;
      bool any_grown = false;
      if (warp_live) {
        if (masked) {
          // Blocks from `stop` on may never have been written, and an unmapped page has page
          // 0's exponents: any byte.  They count as 0, for -inf * 2^e is a NaN where 2^e
          // leaves fp32's range.
          const uint32_t written = bits_below((stop - tile0 - 64 * h + kKvqSub - 1) / kKvqSub * 8);
          ex_now.x &= written;
          ex_now.y &= written;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t vis = visible32(p, tile0 + 64 * h + 32 * c, stop, ctx, jr, anc);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * c + i] = (vis >> i) & 1u ? s[32 * c + i] : -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ck[i] = q_scale * pow2i((int)(int8_t)(ex_now.x >> (8 * i)));
          ev[i] = (float)(int)(int8_t)(ex_now.y >> (8 * i));
          float bm = s[16 * i];
#pragma unroll
          for (int k = 1; k < 15; k += 2) bm = fmaxf(fmaxf(bm, s[16 * i + k]), s[16 * i + k + 1]);
          bm = fmaxf(bm, s[16 * i + 15]);
          mx = fmaxf(mx, fmaf(bm, ck[i], ev[i]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const bool grown = mx > m_used + kLazyLog2;
        any_grown = __any_sync(0xffffffffu, grown);
        if (any_grown) {
          const float alpha = grown ? ex2(m_used - mx) : 1.f;
          if (h == 0) reinterpret_cast<float*>(sm + kAOffAlpha)[(t & 1) * 64 + row] = alpha;
          l *= alpha;
          if (grown) m_used = mx;
        }
      }
      // (the factors of two tiles ago are used: S of this tile was issued after their O^T)
      if (lane == 0) reinterpret_cast<int*>(sm + kAOffGrown)[(t & 1) * 4 + warp] = any_grown;
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[t & 1]);
      // (O^T(t - 2) is done, see the MMA issuer: this Z buffer is free)
      if (warp_live) {
        const float m = m_used == -INFINITY ? 0.f : m_used;
        float add[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) add[i] = ev[i] + (kTopLog2 - m);
        if (__any_sync(0xffffffffu, fabsf(m) > kFarLog2)) {
          // such an addend is off by more than z has room for: u (rounded as in the maximum, so
          // that the largest is the maximum) less the maximum, which is exact, first
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int k = 0; k < 16; ++k) s[16 * i + k] = fmaf(s[16 * i + k], ck[i], ev[i]) - m;
            ck[i] = 1.f;
            add[i] = kTopLog2;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t zh[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = 16 * i + 8 * w + 2 * k;
              const float2 x = fma2(make_float2(s[at], s[at + 1]), ck[i], add[i]);
              const float2 z = make_float2(ex2(x.x), ex2(x.y));
              sum = add2(sum, z);
              const __half2 z16 = __floats2half2_rn(z.x, z.y);
              zh[k] = *reinterpret_cast<const uint32_t*>(&z16);
            }
            *reinterpret_cast<uint4*>(z_row + (t & 1) * (2 * kZBlock) + (((2 * i + w) ^ (t16 & 7)) << 4)) =
                make_uint4(zh[0], zh[1], zh[2], zh[3]);
          }
          l = fmaf(sum.x + sum.y, pow2i(-(int)ev[i]), l);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(b_z_full + odd8);
      // a tile that some rows see and others do not: NaN of V, noted by the warps that convert it
      if (masked) {
        if (!(ok = wait_for(smem_u32(nan_full), marked & 1))) break;
        if (nan_any[marked++ & 1]) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t vis = visible32(p, tile0 + 64 * h + 32 * c, stop, ctx, jr, anc);
#pragma unroll 1
            while (vis) {
              const int at = 64 * h + 32 * c + __ffs(vis) - 1;
              vis &= vis - 1;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                bad[k] |= *reinterpret_cast<const uint32_t*>(nan_bits(sm, t % kAStages, at, k));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(nan_read);
      }
    }
    // ---- epilogue: lane d of warp w has dim 32 w + d of every row's O
    l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) bad[k] |= __shfl_xor_sync(0xffffffffu, bad[k], 16);
    if (ok) ok = wait_for(smem_u32(o_done), 0);
    if (ok) {
      tc_fence_after();
      // Through shared memory (Q and Z are done with): rows of dims, padded
#pragma unroll 1
      for (int c = 0; c < rows16; c += 16) {
        float o[16];
        tmem_ld16(lane_base + kTmemOCol + c, o);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          *reinterpret_cast<float*>(sm + (c + i) * kORow + (32 * warp + lane) * 4) = o[i];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      ok = wait_for(smem_u32(meet), 0);
    }
    if (ok && warp_live) {
      const bool none = l == 0.f;
      if (q_signed < 0.f && !none) l = __int_as_float(0x7fffffff);
      const bool whole = span.used == 1;
      const uint8_t* const stage = sm + warp * 16 * kORow;
      const long long rh = grow * p.H + hr;
      const long long part_row = (long long)split * p.batch * p.block * p.H + rh;
      const long long out_at = (whole ? rh : part_row) * kKvqHd;
      if (live && h == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + part_row * 2) = make_float2(m_used, l);
        else if (p.lse)
          p.lse[rh] = none ? -INFINITY : lse_of(m_used, l);
      }
      const float scale = none ? 0.f : (whole ? rcp(l) : 1.f);
      const bool any_bad = __any_sync(0xffffffffu, (bad[0] | bad[1] | bad[2] | bad[3]) != 0u);
      const int n_live = __popc(__ballot_sync(0xffffffffu, live) & 0xffffu);  // rows 0 .. n_live - 1
#pragma unroll 2
      for (int i = 0; i < n_live; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(stage + i * kORow + 16 * lane);
        const float sc = __shfl_sync(0xffffffffu, scale, i);
        const long long at = __shfl_sync(0xffffffffu, out_at, i) + 4 * lane;
        // (a row that saw nothing has sc = 0: zeros, not 0 * NaN)
        float4 v = make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
        if (sc == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (any_bad) {
          uint32_t nan = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t x4 = __shfl_sync(0xffffffffu, bad[k], i);
            if (k == lane >> 3) nan = x4 >> (4 * (lane & 7));
          }
          if (nan & 1u) v.x = __int_as_float(0x7fffffff);
          if (nan & 2u) v.y = __int_as_float(0x7fffffff);
          if (nan & 4u) v.z = __int_as_float(0x7fffffff);
          if (nan & 8u) v.w = __int_as_float(0x7fffffff);
        }
        if (whole) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
          uint2 w;
          w.x = *reinterpret_cast<const uint32_t*>(&lo);
          w.y = *reinterpret_cast<const uint32_t*>(&hi);
          *reinterpret_cast<uint2*>(p.out + at) = w;
        } else {
          *reinterpret_cast<float4*>(p.part_o + at) = v;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, kAttnQTmem);
}

// Merge of the splits of a row: one warp per (row, head), lane l holding dims
// 4 l .. 4 l + 3.  The used splits' (m, l) sit one a lane, their outputs are loaded sixteen
// at a time; sums run in split order.
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(32 * kMergeWarps) kvq_merge_kernel(const KvqAttnK p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  // (rows x heads of a launch are below 2^31)
  const int rh = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int64_t stride = (int64_t)p.batch * p.block * p.H;
  if (rh >= stride) return;
  const int row = rh / p.H, b = row / p.block, j = row - b * p.block;
  const float2* const ml = reinterpret_cast<const float2*>(p.part_ml) + rh;
  const float4* const po = reinterpret_cast<const float4*>(p.part_o + (int64_t)rh * kKvqHd) + lane;
  // the first splits are read before it is known how many are used (the
  // partials of all of them are in bounds)
  constexpr int kB = 16;
  float4 o[kB];
#pragma unroll
  for (int i = 0; i < kB; ++i)
    if (i < p.n_splits) o[i] = po[i * (stride * (kKvqHd / 4))];
  float2 x = lane < p.n_splits ? ml[lane * stride] : make_float2(-INFINITY, 0.f);
  int seq, n, r, key_end;
  if (!kvq_entry(p, b, seq, n, r, key_end) || j >= r) return;
  const int POS = p.pos;
  const KvqSpan span = kvq_span(p, n, r, key_end, min(j / POS * POS + POS, r));
  if (span.used <= 1) return;  // written whole
  // a split whose sum is zero saw nothing (its m is -inf)
  float m = lane < span.used && x.y != 0.f ? x.x : -INFINITY;
#pragma unroll 1
  for (int s = lane + 32; s < span.used; s += 32) {
    const float2 y = ml[s * stride];
    if (y.y != 0.f) m = fmaxf(m, y.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (m == -INFINITY) m = 0.f;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 0; s0 < span.used; s0 += kB) {
    if (s0 > 0) {
      if ((s0 & 31) == 0)
        x = s0 + lane < span.used ? ml[(s0 + lane) * stride] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < kB; ++i)
        if (s0 + i < span.used) o[i] = po[(s0 + i) * (stride * (kKvqHd / 4))];
    }
    const float w = x.y != 0.f ? ex2(x.x - m) : 0.f;
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      if (s0 + i >= span.used) break;
      const float wi = __shfl_sync(0xffffffffu, w, (s0 + i) & 31);
      l += wi * __shfl_sync(0xffffffffu, x.y, (s0 + i) & 31);
      acc.x += wi * o[i].x;
      acc.y += wi * o[i].y;
      acc.z += wi * o[i].z;
      acc.w += wi * o[i].w;
    }
  }
  const float inv = l == 0.f ? 0.f : rcp(l);
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 pk;
  pk.x = *reinterpret_cast<const uint32_t*>(&a);
  pk.y = *reinterpret_cast<const uint32_t*>(&c);
  *reinterpret_cast<uint2*>(p.out + (int64_t)rh * kKvqHd + lane * 4) = pk;
  if (p.lse && lane == 0) p.lse[rh] = l == 0.f ? -INFINITY : lse_of(m, l);
}

// Splits of a launch of `ctas` CTAs over max_keys slots: the count, as many as the
// workspace holds, that minimises the time of the fullest SM in units of a tile when
// two CTAs share the SM.  Such a pair takes 2 units a tile of each, a CTA alone 1.4; a CTA's
// set-up and output cost 6 beside its tiles; merging costs a unit for every 7200
// (row, head) outputs of a split.  (Measured at a batch of 8, 16,400 slots, 16 rows, 32 heads
// over 8: 1 to 9 splits 126, 73, 68, 57, 77, 77, 70, 67, 63 us, 4 taken; 1000 rows over about
// 4000 slots: 213 us unsplit, 261 with 2 splits; 32 sequences of one row over 32,769 slots: 304 to
// 326 us at 1 to 10 splits, 307 at 7, taken.)
constexpr int kKvqMaxSplits = 256;
static int kvq_plan_splits(int sm_count, int64_t ctas, int64_t max_keys, int64_t max_splits,
                           int64_t merge_rows) {
  const int64_t tiles = (max_keys + kTile - 1) / kTile;
  const int64_t top = std::min(std::min<int64_t>(kKvqMaxSplits, tiles), max_splits);
  int64_t best = 1;
  double best_cost = 0;
  for (int64_t sp = 1; sp <= top; ++sp) {
    const int64_t per = (tiles + sp - 1) / sp;
    if (sp > 1 && (tiles + per - 1) / per < sp) continue;  // some would be empty
    const int64_t on_sm = (ctas * sp + sm_count - 1) / sm_count;
    const double cost = (on_sm / 2) * (2.0 * per + 6) + (on_sm % 2) * (1.4 * per + 6) +
                        (sp > 1 ? sp * (merge_rows / 7200.0) + 1 : 0);
    if (sp == 1 || cost < best_cost) {
      best_cost = cost;
      best = sp;
    }
  }
  return (int)best;
}

static int64_t kvq_q_tiles(int block, int G) { return ((int64_t)block + 64 / G - 1) / (64 / G); }

// ---------------------------------------------------------------------------
// Accumulated weights.  The same product the other way round: S^T = K Q^T, a page of
// 128 slots as the M = 128 operand, 64 query rows (in their two e4m3 parts) as the
// other, so a thread owns a slot and sums the weights of its row of 64 scores
// without talking to another.  K alone is read, once: 128 bytes a slot and head.
//
// One CTA: a span of pages of one sequence and KV head, in groups of four; for each
// group all q tiles in turn (one, unless a pass has more than 64 rows a KV head), so
// the weights of a slot are summed in one register in a fixed order.
// Shared memory: K ring [4][128][128], Q [2 buffers][2 parts][64][128], the rows'
// (scale, log2 lse).  Tensor memory: four S^T tiles [128 slots][64 rows], one per
// page of the group; two CTAs share an SM.
// Warps 0-3: the rows' conversion (for the next q tile ahead of this one's sums),
// weights and sums; warp 4: TMA of K; warp 5: MMAs.
// Measured: 8 sequences of 16 rows x 32 heads over 16,400 slots (144 MB) 46 us, 3.1 TB/s: of
// a page's cycles in a CTA about 1050 are the weights (two pages at a time share the
// rows' scales), the rest waits and the group's set-up and output; two CTAs share an SM.
// ---------------------------------------------------------------------------
constexpr int kSGroup = 4;
constexpr uint32_t kSOffQ = kSGroup * kTileBytes;
constexpr uint32_t kSOffRow = kSOffQ + 2 * 2 * kQPart;   // [3][64] float2
constexpr uint32_t kSOffQs = kSOffRow + 3 * 64 * 8;      // [64] float, conversion scratch
constexpr uint32_t kSOffSlot = kSOffQs + 64 * 4;         // [4][128] float2: K's scale, the sum
constexpr uint32_t kSOffBar = kSOffSlot + kSGroup * kTile * 8;
constexpr int kScoreSmem = (int)kSOffBar + 256 + 1024;
constexpr uint32_t kSOffMute = kSOffBar + 192;  // [3][64] bits: rows with lse -inf
constexpr uint32_t kScoreTmem = 256;
constexpr int kScoreThreads = 192;

__global__ void __launch_bounds__(kScoreThreads, 2)
    kvq_score_kernel(const __grid_constant__ KvqMaps maps, const KvqAttnK p) {
  pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, kvh = blockIdx.y;
  int32_t* const status = p.c.status;
  const KvqEntry entry = kvq_entry_load(p, b);
  uint4 q_raw[8];
  if (warp < 4 && p.q_tiles == 1) load_q(p, b, kvh, 0, warp, lane, q_raw);

  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + kSOffBar);
  uint64_t* const q_full = bars;  // one for each Q buffer
  uint64_t* const k_full = bars + 2;
  uint64_t* const k_empty = k_full + kSGroup;
  uint64_t* const d_full = k_empty + kSGroup;
  uint64_t* const d_free = d_full + kSGroup;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(d_free + kSGroup);
  if (threadIdx.x == 0) {
    mbar_init(&q_full[0], 4);
    mbar_init(&q_full[1], 4);
    for (int i = 0; i < kSGroup; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], 4);
    }
    mbar_fence_init();
  }
  if (warp == 4) {
    tmem_alloc(tslot, kScoreTmem);
    tmem_relinquish();
  }
  int key_end;
  const bool work = kvq_entry_check(p, entry, key_end);
  const int seq = entry.seq, n = entry.n, r = entry.r, ctx = n - r;
  const int tiles = work ? (key_end + kTile - 1) / kTile : 0;
  const int per = max(1, (tiles + (int)gridDim.x - 1) / (int)gridDim.x);
  const int t_begin = blockIdx.x * per, t_end = min(tiles, t_begin + per);
  const int n_tiles = max(0, t_end - t_begin);
  // q tiles that can see a slot from `tile` on (causal: rows j >= slot - ctx)
  const int q_tiles = (r + p.pos - 1) / p.pos;
  auto q_first = [&](int tile) -> int {
    const int i = tile * kTile - ctx;  // block slot of the page's first one
    if (p.mask != DFLASH_MASK_CAUSAL || i <= 0) return 0;
    return min(i / p.pos, q_tiles);
  };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // every CTA holds its tensor memory (see kvq_attn_kernel)
  const uint32_t tmem = *tslot;

  if (n_tiles == 0) {
  } else if (warp == 4) {
    // ---- producer: page t of the span into stage t % 4
    const bool leader = elect_one();
    if (leader) tma_prefetch_desc(&maps.k);
    int issued = 0;
    int raw = kvq_page_load(p.c, seq, t_begin);
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      const int pg = kvq_page_check(p.c, raw);
      raw = t + 1 < n_tiles ? kvq_page_load(p.c, seq, t_begin + t + 1) : 0;
      const int st = t % kSGroup;
      if (t >= kSGroup &&
          !__all_sync(0xffffffffu, warp_wait(&k_empty[st], ((t / kSGroup) - 1) & 1, status)))
        break;
      if (pg < 0) set_dev_status(status, kDevCapacity);
      if (leader) {
        mbar_arrive_expect_tx(&k_full[st], kTileBytes);
        tma_load_2d(sm + st * kTileBytes, &maps.k, 0, (max(pg, 0) * p.c.Hkv + kvh) * kPageSlots,
                    &k_full[st]);
      }
      __syncwarp();
      issued = t + 1;
    }
#pragma unroll 1
    for (int t = max(0, issued - kSGroup); t < issued; ++t)
      warp_wait(&k_full[t % kSGroup], (t / kSGroup) & 1, status);
    __syncwarp();
  } else if (warp == 5) {
    // ---- MMA issuer
    const uint32_t cols = (uint32_t)min(p.block, p.pos) * p.G > 32 ? 64u : 32u;
    const uint32_t id = idesc_e4m3_f32(128, 0) | ((cols >> 3) << 17);
    const uint64_t k_desc = sw128_desc(smem_u32(sm)), q_desc = sw128_desc(smem_u32(sm + kSOffQ));
    const bool leader = elect_one();
    bool ok = true;
    int conv = 0;    // conversions used so far
    int rounds = 0;  // q tiles so far: writes of each S^T tile (only the last group is short)
#pragma unroll 1
    for (int g = 0; ok && g < n_tiles; g += kSGroup) {
      const int members = min(kSGroup, n_tiles - g);
      const int q0 = q_first(t_begin + g);
#pragma unroll 1
      for (int qt = q0; ok && qt < max(q_tiles, q0 + 1); ++qt) {
        // (a group no row sees still passes its pages through, with no q tile)
        const bool any = qt < q_tiles, last = qt + 1 >= q_tiles;
        if (any && (p.q_tiles > 1 || conv == 0)) {
          ok = __all_sync(0xffffffffu, warp_wait(&q_full[conv & 1], (conv >> 1) & 1, status));
          ++conv;
        }
        const int buf = p.q_tiles > 1 ? (conv - 1) & 1 : 0;
#pragma unroll 1
        for (int m = 0; ok && m < members; ++m) {
          if (qt == q0) ok = warp_wait(&k_full[m], (g / kSGroup) & 1, status);
          if (ok && any && rounds > 0) ok = warp_wait(&d_free[m], (rounds - 1) & 1, status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            if (any) {
              const uint64_t kd = k_desc + m * (kTileBytes >> 4);
              const uint64_t qd = q_desc + buf * 2 * (kQPart >> 4);
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_f8(tmem + m * 64, kd + kk * 2, qd + part * (kQPart >> 4) + kk * 2, id,
                            part + kk > 0 ? 1u : 0u);
              tc_commit(&d_full[m]);
            }
            if (last) tc_commit(&k_empty[m]);
          }
          __syncwarp();
        }
        if (any) ++rounds;
      }
    }
    __syncwarp();
  } else {
    // ---- weights: thread = slot of the page
    const int slot = warp * 32 + lane;
    float* const q_scales = reinterpret_cast<float*>(sm + kSOffQs) + warp * 16;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    bool ok = true;
    int conv = 0;
    // q tile qt into Q buffer conv % 2 (its MMAs of two tiles ago are done: this warp
    // has seen their results) and row buffer conv % 3 (a slower warp may still read
    // those of two tiles ago, but not older ones: it has converted the last tile)
    auto convert = [&](int qt) {
      const int buf = conv & 1, j0 = qt * p.pos;
      const int row = warp * 16 + (lane & 15), pos = row_pos(p, row), j = j0 + pos;
      const bool live = row < p.pos * p.G && j < r;
      float lse = 0.f;
      if (live)
        lse = p.lse[((long long)b * p.block + j) * p.H + kvh * p.G + row - pos * p.G];
      if (p.q_tiles > 1) load_q(p, b, kvh, j0, warp, lane, q_raw);
      // Rows behind the sequence's last one hold anything: as zeros, for an element that
      // becomes the code of NaN would be 0 * NaN in every slot's sum.
      if (j0 + p.pos > r) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j0 + row_pos(p, warp * 16 + 2 * i + (lane >> 4)) >= r) q_raw[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      convert_q(q_raw, warp, lane, sm + kSOffQ + buf * 2 * kQPart, q_scales);
      __syncwarp();
      if (lane < 16) {
        float2 v = make_float2(0.f, INFINITY);  // weight 2^-inf = 0
        if (live) {
          const float sc = q_scales[lane];
          v.x = fabsf(sc);
          v.y = sc < 0.f ? __int_as_float(0x7fffffff) : lse == -INFINITY ? INFINITY : lse * kLog2e;
        }
        reinterpret_cast<float2*>(sm + kSOffRow)[conv % 3 * 64 + row] = v;
      }
      // (such a row adds nothing, and its weights are 0 * NaN where K or it holds a NaN)
      const uint32_t mute = __ballot_sync(0xffffffffu, live && lse == -INFINITY) & 0xffffu;
      if (lane == 0)
        reinterpret_cast<uint16_t*>(sm + kSOffMute)[conv % 3 * 4 + warp] = (uint16_t)mute;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[buf]);
      ++conv;
    };
    // the thread's slot of each page of the group: K's scale and the sum so far
    float2* const mine = reinterpret_cast<float2*>(sm + kSOffSlot) + slot;
    const int chunks = min(p.block, p.pos) * p.G > 32 ? 2 : 1;  // of 32 rows
    const int64_t out_row = ((int64_t)seq * p.c.Hkv + kvh) * ((int64_t)p.c.pps * kPageSlots);
    // What a group's pages need is read ahead: the exponents and old scores of the
    // next group, the page ids of the one after that (the raw values, so that no
    // load is waited for before its group begins).
    int page[kSGroup], exps[kSGroup];
    float old[kSGroup];
    uint32_t mapped = 0;  // a bit for each page of the group just read
    const int32_t* const ids = p.c.tab + (int64_t)seq * p.c.pps + t_begin;
    const int8_t* const k_ex = p.c.ex[0] + kvh * kKvqSubs + slot / kKvqSub;
    const int page_ex = p.c.Hkv * kKvqSubs;
    const float* const in_row = p.score_in ? p.score_in + out_row + (int64_t)t_begin * kTile : nullptr;
    const int last_slot = key_end - 1 - t_begin * kTile;  // of the span's, from t_begin on
    auto read_pages = [&](int g) {
#pragma unroll
      for (int m = 0; m < kSGroup; ++m) page[m] = ids[min(g + m, n_tiles - 1)];
    };
    auto read_group = [&](int g) {  // (loads without conditions: nothing waits for them here)
      mapped = 0;
#pragma unroll
      for (int m = 0; m < kSGroup; ++m) {
        const int pg = kvq_page_check(p.c, page[m]);
        mapped |= (pg >= 0 ? 1u : 0u) << m;
        exps[m] = k_ex[(int64_t)max(pg, 0) * page_ex];
        old[m] = in_row ? in_row[min((g + m) * kTile + slot, last_slot)] : 0.f;
      }
    };
    // conversions run one q tile ahead: the next one is tile cq, for group cg
    int cg = 0, cq = q_first(t_begin);
    bool more = cq < q_tiles;
    // waits, once, for conversion c by all four warps (c in order).  Each buffer has a barrier
    // of its own, whose next phase begins only after this warp and the MMAs have used the
    // buffer: a phase's parity says nothing any more once the next one has completed.
    int known = 0;
    auto converted = [&](int c) -> bool {
      if (known > c) return true;
      known = c + 1;
      return __all_sync(0xffffffffu, warp_wait(&q_full[c & 1], (c >> 1) & 1, status));
    };
    read_pages(0);
    read_group(0);
    read_pages(kSGroup);
    int rounds = 0;
    int g = 0, qt = cq;
    float base[kSGroup];
#pragma unroll 1
    while (g < n_tiles) {
      const int members = min(kSGroup, n_tiles - g);
      const int q0 = q_first(t_begin + g);
      const int now = p.q_tiles > 1 ? rounds : 0;  // this q tile's conversion
#pragma unroll 1
      while (more && conv < now + 2) {
        // the rows' scales of all four warps: before a buffer is written again
        if (conv > now && !(ok = converted(now))) break;
        convert(cq++);
        if (p.q_tiles == 1) more = false;
        while (more && cq >= q_tiles) {
          cg += kSGroup;
          more = cg < n_tiles;
          cq = q_first(t_begin + cg);
        }
      }
      if (!ok) break;
      if (qt == q0) {
#pragma unroll
        for (int m = 0; m < kSGroup; ++m) {
          mine[m * kTile] = make_float2((mapped >> m) & 1u ? pow2i(exps[m]) : 0.f, 0.f);
          base[m] = in_row ? p.decay * old[m] : 0.f;
        }
        if (g + kSGroup < n_tiles) {
          read_group(g + kSGroup);
          read_pages(g + 2 * kSGroup);
        }
      }
      if (qt < q_tiles) {
        if (!(ok = converted(now))) break;
        const int rbuf = now % 3;
        const float4* const rows = reinterpret_cast<const float4*>(sm + kSOffRow) + rbuf * 32;
        const int j0 = qt * p.pos;
        // block slots from here on are not seen by every row of the q tile
        const int mask_from = p.mask == DFLASH_MASK_NONE     ? 0x7fffffff
                              : p.mask == DFLASH_MASK_CAUSAL ? ctx + j0 + 1
                                                             : ctx;
        // rows that count; where all do, or those that do not are behind the last row
        // (zeros, so their weights are zero too, and they see a NaN of K only beside a row that
        // counts), no bit is looked at
        const uint64_t mute = *reinterpret_cast<const uint64_t*>(sm + kSOffMute + rbuf * 8);
        const int n_rows = min(p.pos, r - j0) * p.G;
        const uint64_t count = mute == 0 ? ~0ull : ~mute & (n_rows < 64 ? (1ull << n_rows) - 1 : ~0ull);
        // two pages at a time: a row's (scale, log2 lse) is read once for both
#pragma unroll 1
        for (int m = 0; m < members; m += 2) {
          const int m1 = min(m + 1, members - 1);  // (a last page alone goes with itself)
          ok = __all_sync(0xffffffffu, warp_wait(&d_full[m], rounds & 1, status) &&
                                           warp_wait(&d_full[m1], rounds & 1, status));
          if (!ok) break;
          tc_fence_after();
          const float2 st0 = mine[m * kTile], st1 = mine[m1 * kTile];
          const int k0 = (t_begin + g + m) * kTile + slot, k1 = (t_begin + g + m1) * kTile + slot;
          const bool partly = (t_begin + g + m1 + 1) * kTile > mask_from;
          const bool masked = partly || mute != 0;
          uint64_t vis0 = count, vis1 = count;  // rows that see the slots
          if (partly) {
            if (k0 >= ctx) vis0 &= score_rows_seeing(p, b, k0 - ctx, j0, r);
            if (k1 >= ctx) vis1 &= score_rows_seeing(p, b, k1 - ctx, j0, r);
          }
          float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t s0[32], s1[32];
            tmem_ld32_nowait(lane_base + m * 64 + 32 * c, s0);
            tmem_ld32_nowait(lane_base + m1 * 64 + 32 * c, s1);
            tmem_wait_ld();
            const float4* const rc = rows + 16 * c;
            const uint32_t v0 = (uint32_t)(vis0 >> (32 * c)), v1 = (uint32_t)(vis1 >> (32 * c));
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float4 rw = rc[i / 2];
              const float2 x =
                  mul2(make_float2(__uint_as_float(s0[i]), __uint_as_float(s0[i + 1])), st0.x);
              const float2 y =
                  mul2(make_float2(__uint_as_float(s1[i]), __uint_as_float(s1[i + 1])), st1.x);
              float2 w = make_float2(ex2(fmaf(x.x, rw.x, -rw.y)), ex2(fmaf(x.y, rw.z, -rw.w)));
              float2 z = make_float2(ex2(fmaf(y.x, rw.x, -rw.y)), ex2(fmaf(y.y, rw.z, -rw.w)));
              if (masked) {
                w.x = (v0 >> i) & 1u ? w.x : 0.f;
                w.y = (v0 >> i) & 2u ? w.y : 0.f;
                z.x = (v1 >> i) & 1u ? z.x : 0.f;
                z.y = (v1 >> i) & 2u ? z.y : 0.f;
              }
              sum0 = add2(sum0, w);
              sum1 = add2(sum1, z);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&d_free[m]);
            if (m1 != m) mbar_arrive(&d_free[m1]);
          }
          mine[m * kTile].y = st0.y + (sum0.x + sum0.y);
          if (m1 != m) mine[m1 * kTile].y = st1.y + (sum1.x + sum1.y);
        }
        ++rounds;
      }
      if (!ok) break;
      if (++qt < q_tiles) continue;
      // the group's last q tile
#pragma unroll
      for (int m = 0; m < kSGroup; ++m) {
        const int k = (t_begin + g + m) * kTile + slot;
        if (m < members && k < key_end) {
          const float2 st = mine[m * kTile];  // (a slot on no page has scale 0)
          p.score_out[out_row + k] = st.x > 0.f ? base[m] + st.y : base[m];
        }
      }
      g += kSGroup;
      qt = q_first(t_begin + g);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) tmem_dealloc(tmem, kScoreTmem);
}

static bool kvq_attn_shape_ok(int batch, int H, int Hkv, int block, int max_keys) {
  return batch >= 1 && batch <= 65535 && H >= 1 && Hkv >= 1 && Hkv <= 65535 && H % Hkv == 0 &&
         H / Hkv <= 64 && block >= 1 && max_keys >= 1 && max_keys <= (1 << 29) &&
         (int64_t)batch * block < ((int64_t)1 << 31) &&
         (int64_t)batch * block * H < ((int64_t)1 << 31);
}

// fp32 partial outputs and (m, l) of one split
static int64_t kvq_part_bytes(int batch, int block, int H) {
  return (int64_t)batch * block * H * (kKvqHd + 2) * (int64_t)sizeof(float);
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
      q_row_stride >= ((int64_t)1 << 31) || !kvq_ints_aligned({seq_ids, kv_lens, q_lens}))
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
  p->pos = 64 / p->G;
  p->q_tiles = (int)kvq_q_tiles(block, p->G);
  p->g_inv = (65536 + p->G - 1) / p->G;
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
  const int64_t ctas = kvq_q_tiles(block, n_heads / n_kv_heads) * n_kv_heads * batch;
  const int splits = kvq_plan_splits(kvq_sms(), ctas, max_keys, 65535 / batch,
                                     (int64_t)batch * block * n_heads);
  return splits == 1 ? 0 : splits * kvq_part_bytes(batch, block, n_heads);
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
  const int64_t q_tiles = kvq_q_tiles(block, p.G), rh = (int64_t)batch * block * n_heads;
  const int64_t room = workspace ? workspace_bytes / kvq_part_bytes(batch, block, n_heads) : 0;
  p.n_splits = kvq_plan_splits(kvq_sms(), q_tiles * cache->n_kv_heads * batch, max_keys,
                               std::max<int64_t>(1, std::min<int64_t>(room, 65535 / batch)), rh);
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.part_o + p.n_splits * rh * kKvqHd;
  KvqMaps maps;
  const uint64_t kv_rows = (uint64_t)cache->n_pages * cache->n_kv_heads * kPageSlots;
  if (!encode_tmap_rows128(&maps.k, cache->k8_dev, kv_rows, kTile) ||
      !encode_tmap_rows128(&maps.v, cache->v8_dev, kv_rows, kTile))
    return DFLASH_E_CUDA;
  static std::atomic<bool> smem_done[kMaxDevices];
  if (ensure_smem_attr(smem_done, kvq_attn_kernel, kAttnQSmem) != cudaSuccess) return DFLASH_E_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)q_tiles, cache->n_kv_heads, batch * p.n_splits);
  if (launch_k(true, kvq_attn_kernel, grid, dim3(kAttnQThreads), kAttnQSmem, st, maps, p) !=
      cudaSuccess)
    return DFLASH_E_CUDA;
  if (p.n_splits > 1) {
    const dim3 mg((unsigned)((rh + kMergeWarps - 1) / kMergeWarps));
    if (launch_k(true, kvq_merge_kernel, mg, dim3(32 * kMergeWarps), 0, st, p) != cudaSuccess)
      return DFLASH_E_CUDA;
  }
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
  // spans of pages: as for the attention's splits, with nothing to merge
  const int splits = kvq_plan_splits(kvq_sms(), (int64_t)cache->n_kv_heads * batch, max_keys, 65535, 0);
  KvqMaps maps;
  const uint64_t kv_rows = (uint64_t)cache->n_pages * cache->n_kv_heads * kPageSlots;
  if (!encode_tmap_rows128(&maps.k, cache->k8_dev, kv_rows, kTile)) return DFLASH_E_CUDA;
  maps.v = maps.k;
  static std::atomic<bool> smem_done[kMaxDevices];
  if (ensure_smem_attr(smem_done, kvq_score_kernel, kScoreSmem) != cudaSuccess) return DFLASH_E_CUDA;
  const dim3 grid(splits, cache->n_kv_heads, batch);
  if (launch_k(true, kvq_score_kernel, grid, dim3(kScoreThreads), kScoreSmem, (cudaStream_t)stream,
               maps, p) != cudaSuccess)
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
