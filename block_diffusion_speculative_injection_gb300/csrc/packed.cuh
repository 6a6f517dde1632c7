// Packed batches: sequence b's rows are offsets[b] .. offsets[b + 1] - 1 of one run of n_rows
// rows.  The lengths are known on the device only, so launches are sized from n_rows and
// batch, and a CTA or warp finds the sequence its work lies in.
#pragma once

#include "internal.cuh"

namespace dflash {

// Work units of `unit` rows (1..256): sequence b has the units from offsets[b] / unit + extra * b
// on, up to the next sequence's.  floor(x + y) >= floor(x) + floor(y), so that leaves it
// floor(rows / unit) + extra or more, and all of them lie below n_rows / unit + extra * batch.
struct PackedUnits {
  uint64_t magic;  // ceil(2^38 / unit): n * magic >> 38 is n / unit where n * magic < 2^64 (n up
                   // to 2^26 * unit), as n * (magic * unit - 2^38) < 2^38 then
  int extra;
};
inline PackedUnits packed_units_of(int unit, int extra) {
  return PackedUnits{((1ull << 38) + unit - 1) / unit, extra};
}
inline int64_t packed_units(int64_t n_rows, int64_t batch, int unit, int extra) {
  return n_rows / unit + extra * batch;
}

// First unit of sequence b (offsets out of range: any number)
__device__ __forceinline__ long long packed_base(const int32_t* offsets, int b, const PackedUnits& u) {
  return (long long)((uint64_t)(uint32_t)offsets[b] * u.magic >> 38) + (long long)u.extra * b;
}

// The sequence that unit `at` lies in (the last b with base <= at), or -1 before the first: a whole
// warp searches, 32 probes at a time, so a batch of up to 32 takes one load.
__device__ __forceinline__ int packed_find(const int32_t* offsets, int batch, const PackedUnits& u,
                                           long long at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, end = batch;
  while (true) {
    const int step = (end - lo + 31) / 32;
    const int probe = lo + lane * step;
    const bool below = probe < end && packed_base(offsets, probe, u) <= at;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    if (n == 0) return -1;
    lo += (n - 1) * step;
    // (in a list that is not in order, the last of n probes need not be one of those below)
    if (step == 1) return packed_base(offsets, lo, u) <= at ? lo : -1;
    end = min(end, lo + step);
  }
}

// Whether sequence b's rows lie in [0, n_rows) in order; its first row and count.
__device__ __forceinline__ bool packed_rows(const int32_t* offsets, int b, int n_rows, int& first,
                                            int& count) {
  first = offsets[b];
  const int end = offsets[b + 1];
  count = end - first;
  return first >= 0 && first <= end && end <= n_rows;
}

// Every thread of the launch looks at the entries i, i + all, ...: a list that is not in order,
// or leaves [0, n_rows], sets the status even where no unit falls into the bad entry.
__device__ __forceinline__ void packed_check(const int32_t* offsets, int batch, int n_rows,
                                             long long i, long long all, int32_t* status) {
  for (; i < batch; i += all) {
    int first, count;
    if (!packed_rows(offsets, (int)i, n_rows, first, count)) set_dev_status(status, kDevCheck);
  }
}

}  // namespace dflash
