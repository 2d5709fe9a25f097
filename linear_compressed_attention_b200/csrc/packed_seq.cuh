// Sequences packed end to end in the rows of a tensor: lookup and bounds of a
// sequence from its device-side offsets. Offsets are never trusted: whatever
// they hold is clamped to the rows given, so that a bad value gives a wrong
// result and a status code, never an access outside.
#pragma once

#include "common.cuh"

namespace edit {

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// After a wait that gave up: time for the copies this block has under way, which
// must not land in the shared memory of a block after it.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 2000000ull) {
  }
}

struct SeqRows {
  int begin, len;
};

__device__ __forceinline__ SeqRows seq_rows(const int32_t* offsets, int s, int rows) {
  SeqRows r;
  r.begin = clamp_int(offsets[s], 0, rows);
  r.len = clamp_int(offsets[s + 1], r.begin, rows) - r.begin;
  return r;
}

// Row tiles of R rows that never straddle two sequences, numbered without a
// prefix sum over the sequences: sequence s owns the slots from
// offsets[s] / R + s up to the next sequence's first one, which are at least
// ceil(len / R) (some slots are empty). rows / R + nseq slots cover all.
// Returns the sequence of slot t, the same in all 32 lanes (which must all call).
__device__ __forceinline__ int seq_of_slot(const int32_t* offsets, int nseq, int rows, int R, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = nseq;  // the answer lies in lo .. lo + n - 1; slot(lo) <= t
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && clamp_int(offsets[i], 0, rows) / R + i <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// All threads of one block: EDIT_ERR_SHAPE in *status when the offsets are not
// non-decreasing within 0 .. rows, else EDIT_OK, of up to two offset arrays and
// one list of lengths (each length within its sequence's keys and max_len).
// The block writes the word whatever it was (a call resets it).
__device__ __forceinline__ void check_offsets(const int32_t* a, long rows_a, const int32_t* b, long rows_b,
                                              const int32_t* lens, int max_len, int nseq, int* status) {
  int bad = 0;
  for (int s = threadIdx.x; s < nseq; s += blockDim.x) {
    if (a[s] < 0 || a[s + 1] < a[s] || a[s + 1] > rows_a) bad = 1;
    if (b) {
      if (b[s] < 0 || b[s + 1] < b[s] || b[s + 1] > rows_b) bad = 1;
      const long cap = static_cast<long>(b[s + 1]) - b[s];
      const long n = lens ? lens[s] : cap;
      if (n < 0 || n > cap || n > max_len) bad = 1;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? EDIT_ERR_SHAPE : EDIT_OK;
}

}  // namespace edit
