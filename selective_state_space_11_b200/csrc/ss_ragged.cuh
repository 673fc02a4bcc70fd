// ss_ragged.cuh -- ragged sequences of a packed token axis, and their slots in
// a state cache, as the time-major operators see them (sm_100a).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ss_internal.h"

namespace ss {

// First and last + 1 token of sequence i.  Offsets come from device memory the
// host has not seen, so both are clamped into [0, tokens]: a bad offset can
// give a wrong answer but no access out of range.
__device__ __forceinline__ int seq_begin(const Ragged& r, int i) {
  return r.cu ? min(max(r.cu[i], 0), r.tokens) : i * r.seqlen;
}
__device__ __forceinline__ int seq_end(const Ragged& r, int i, int begin) {
  return r.cu ? min(max(r.cu[i + 1], begin), r.tokens) : begin + r.seqlen;
}

// Tiles of `tile` tokens that never straddle two sequences, without a prefix
// sum over the sequences: sequence i owns the tile numbers from
// floor(begin_i / tile) + i on.  Its ceil(len_i / tile) tiles (at least one,
// also when it is empty) fit before those of i + 1, so
// floor(tokens / tile) + nseq numbers are enough, and a number finds its sequence by bisection.
// Numbers behind a sequence's last tile give k >= its tile count, and those
// ahead of sequence 0's first tile, where the offsets start above 0, k < 0:
// the caller leaves both out.
__host__ __device__ __forceinline__ long long ragged_tiles(const Ragged& r, int tile) {
  return r.nseq > 0 ? (long long)r.tokens / tile + r.nseq : 0;
}
struct RaggedTile {
  int seq, k;      // sequence, tile within it (of no sequence: k < 0 or >= its tile count)
  int begin, end;  // the whole sequence's tokens
};
__device__ __forceinline__ RaggedTile ragged_tile(const Ragged& r, long long v, int tile) {
  int lo = 0, hi = r.nseq - 1;  // the last i with floor(begin_i / tile) + i <= v
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)(seq_begin(r, mid) / tile) + mid <= v) lo = mid;
    else hi = mid - 1;
  }
  RaggedTile t;
  t.seq = lo;
  t.begin = seq_begin(r, lo);
  t.end = seq_end(r, lo, t.begin);
  t.k = (int)(v - ((long long)(t.begin / tile) + lo));
  return t;
}

// Offsets that decrease or leave [0, tokens] set bit 3 of the device fault
// word; one block of a launch checks them for all.
__device__ __forceinline__ void check_offsets(const Ragged& r, unsigned* fault) {
  if (!r.cu) return;
  bool bad = false;
#pragma unroll 1
  for (int i = threadIdx.x; i <= r.nseq; i += blockDim.x) {
    const int c = r.cu[i];
    bad |= c < 0 || c > r.tokens || (i > 0 && c < r.cu[i - 1]);
  }
  if (bad) atomicOr(fault, 8u);
}

// The cache slot of sequence i, or -1 when the sequence is to be skipped: a
// negative slot (padding), or one that is out of range or that an earlier
// sequence of the call already has (two sequences would race on one state);
// the last two set bit 3 of the device fault word.  All threads of the block
// call it with the same i and get the same answer; it holds a block barrier.
__device__ __forceinline__ int claim_slot(const Slots& s, int i, unsigned* fault) {
  if (!s.index) return i;
  const int slot = s.index[i];
  bool bad = slot >= s.count;
  if (slot >= 0 && !bad)
#pragma unroll 1
    for (int j = threadIdx.x; j < i; j += blockDim.x) bad |= s.index[j] == slot;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(fault, 8u);
    return -1;
  }
  return slot < 0 ? -1 : slot;
}

// The same for the lanes of one warp.
__device__ __forceinline__ int claim_slot_warp(const Slots& s, int i, unsigned* fault) {
  if (!s.index) return i;
  const int slot = s.index[i];
  bool bad = slot >= s.count;
  if (slot >= 0 && !bad)
#pragma unroll 1
    for (int j = threadIdx.x & 31; j < i; j += 32) bad |= s.index[j] == slot;
  if (__any_sync(0xffffffffu, bad)) {
    if ((threadIdx.x & 31) == 0) atomicOr(fault, 8u);
    return -1;
  }
  return slot < 0 ? -1 : slot;
}

}  // namespace ss
