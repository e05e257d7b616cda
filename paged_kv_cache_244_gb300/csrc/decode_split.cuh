// How a decode launch is cut into pieces: shared by the decode kernels and the merge, which finds
// the pieces of a sequence from the same arithmetic.
#pragma once

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

// Per CTA in shared memory: the block-count prefix N_s (S + 1 ints), then per sequence the
// valid rows of its last block (1..16; one byte each).
__host__ __device__ inline int prefix_bytes(int num_seqs) {
  return (((num_seqs + 1) * 4 + 15) & ~15) + ((num_seqs + 15) & ~15);
}

// Job flags (low bits of a descriptor's flag word; valid tokens sit at bits 8-12, the KV head
// at bits 16-31).
constexpr uint32_t kFirst = 1u, kLast = 2u, kWhole = 4u, kHasData = 8u;
constexpr uint32_t kNew = 16u;   // fused step: the block holding the segment's new token
constexpr uint32_t kRope = 32u;  // fused step: the sequence's position has a cos/sin row
constexpr uint32_t kGap = 64u;   // the piece starts at a range boundary that is also a partition
                                 // boundary inside the segment: the slot before it is a gap
constexpr int kMinRangeBlocks = PA_DECODE_MIN_RANGE;

// Flattened-axis ranges: V = min(num_warps, ceil(T / kMinRangeBlocks)) equal ranges, range
// v = [floor(v T / V), floor((v+1) T / V)), none shorter than kMinRangeBlocks blocks unless T
// is, so that a small batch is not cut into one-block pieces that the merge must then gather.
// With V <= #warps of the grid, every warp has at most one range.
struct Ranges {
  long long T;
  int V;
  // below 2^20 blocks (V < 2^12) both products fit 32 bits, whose division is several times shorter
  __device__ __forceinline__ long long begin(int v) const {
    if (T < (1 << 20)) return static_cast<uint32_t>(v) * static_cast<uint32_t>(T) / static_cast<uint32_t>(V);
    return (static_cast<long long>(v) * T) / V;
  }
  __device__ __forceinline__ int owner(long long x) const {
    if (T < (1 << 20))
      return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(V) - 1) / static_cast<uint32_t>(T));
    return static_cast<int>(((x + 1) * V - 1) / T);
  }
};

__device__ __forceinline__ Ranges make_ranges(long long T, const DecodeArgs& a) {
  Ranges r;
  r.T = T;
  r.V = static_cast<int>(min(static_cast<long long>(a.num_warps), (T + kMinRangeBlocks - 1) / kMinRangeBlocks));
  return r;
}

// Partial slot of the piece of segment `seg` in range v and P-token partition `part` (0
// without partitions; max_parts = partitions of the longest segment, 1 without).  Along the
// job axis consecutive pieces differ in range, partition or segment, and each such step
// raises the slot by at least one, so slots are distinct and below V + (#segments) * max_parts.
// Within one segment a step raises it by exactly one, except where a range boundary is also a
// partition boundary: there it skips one slot, which the warp whose range starts there marks
// empty (shift -inf, sum 0).  So a segment's pieces, with those gaps, fill the slots from
// v_first + seg * max_parts to v_last + seg * max_parts + (its last partition), in axis order.
__device__ __forceinline__ long long piece_slot(int v, int seg, int part, int max_parts) {
  return static_cast<long long>(v) + static_cast<long long>(seg) * max_parts + part;
}

__device__ __forceinline__ int clamp_len(int len, int max_len) {
  return len < 0 ? 0 : (len > max_len ? max_len : len);
}

// Exclusive prefix N_s of per-sequence block counts, and the valid rows of each sequence's last
// block, by the whole CTA (of `threads` threads, kWarps warps at most); raises the flag of lengths out of range.
template <int kWarps>
__device__ __forceinline__ void build_prefix(const DecodeArgs& a, int* prefix, unsigned char* last_rows,
                                             const int threads = kWarps * 32) {
  const int S = a.num_seqs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int warp_sums[kWarps];
  const int per = S <= threads ? 1 : (S + threads - 1) / threads;
  const int lo = min(S, tid * per), hi = min(S, lo + per);
  int sum = 0;
  for (int s = lo; s < hi; ++s) {
    const int len = a.context_lens[s];
    if ((len < 0 || len > a.max_context_len) && blockIdx.x == 0)
      raise_flag(a.status, PA_FLAG_CONTEXT_LEN_OOB);
    sum += (clamp_len(len, a.max_context_len) + kBlockSize - 1) / kBlockSize;
  }
  int incl = sum;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int y = __shfl_up_sync(kFullMask, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  const int of_warp = lane < threads / 32 ? warp_sums[lane] : 0;
  int run = incl - sum + __reduce_add_sync(kFullMask, lane < warp ? of_warp : 0);
  for (int s = lo; s < hi; ++s) {
    prefix[s] = run;
    const int len = clamp_len(a.context_lens[s], a.max_context_len);
    run += (len + kBlockSize - 1) / kBlockSize;
    last_rows[s] = static_cast<unsigned char>(((len - 1) & (kBlockSize - 1)) + 1);  // unused if len == 0
  }
  const int total = __reduce_add_sync(kFullMask, of_warp);
  if (tid == 0) prefix[S] = total;
  __syncthreads();
}

}  // namespace pa
