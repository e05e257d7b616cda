// The metadata of one serving step, built on the GPU from request lengths (pa_plan_step).
//
// "从零实现 LLM 推理引擎：深挖 vLLM 的六大核心优化", §3.1 (block tables grown from a free list),
// §3.2 (append_slot) and §3.3 (the rows of a chunk).
//
// Two exclusive sums over the sequences say everything: start_s of their new rows and x_s of
// their new table entries (a sequence that is in error brings neither).  Entry x takes
// free_blocks[F - 1 - x]; s is granted when it needs no block or x_{s+1} <= F, so the granted
// entries are exactly x < `taken`.  Rows and entries are then written independently: a thread
// finds the sequence of its row (or entry) by binary search in the sums.
//
// Every CTA forms both sums for itself in shared memory (S <= 8192: at most 64 KiB read from
// L2) and writes its own slice of the sequences, entries and rows, so there is one launch and
// nothing to wait for between CTAs.  num_free is read by every CTA: where num_free_out is the
// same word, a grid of several CTAs leaves it to a second launch of one CTA.
//
// The longest chain of dependent loads and barriers bounds it: lengths, two sums over the CTA, search,
// free-list entry, store.  256 sequences of one token: 4.6 us replayed from a graph (an empty
// kernel: 1.9; 5.8 before the loads of a phase were asked for ahead of the sums).  8192 of one token: 10.0 us
// (26.3 when each thread read its share of the lengths from memory itself, in one CTA).  512 prompts
// of 548,920 rows, where 12 bytes a row are written: 6.6 us, of which the writing takes 1.0 at the copy rate.

#include <mutex>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 512;          // of a CTA
constexpr int kPlanRowsPerThread = 4;
// Rows that one CTA takes before another is launched.
constexpr int kPlanRowsPerCta = kPlanThreads * kPlanRowsPerThread;
// One CTA an SM: each forms the sums anew, so more of them repeat work and fewer leave the writing
// thin.  512 prompts, 548,920 rows, CTAs of 512 threads: 7.0 us with 152, 7.6 with 228, 8.5 with 304 and 608.
constexpr int kPlanMaxCtas = 152;
// A call of more rows than those hold takes CTAs of twice the threads; smaller ones stay at 512, whose sums are
// shorter: 548,864 rows 6.4 us (6.9 with 512), 2 M rows 15.1 (18.2), but 262,144 rows 6.1 (4.7), 256 rows 4.2 (3.9).
constexpr int kPlanManyThreads = 1024, kPlanManyRows = kPlanMaxCtas * kPlanRowsPerCta;
// Sequences of a CTA where the count is not in place (an in-place count of several CTAs is a launch more: 8192 sequences
// of one token 17.6 us in place, 11.3 not):
// 2048 sequences of one token 6.9 us (9.0 in one CTA), 8192: 10.0 (13.2).
constexpr int kPlanSeqsPerCta = 512;

// start [S + 1], x [S + 1] (int32), good [S] (bytes)
__host__ __device__ inline int plan_smem(int S) { return 2 * 4 * (S + 1) + S + 16; }

// Largest s with sums[s] <= v, for 0 <= v < sums[n].
__device__ __forceinline__ int plan_find(const int* sums, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Exclusive sum over the CTA's threads, `sums` a shared word per warp; *total receives the whole sum.
template <int kThreads>
__device__ __forceinline__ long long block_exclusive(long long v, long long* sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFullMask, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  // lane w takes warp w's sum: the warps before this one, and all of them
  long long upto = lane < kThreads / 32 ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < kThreads / 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFullMask, upto, d);
    if (lane >= d) upto += y;
  }
  *total = __shfl_sync(kFullMask, upto, kThreads / 32 - 1);
  const long long before = __shfl_sync(kFullMask, upto, warp == 0 ? 0 : warp - 1);
  return (warp == 0 ? 0 : before) + incl - v;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// count_only: only num_free_out is written (the second launch of an in-place count).
template <int kThreads, bool kCountOnly>
__global__ void __launch_bounds__(kThreads) plan_step_kernel(const PlanArgs a, const int write_count) {
  extern __shared__ int smem[];
  __shared__ long long row_sums[kThreads / 32], need_sums[kThreads / 32];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int S = a.num_seqs, T = a.num_tokens, tid = threadIdx.x;
  int* start = smem;             // [S + 1]
  int* x = smem + S + 1;         // [S + 1]
  unsigned char* good = reinterpret_cast<unsigned char*>(smem + 2 * (S + 1));
  const bool first_cta = blockIdx.x == 0;

  // ---- the two sums: each thread takes a contiguous share of the sequences ----------------
  // The lengths come through the arrays that the sums are formed in, whole lines at a time; shares are of odd
  // size, so that a warp's lanes meet distinct banks.  Everything that a later phase waits for is asked for
  // at once: the count, both lengths.
  int per = (S + kThreads - 1) / kThreads;
  if (per > 1) per |= 1;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  const long long table_tokens = static_cast<long long>(a.max_blocks) * kBlockSize;
  int F = a.num_free[0];
  for (int s = tid; s < S; s += kThreads) {
    start[s] = a.new_lens[s];
    x[s] = a.cached_lens[s];
  }
  if (per > 1) __syncthreads();
  long long rows = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = start[s];
    if (n > 0 && n <= T) rows += n;
  }
  long long all_rows;
  long long r = block_exclusive<kThreads>(rows, row_sums, &all_rows);
  // Needs: of the sequences whose lengths and rows are in order.  Each is at most max_blocks
  // < 2^27 blocks and there are at most 8192, so their sum is kept in 64 bits, and clamped
  // to 2^31 - 1 where it is stored (a free list holds at most kMaxFreeBlocks, so the order is unchanged).
  long long need_sum = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = start[s], c = x[s];
    const bool in_rows = n >= 0 && n <= T;
    start[s] = static_cast<int>(min(r, static_cast<long long>(T)));
    if (in_rows) r += n;
    const bool ok = in_rows && c >= 0 && static_cast<long long>(c) + n <= table_tokens && r <= T;
    good[s] = ok ? 1 : 0;
    if (!ok && first_cta && !kCountOnly) raise_flag(a.status, PA_FLAG_CONTEXT_LEN_OOB);
    x[s] = ok ? blocks_of(c + n) - blocks_of(c) : 0;
    need_sum += x[s];
  }
  long long all_need;
  long long e = block_exclusive<kThreads>(need_sum, need_sums, &all_need);
  constexpr long long kTop = 0x7fffffffll;
  for (int s = s0; s < s1; ++s) {
    const int need = x[s];
    x[s] = static_cast<int>(min(e, kTop));
    e += need;
  }
  const int total_rows = static_cast<int>(min(all_rows, static_cast<long long>(T)));
  if (tid == 0) {
    start[S] = total_rows;
    x[S] = static_cast<int>(min(all_need, kTop));
  }
  if (F < 0 || F > a.free_capacity) {
    if (first_cta && tid == 0 && !kCountOnly) raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
    F = F < 0 ? 0 : a.free_capacity;
  }
  __syncthreads();
  // taken = the largest x_{s} <= F: the sums do not fall, so it is found by binary search
  int taken;
  if (x[S] <= F) {
    taken = x[S];
  } else {
    taken = x[plan_find(x, S, F)];   // x[S] > F: largest s with x[s] <= F
  }
  if (write_count && first_cta && tid == 0) a.num_free_out[0] = F - taken;
  if (kCountOnly) return;

  // granted: x[s + 1] <= F, or nothing needed
  auto is_granted = [&](int s) { return good[s] && (x[s + 1] == x[s] || x[s + 1] <= F); };
  const int nb = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  const int gtid = b * kThreads + tid, gthreads = nb * kThreads;

  // In a call of one CTA each kind of output starts with warps of its own, so that their loads overlap.
  const int entry_tid = nb > 1 ? gtid : (tid + kThreads / 4) % kThreads;
  const int row_tid = nb > 1 ? gtid : (tid + kThreads / 2) % kThreads;
  for (int s = gtid; s <= S; s += gthreads) {
    a.q_start[s] = start[s];
    if (s == S) break;
    const bool g = is_granted(s);
    a.context_lens[s] = g ? a.cached_lens[s] + a.new_lens[s] : 0;
    a.granted[s] = g ? 1 : 0;
    if (!g && good[s]) raise_flag(a.status, PA_FLAG_POOL_EXHAUSTED);
  }
  // new table entries
  for (int k = entry_tid; k < taken; k += gthreads) {
    const int s = plan_find(x, S, k);
    int id = a.free_blocks[F - 1 - k];
    if (id < 0 || id >= a.num_blocks) {
      raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
      id = -1;
    }
    a.block_tables[static_cast<size_t>(s) * a.max_blocks + blocks_of(a.cached_lens[s]) + (k - x[s])] = id;
  }
  // rows: each thread takes groups of kPlanRowsPerThread neighbours
  const int groups = (T + kPlanRowsPerThread - 1) / kPlanRowsPerThread;
  for (int gidx = row_tid; gidx < groups; gidx += gthreads) {
    const int t0 = gidx * kPlanRowsPerThread;
    int s = t0 < total_rows ? plan_find(start, S, t0) : S;
    int pos[kPlanRowsPerThread];
    long long slot[kPlanRowsPerThread];
    int cur = -1, c = 0, old = 0, id = -1, id_block = -1;
    bool live = false;
#pragma unroll
    for (int i = 0; i < kPlanRowsPerThread; ++i) {
      const int t = t0 + i;
      pos[i] = 0;
      slot[i] = -1;
      if (t >= total_rows) continue;
      while (start[s + 1] <= t) ++s;   // sequences without rows are passed over
      if (s != cur) {
        cur = s;
        live = is_granted(s);
        c = a.cached_lens[s];
        old = blocks_of(c);
        id_block = -1;
      }
      if (!live) continue;
      const int p = c + (t - start[s]);
      const int j = p / kBlockSize;
      if (j != id_block) {
        id_block = j;
        id = j < old ? a.block_tables[static_cast<size_t>(s) * a.max_blocks + j]
                     : a.free_blocks[F - 1 - (x[s] + (j - old))];
        if (id < 0 || id >= a.num_blocks) {
          raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
          id = -1;
        }
      }
      pos[i] = p;
      slot[i] = id < 0 ? -1 : static_cast<long long>(id) * kBlockSize + (p % kBlockSize);
    }
    if (t0 + kPlanRowsPerThread <= T) {
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      longlong2* dst = reinterpret_cast<longlong2*>(a.slot_mapping + t0);
      dst[0] = make_longlong2(slot[0], slot[1]);
      dst[1] = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kPlanRowsPerThread; ++i) {
        if (t0 + i >= T) break;
        a.positions[t0 + i] = pos[i];
        a.slot_mapping[t0 + i] = slot[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_plan_step(const PlanArgs& a, cudaStream_t stream) {
  const int smem = plan_smem(a.num_seqs);
  {  // opt in to the largest size once per device (without it 48 KiB bound this and the kernel's own together)
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      auto opt_in = [&](auto kernel) {
        if (err == cudaSuccess)
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, plan_smem(kMaxDecodeSeqs));
      };
      opt_in(plan_step_kernel<kPlanThreads, false>);
      opt_in(plan_step_kernel<kPlanThreads, true>);
      opt_in(plan_step_kernel<kPlanManyThreads, false>);
      if (err != cudaSuccess) return err;
      done[dev] = true;
    }
  }
  long long ctas = (static_cast<long long>(a.num_tokens) + kPlanRowsPerCta - 1) / kPlanRowsPerCta;
  if (ctas < 1) ctas = 1;
  if (a.num_free != a.num_free_out) {
    const long long by_seqs = (a.num_seqs + kPlanSeqsPerCta - 1) / kPlanSeqsPerCta;
    if (ctas < by_seqs) ctas = by_seqs;
  }
  if (ctas > kPlanMaxCtas) ctas = kPlanMaxCtas;
  const bool later = a.num_free == a.num_free_out && ctas > 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  const bool many = a.num_tokens > kPlanManyRows;
  cfg.blockDim = dim3(many ? kPlanManyThreads : kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = many ? plan_step_kernel<kPlanManyThreads, false> : plan_step_kernel<kPlanThreads, false>;
  cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a, later ? 0 : 1);
  if (err != cudaSuccess || !later) return err;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  return cudaLaunchKernelEx(&cfg, plan_step_kernel<kPlanThreads, true>, a, 1);
}

}  // namespace pa
