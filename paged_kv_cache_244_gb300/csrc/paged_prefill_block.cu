// Paged (chunked) prefill attention over block-scaled E4M3 caches, on the tcgen05 tensor cores.
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现", §2 Kernel层 (PagedAttention prefill kernel); "从零实现 LLM
// 推理引擎：深挖 vLLM 的六大核心优化", §3.1 and §3.3 Chunked Prefill; "nano-vllm：vLLM 极简实现与大模型推理
// 流程解析", §学习要点 (8-bit quantisation of the cache).
//
// The work is cut as in the bf16 prefill: CTA = (sequence, KV head, tile of floor(128 / G)
// queries), 128 matrix rows = (query, head) pairs, keys 64 at a time (four blocks), two CTAs per
// SM.  The codes enter the matrix products unscaled, and the scales k_b, v_b of key t's block act
// on the scores:
//   x_t = scale_log2 k_b (q . Kcode_t) + log2 v_b,   p_t = 2^(x_t - m),
//   O = sum p_t Vcode_t,   L = sum p_t / v_b,   out = O / L.
// Both sums carry 2^m, and v_b cancels in the second.  The shift m follows the largest
// contribution p_t lazily, from 7 below it (the largest p_t is 2^7 when the shift is set and at
// most 2^15 before it moves), so P fits f16 whatever the scales and tokens far below the largest
// are still normal f16 values.  Inside a block k_b and v_b are constants: the row maximum is taken
// per block on the raw products (k_b > 0) and then scaled, each exponent's argument stays one FMA,
// and L costs one FMA a block.
//
// K codes are the B operand as they lie in the cache (kind::f8f6f4).  A bf16 q has 8 significant
// bits and E4M3 four, so a row of q, scaled by a power of two to put its largest magnitude in
// [128, 256), is the sum of two E4M3 rows, q = hi + lo, exact for values of 2^-9 of that largest and
// more, within 2^-17 of it for smaller ones: S = hi K + lo K, two products of twice the f16
// rate, with no K tile to widen.  V codes widen exactly to f16 (P V in f16 keeps P's 11 bits).
//
// Warpgroups of a CTA (registers split with setmaxnreg):
//   0   softmax, one thread per row
//   1   warp 4 K tiles and warp 6 V tiles by TMA (one 2 KiB box a block), warp 5 the MMAs
//   2   converters: 128 threads widen a stage's V codes from the TMA's ring into the f16 operand
//       ring, 16 codes a load, in the MN-major layout that the MMA reads (two 64-dim halves a
//       block, 128-byte swizzle).  V rows past the context, and V of absent blocks, are written
//       as zeros; so is a NaN in a token that some of the tile's rows do not see (0 * NaN would
//       reach them), and the rows that do get it back when out is written.
// Tensor memory per CTA (256 columns): S_j in columns 64 (j & 1) .. + 63, O in 128-255; a row's
// P_j (64 f16, 32 columns) is written by its thread over the S_j it has read, and is the A operand
// of P V from there.  So S_{j+1} is computed while the softmax works on S_j, and S_{j+2}, which
// takes the columns of P_j, is issued behind P_j V_j.  Shared memory per CTA: q hi and lo (16 KiB
// each, the A operand of S; out leaves through the first), three 8 KiB K stages, two 8 KiB stages of
// V codes, two 16 KiB stages of f16 V, barriers, the scales of 8 stages: 106 KiB.  Every wait is
// bounded.
//
// What bounds it: the path of shared and tensor memory in an SM, 87% busy (ncu, 4 x 2048 tokens, 12 / 2
// heads: loads and stores 51.3% of its wavefronts, the tensor core's reads of A and B 18.1% each) with
// the tensor pipe 36% active.  A tile of 128 rows and 64 keys puts q hi and lo (32 KiB), K twice (16),
// f16 V (16), S out (32), P in (16), the codes of V in and f16 V out (24) and the TMA's writes (16) on
// it.  4 x 2048 tokens: 64.0-64.9 us, 0.41-0.42 of the measured bf16 peak; 16 chunks of 256 over 1792: 62.6-63.3 us
// (61.8-62.7 and 59.6-60.7 with S_{j+2} issued right behind P_j V_j, an order that nothing guarantees, and V's NaN left
// to reach earlier rows).  A
// first form that widened K too and gave each thread its own row of q and out to load and store: 87 us.
// Measured and left: S of two stages by one product of 128 keys (a q operand read half as often, but S
// no longer double: 71 us); two threads a row, 16 softmax warps on an SM (65 us); one lane waiting for its
// warp at barriers (92 us); eight warps preparing q (65 us); all of q asked for at once, or ahead of the
// set-up barrier (no change); pairs of CTAs on two SMs sharing B (M = 256: the path is then half idle, but
// a stage's eight products with N = 64 take as long as before and each hand-over crosses the cluster: 66).
//
// Few tiles over a long context: a tile's stages are split over a cluster of 2, 4 or 8 CTAs
// (template kSplit; CTA r of C takes stages nst r / C .. nst (r + 1) / C).  The CTAs exchange each
// row's (m, L) through distributed shared memory, scale their O to the common shift, and CTA r
// collects dims 128 r / C .. of every row from all of them, in rank order: no workspace, one launch,
// the same sums whatever the timing.  11 sequences of one new token after 10,812 cached, 28 / 4 heads:
// 50.9 us, 142.8 unsplit; 4 of 71 after 2342, 32 / 8 heads: 32.5-33.2.

#include <atomic>
#include <mutex>

#include <cuda.h>

#include "pa_device.cuh"
#include "pa_launch.h"
#include "umma_desc.h"

namespace pa {
namespace {

constexpr int kBpRows = 128;
constexpr int kBpKB = 4;                             // key blocks per stage
constexpr int kBpKeys = kBpKB * kBlockSize;          // 64
constexpr int kBpKRing = 3, kBpCRing = 2, kBpVRing = 2;   // stages of K codes, V codes, f16 V
constexpr int kBpTile = kBlockSize * 128;            // a block's codes, or 16 rows x 64 f16: 2 KiB
constexpr int kBpCodes = kBpKB * kBpTile;            // codes of K (or V) of a stage: 8 KiB
constexpr int kBpVStage = 2 * kBpCodes;              // f16 V of a stage: 16 KiB
constexpr int kBpCOff = kBpKRing * kBpCodes;
constexpr int kBpVOff = kBpCOff + kBpCRing * kBpCodes;
constexpr int kBpQOff = kBpVOff + kBpVRing * kBpVStage;
constexpr int kBpQBytes = kBpRows * kHeadDim;        // hi (or lo) codes of the rows: 16 KiB
constexpr int kBpHdrOff = kBpQOff + 2 * kBpQBytes;
constexpr int kBpHeader = 256;
constexpr int kBpFoldOff = kBpHdrOff + kBpHeader;    // a float per row
constexpr int kBpScaleOff = kBpFoldOff + kBpRows * 4;   // a float4 per block of the stage, stage j in slot j % 8
constexpr int kBpScaleSlots = 8;
constexpr int kBpMlOff = kBpScaleOff + kBpScaleSlots * kBpKB * 16;   // split: a row's (m, L)
constexpr int kBpNanOff = kBpMlOff + kBpRows * 8;    // a dim's first NaN in V (key of this CTA), and the first of all
constexpr int kBpSmem = kBpNanOff + (kHeadDim + 4) * 4 + 1024;   // + alignment of the first stage
static_assert(kBpRows * kHeadDim * 4 <= kBpHdrOff, "the partial rows of a split tile fit the stages");
static_assert(2 * (kBpSmem + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr int kBpThreads = 384;
// registers per thread at launch, and the split (their sums per warpgroup are equal)
constexpr int kBpRegsSoftmax = 128, kBpRegsIssue = 48, kBpRegsConvert = 64;
static_assert(kBpRegsSoftmax + kBpRegsIssue + kBpRegsConvert <= 3 * 80, "of the 80 a thread launched with");
// A tile's keys are split over 2, 4 or 8 CTAs as long as there are at most kSplitCtas CTAs (two per SM) and
// at least kMinSplitStages stages for each; not below kSplitFrom stages (the exchange costs what some five
// stages do).
// The stages are those of the host's bound.  16 sequences of 16 tokens over 1000, 12 / 2 heads: 13.6 us, 20.2
// with a bound of 131,072 (27.0 when a cluster's CTAs beyond what the sequence wants stood idle: the working
// ones then share fewer SMs).
constexpr int kSplitCtas = 304, kMinSplitStages = 3, kSplitFrom = 10;
constexpr uint32_t kBpTmemCols = 256, kBpSCols = 64, kBpOCol = 128;   // S (and P) at 0 and 64

// header (byte offsets): mbarriers, one per ring slot, then the TMEM address
constexpr int kKFull = 0;                            // K TMA -> MMA (S)
constexpr int kKFree = kKFull + 8 * kBpKRing;        // MMA (S done) -> K TMA
constexpr int kCFull = kKFree + 8 * kBpKRing;        // V TMA -> converters
constexpr int kCFree = kCFull + 8 * kBpCRing;        // converters (a warp each: 4) -> V TMA
constexpr int kVFull = kCFree + 8 * kBpCRing;        // converters (4) -> MMA (P V)
constexpr int kVFree = kVFull + 8 * kBpVRing;        // MMA (P V done) -> converters, MMA (S over P), softmax (O, when it rescales)
constexpr int kSFull = kVFree + 8 * kBpVRing;        // [2] MMA (S done) -> softmax
constexpr int kPFull = kSFull + 16;                  // [2] softmax (a warp each: 4) -> MMA
constexpr int kDone = kPFull + 16;                   // MMA: its last MMAs finished; its own arrival passes on the converters'
constexpr int kQReady = kDone + 8;                   // softmax (one thread, all rows in place) -> MMA
constexpr int kTmemAt = kQReady + 8;
static_assert(kTmemAt + 4 <= kBpHeader, "header");

// Timing jitter, a test hook (pa_set_timing_jitter): a role sleeps below max_ns at each of its stages.  A
// kernel variant (kJitter), taken while the hook is set, so that the ordinary one has nothing of it in its stages.
__constant__ uint32_t c_bp_jitter[2];
std::atomic<bool> jitter_on{false};

// Four bf16 values times `raise` (a power of two that keeps them below 256) as the sum of two E4M3
// values each: the codes of the nearest, and of what it leaves.  f16 holds the 8 significant bits
// of a value down to 2^-17, and the difference exactly.
__device__ __forceinline__ void split_e4m3(uint32_t w0, uint32_t w1, float raise, uint32_t& hi, uint32_t& lo) {
  uint16_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? w1 : w0;
    const uint32_t x = pack_f16x2(bf16lo(w) * raise, bf16hi(w) * raise);
    h[i] = e4m3x2_of_f16x2(x);
    l[i] = e4m3x2_of_f16x2(sub_f16x2(x, e4m3x2_to_f16x2(h[i])));
  }
  hi = h[0] | (static_cast<uint32_t>(h[1]) << 16);
  lo = l[0] | (static_cast<uint32_t>(l[1]) << 16);
}

// The top bit of each byte that is a NaN among four codes.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Zeros in the place of the NaN among 16 codes of V (dims d .. d + 15), `key` noted as the dim's first.
__device__ __forceinline__ void take_nans(uint32_t* codes, int* nan_from, int d, int key) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint32_t nan = e4m3_nans(codes[i]);
    if (nan == 0) continue;
    codes[i] &= ~((nan >> 7) * 0xffu);
#pragma unroll 1
    for (int u = 0; u < 4; ++u)
      if ((nan >> (8 * u)) & 0x80u) atomicMin(nan_from + d + 4 * i + u, key);
    atomicMin(nan_from + kHeadDim, key);
  }
}

template <bool kSplit, bool kJitter>
__global__ void __launch_bounds__(kBpThreads, 2)
prefill_block_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const PrefillArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads;
  const int G = a.num_q_heads / Hkv;
  const int Tq = kBpRows / G;
  const uint32_t per_g = 65536u / G + 1;              // x / G = x per_g >> 16 for x < 128, G <= 8
  auto over_g = [&](int x) { return static_cast<int>((static_cast<uint32_t>(x) * per_g) >> 16); };
  // Linear order of the CTAs (clusters, split): the same query tile of every (sequence, KV head), latest
  // tile first.
  const int rank = kSplit ? static_cast<int>(blockIdx.x) : 0;
  const int ranks = kSplit ? static_cast<int>(gridDim.x) : 1;      // 2, 4 or 8
  const int log_ranks = 31 - __clz(ranks);
  const unsigned long long pairs = kSplit ? gridDim.z : gridDim.y, tiles = kSplit ? gridDim.y : gridDim.x;
  const unsigned long long lin = kSplit ? blockIdx.z * tiles + blockIdx.y : blockIdx.y * tiles + blockIdx.x;
  const int sg = static_cast<int>(lin % pairs);
  const int tile = static_cast<int>(tiles) - 1 - static_cast<int>(lin / pairs);
  const int s = sg / Hkv;
  const int g = sg - s * Hkv;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  const int q0 = a.q_start[s];
  const int n = a.q_start[s + 1] - q0;
  const int ctx = a.context_lens[s];
  if (q0 < 0 || n < 0 || q0 + n > a.num_tokens || n > a.max_query_len || ctx < n || ctx > a.max_context_len) {
    if (threadIdx.x == 0 && tile == 0 && g == 0) raise_flag(a.status, PA_FLAG_CONTEXT_LEN_OOB);
    return;
  }
  const int i0 = tile * Tq;
  if (i0 >= n) return;
  const int rows_q = min(Tq, n - i0);
  const int pos0 = ctx - n + i0;
  const int nblocks_all = (pos0 + rows_q - 1) / kBlockSize + 1;
  const int nst_all = (nblocks_all + kBpKB - 1) / kBpKB;
  // This CTA's stages j0 .. j0 + nst - 1 and its blocks, numbered from its first.
  auto first_stage = [&](int k) { return (nst_all * k) >> log_ranks; };   // nst_all < 2^26
  const int j0 = kSplit ? first_stage(rank) : 0;
  const int nst = kSplit ? first_stage(rank + 1) - j0 : nst_all;
  const int block0 = kBpKB * j0;
  const int nblocks = min(kBpKB * nst, nblocks_all - block0);

  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t stages = (raw + 1023u) & ~1023u;
  const uint32_t hdr = stages + kBpHdrOff;
  unsigned char* const base = smem_raw + (stages - raw);
  unsigned char* const hdr_gen = smem_raw + (hdr - raw);

  // Lane k holds the id of block 32 w + k of the current window w, and the next window's.
  const int32_t* bt_row = a.block_tables + static_cast<size_t>(s) * a.max_blocks + block0;
  auto load_id = [&](int w) { const int b = 32 * w + lane; return b < nblocks ? bt_row[b] : -1; };
  auto in_pool = [&](int id) { return id >= 0 && id < a.num_blocks; };
  int ids = load_id(0), ids_next = load_id(1);
  auto next_window = [&](int j) {  // at the first stage of a window
    if (j > 0 && ((kBpKB * j) & 31) == 0) {
      ids = ids_next;
      ids_next = load_id((kBpKB * j) / 32 + 1);
      return true;
    }
    return false;
  };
  // the stage's block of lane & 3 is inside the tile's keys and the pool
  auto stage_mask = [&](int j) {
    const int id = __shfl_sync(kFullMask, ids, ((kBpKB * j) & 31) + (lane & (kBpKB - 1)));
    return static_cast<int>(__ballot_sync(kFullMask, in_pool(id)) & ((1u << kBpKB) - 1));
  };
  int* const nan_from = reinterpret_cast<int*>(base + kBpNanOff);
  const int key0 = kBpKeys * j0;                    // this CTA's first key
  if (threadIdx.x <= kHeadDim) nan_from[threadIdx.x] = 0x7fffffff;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBpKRing; ++i) {
      mbar_init(hdr + kKFull + 8 * i, 1);
      mbar_init(hdr + kKFree + 8 * i, 1);
    }
    for (int i = 0; i < kBpCRing; ++i) {
      mbar_init(hdr + kCFull + 8 * i, 1);
      mbar_init(hdr + kCFree + 8 * i, 4);
    }
    for (int i = 0; i < kBpVRing; ++i) {
      mbar_init(hdr + kVFull + 8 * i, 4);
      mbar_init(hdr + kVFree + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(hdr + kPFull + 8 * i, 4);
      mbar_init(hdr + kSFull + 8 * i, 1);
    }
    mbar_init(hdr + kDone, 2);
    mbar_init(hdr + kQReady, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(hdr + kTmemAt, kBpTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(hdr_gen + kTmemAt);

  if (warp >= 8) {
    // ---- converters of V -------------------------------------------------------------------
    regs_dec<kBpRegsConvert>();
    const int t = threadIdx.x - 256;                // 0..127
    const int c = t & 7;                            // 16-code chunk of a row: dims 16c .. 16c + 15
    const int r8 = t >> 3;                          // row 0..15 of a block
    const int half = c >> 2;
    const int valid_last = ctx - kBlockSize * ((ctx - 1) / kBlockSize);
    const int last_blk = (ctx - 1) / kBlockSize - block0;
    // the two f16 chunks of the 16 dims, in an order that keeps eight lanes' stores on distinct banks
    const int f0 = 2 * (c & 3) + half, f1 = 2 * (c & 3) + 1 - half;
    const uint32_t in_off = static_cast<uint32_t>(r8 * 128 + ((c ^ (r8 & 7)) << 4));
    const uint32_t out0 = static_cast<uint32_t>(r8 * 128 + ((f0 ^ (r8 & 7)) << 4));
    const uint32_t out1 = static_cast<uint32_t>(r8 * 128 + ((f1 ^ (r8 & 7)) << 4));
    auto widen = [&](const uint4& w, uint4& lo, uint4& hi) {
      e4m3x4_to_f16x2x2(w.x, lo.x, lo.y);
      e4m3x4_to_f16x2x2(w.y, lo.z, lo.w);
      e4m3x4_to_f16x2x2(w.z, hi.x, hi.y);
      e4m3x4_to_f16x2x2(w.w, hi.z, hi.w);
    };
    bool failed = false;
    for (int j = 0; j < nst; ++j) {
      const int cst = j % kBpCRing, vst = j % kBpVRing;
      if constexpr (kJitter) jitter_sleep(c_bp_jitter, warp, j);
      next_window(j);
      const int mask = stage_mask(j);
      // the codes have landed and (after the ring's first round) the f16 slot is free: the whole
      // warp goes on or gives up
      bool ok = mbar_wait_parked(hdr + kCFull + 8 * cst, (j / kBpCRing) & 1);
      if (ok && j >= kBpVRing) ok = mbar_wait_parked(hdr + kVFree + 8 * vst, ((j / kBpVRing) - 1) & 1);
      if (!__all_sync(kFullMask, ok)) {
        failed = true;
        break;
      }
      unsigned char* const codes = base + kBpCOff + cst * kBpCodes;
      unsigned char* const ops = base + kBpVOff + vst * kBpVStage;
      uint4 w[kBpKB];
      auto load_codes = [&] {
#pragma unroll
        for (int b = 0; b < kBpKB; ++b) {
          w[b] = *reinterpret_cast<const uint4*>(codes + b * kBpTile + in_off);
          const bool live = ((mask >> b) & 1) && (kBpKB * j + b != last_blk || r8 < valid_last);
          if (!live) w[b] = make_uint4(0u, 0u, 0u, 0u);
        }
      };
      load_codes();
      if (kBpKeys * (j + 1) > pos0 + 1 - key0) {    // keys that some rows do not see
        uint32_t nan = 0;
#pragma unroll
        for (int b = 0; b < kBpKB; ++b) nan |= e4m3_nans(w[b].x) | e4m3_nans(w[b].y) | e4m3_nans(w[b].z) | e4m3_nans(w[b].w);
        if (nan) {
#pragma unroll 1
          for (int b = 0; b < kBpKB; ++b) {
            const int key = kBpKeys * j + kBlockSize * b + r8;
            if (key0 + key > pos0 && key0 + key < ctx && ((mask >> b) & 1))
              take_nans(reinterpret_cast<uint32_t*>(codes + b * kBpTile + in_off), nan_from, kBlockSize * c, key);
          }
          load_codes();
        }
      }
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        uint4 lo, hi;
        widen(w[b], lo, hi);
        unsigned char* dst = ops + (2 * b + half) * kBpTile;
        *reinterpret_cast<uint4*>(dst + out0) = half ? hi : lo;
        *reinterpret_cast<uint4*>(dst + out1) = half ? lo : hi;
      }
      fence_proxy_async_smem();                     // before the tensor core reads them
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(hdr + kCFree + 8 * cst);
        mbar_arrive(hdr + kVFull + 8 * vst);
      }
    }
    if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
    if constexpr (kSplit) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else if (warp >= 4) {
    regs_dec<kBpRegsIssue>();
    if (warp == 4 || warp == 6) {
      // ---- TMA producers: warp 4 K, warp 6 V; lanes 0-3 the stage's blocks -------------------
      const bool is_k = warp == 4;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      if (lane == 0) prefetch_tensor_map(tm);
      const int ring = is_k ? kBpKRing : kBpCRing;
      const uint32_t full = hdr + (is_k ? kKFull : kCFull);
      const uint32_t free_ = hdr + (is_k ? kKFree : kCFree);
      const uint32_t slots = stages + (is_k ? 0 : kBpCOff);
      int st = 0;
      uint32_t ph = 1;                              // parity of the slot's previous release
      // K: the scales of the lane's block of the window and the next, as the softmax wants them --
      // K scale, lift of the exponent, weight in L, whether the block is there.  Stage
      // j's lanes write theirs to slot j % 8 before the stage's barrier: the softmax reads them
      // after S_j, and the slot is written again for stage j + 8, after S_{j+5}, which was issued
      // behind P_{j+3} V_{j+3}, so when the softmax had done with stage j.
      auto load_scales = [&](int id) {
        if (!is_k) return make_float4(0.f, 0.f, 0.f, 0.f);
        const bool there = in_pool(id);
        const float2 kv = there ? a.kv_scale[static_cast<size_t>(id) * Hkv + g] : make_float2(1.f, 1.f);
        return make_float4(kv.x, log2_of(kv.y), __frcp_rn(kv.y), there ? 1.f : 0.f);
      };
      float4 scales = load_scales(ids), scales_next = load_scales(ids_next);
      float4* const scale_slots = reinterpret_cast<float4*>(base + kBpScaleOff);
      int issued = 0;
      bool failed = false;
      for (int j = 0; j < nst; ++j) {
        if constexpr (kJitter) jitter_sleep(c_bp_jitter, warp, j);
        if (next_window(j)) {
          scales = scales_next;
          scales_next = load_scales(ids_next);
        }
        const int mask = stage_mask(j);
        const int blk = __shfl_sync(kFullMask, ids, ((kBpKB * j) & 31) + (lane & (kBpKB - 1)));
        bool ok = true;
        if (lane == 0 && j >= ring) ok = mbar_wait_parked(free_ + 8 * st, ph);
        if (!__shfl_sync(kFullMask, ok, 0)) {
          failed = true;
          break;
        }
        // The boxes first: they may land before the arrival that announces them (the phase cannot
        // complete without it), which for K waits for the blocks' scales.
        const uint32_t bar = full + 8 * st;
        if (lane < kBpKB && ((mask >> lane) & 1))
          tma_load_2d(slots + st * kBpCodes + lane * kBpTile, tm, 0, (blk * Hkv + g) * kBlockSize, bar);
        if (is_k) {
          const int b = lane - ((kBpKB * j) & 31);
          if (b >= 0 && b < kBpKB) scale_slots[(j % kBpScaleSlots) * kBpKB + b] = scales;
        }
        __syncwarp();
        if (lane == 0) {
          if (mask) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(mask)) * kBpTile);
          else mbar_arrive(bar);
        }
        if (is_k && lane < kBpKB && kBpKB * j + lane < nblocks && !((mask >> lane) & 1))
          raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
        issued = j + 1;
        if (++st == ring) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (lane == 0) {
        if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
        // let the copies still in flight land before the CTA exits
        for (int j = max(0, issued - ring); j < issued; ++j)
          mbar_wait_parked(full + 8 * (j % ring), (j / ring) & 1, 10000000ull);
      }
    } else if (warp == 5) {
      // ---- MMA issuer --------------------------------------------------------------------------
      const uint32_t id_s = umma_idesc_e4m3(kBpRows, kBpKeys);
      const uint32_t id_pv = umma_idesc_f16(kBpRows, kHeadDim, false, true);
      const uint64_t k_desc0 = umma_smem_desc(stages, 16, 1024);
      const uint64_t q_desc = umma_smem_desc(stages + kBpQOff, 16, 1024);
      const uint64_t v_desc0 = umma_smem_desc(stages + kBpVOff, kBpTile, 1024);
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(kFullMask, mbar_wait_parked(bar, parity));
      };
      // K_j, V_j are there.  A look at a barrier takes 100 to 150 cycles even when its phase is over, so K_{j+2}'s
      // comes while P_j V_j runs and V_{j+1}'s behind S_{j+2}, off the chain from P_j to S_{j+2} (4 x 2048 tokens and
      // 16 chunks of 256, on one GPU: 64.4 and 69.2 us with both before the wait for P_j, 63.5 and 63.9 so).
      auto k_there = [&](int j) { return wait_all(hdr + kKFull + 8 * (j % kBpKRing), (j / kBpKRing) & 1); };
      auto v_there = [&](int j) { return wait_all(hdr + kVFull + 8 * (j % kBpVRing), (j / kBpVRing) & 1); };
      // one lane: S_j = Q K_j^T (its columns hold P_{j-2}, which P V has read)
      auto issue_s = [&](int j) {
        const int st = j % kBpKRing;
        const uint64_t kd = k_desc0 + static_cast<uint64_t>((st * kBpCodes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)              // q hi, then q lo, over the four 32-dim steps of K
          umma_e4m3(tmem + kBpSCols * (j & 1), q_desc + static_cast<uint64_t>(((kk >> 2) * kBpQBytes + (kk & 3) * 32) >> 4),
                    kd + static_cast<uint64_t>(((kk & 3) * 32) >> 4), id_s, kk > 0);
        umma_commit(hdr + kSFull + 8 * (j & 1));
        umma_commit(hdr + kKFree + 8 * st);
      };
      bool failed = !wait_all(hdr + kQReady, 0);
      for (int j = 0; j < 2 && j < nst && !failed; ++j) {
        failed = !k_there(j);
        tc_fence_after();
        if (!failed && elect_one()) issue_s(j);
        __syncwarp();
      }
      if (nst > 0 && !failed) failed = !v_there(0);  // (a split tile may leave a CTA without stages)
      for (int j = 0; j < nst && !failed; ++j) {
        const int st = j % kBpVRing;
        if constexpr (kJitter) jitter_sleep(c_bp_jitter, warp, j);
        if (!wait_all(hdr + kPFull + 8 * (j & 1), (j >> 1) & 1)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint64_t vd = v_desc0 + static_cast<uint64_t>((st * kBpVStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kBpKB; ++i)
            umma_bf16_tmem_a(tmem + kBpOCol, tmem + kBpSCols * (j & 1) + 8 * i, vd + static_cast<uint64_t>((i * 2 * kBpTile) >> 4), id_pv, j > 0 || i > 0);
          umma_commit(hdr + kVFree + 8 * st);
        }
        __syncwarp();
        if (j + 1 == nst) break;
        if (j + 2 < nst) {
          // S_{j+2} is written over P_j: MMAs keep their order of issue only among those of one accumulator and
          // shape, so P_j V_j has to be done first (the slot's next phase is this warp's own P_{j+2} V_{j+2}).
          if (!k_there(j + 2) || !wait_all(hdr + kVFree + 8 * st, (j / kBpVRing) & 1)) {
            failed = true;
            break;
          }
          tc_fence_after();
          if (elect_one()) issue_s(j + 2);
          __syncwarp();
        }
        failed = !v_there(j + 1);
      }
      __syncwarp();
      if (elect_one()) umma_commit(hdr + kDone);    // a commit follows the MMAs of its own thread
      if (lane == 0) {
        if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
        mbar_arrive(hdr + kDone);
        mbar_wait_parked(hdr + kDone, 0);
      }
    }
    if constexpr (kSplit) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
    __syncwarp();
  } else {
    // ---- q into shared memory, then the softmax: thread = row r of the tile ---------------------
    regs_inc<kBpRegsSoftmax>();
    const int r = threadIdx.x;
    const int p_r = pos0 + over_g(r);
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // q comes in and out leaves 8 lanes a row, so that global memory sees whole 128-byte lines; a
    // 16-byte chunk c of row x of a 128-byte-wide buffer sits at c ^ (x % 8).
    unsigned char* const qbuf = base + kBpQOff;
    const int hr = r >> 3, hc = r & 7;              // rows hr + 16 k, chunk hc of the half
    auto global_row = [&](int x) {                  // matrix row x of q and out, -1 past the queries
      const int xi = over_g(x);
      return xi < rows_q ? (static_cast<long long>(q0 + i0 + xi) * a.num_q_heads + g * G + (x - xi * G)) * kHeadDim
                         : -1ll;
    };
    float* const folds = reinterpret_cast<float*>(base + kBpFoldOff);
    {
      // Rows hr + 16 k, their dims 8 hc .. + 7 and 64 + 8 hc .. + 7 in this thread.  The row's
      // largest magnitude (over its 8 lanes) gives the power of two that brings it to [128, 256);
      // an infinity or a NaN makes the row's scores NaN.
#pragma unroll
      for (int k4 = 0; k4 < 8; k4 += 4) {
        uint4 v[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const long long at = global_row(hr + 16 * (k4 + k));
          v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
          if (at >= 0) {
            v[k][0] = reinterpret_cast<const uint4*>(a.q + at)[hc];
            v[k][1] = reinterpret_cast<const uint4*>(a.q + at)[8 + hc];
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = hr + 16 * (k4 + k);
          uint32_t top = 0;
#pragma unroll
          for (int p = 0; p < 2; ++p)
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[k][p].x & 0x7fff7fffu, v[k][p].y & 0x7fff7fffu),
                                         __vmaxu2(v[k][p].z & 0x7fff7fffu, v[k][p].w & 0x7fff7fffu)));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, o));
          top = max(top & 0xffffu, top >> 16);
          // below 2^-119 not as far: multiples of 2^-133 become multiples of 2^-7, exact all the same
          const int e = min(7 + 127 - static_cast<int>(top >> 7), 126);
          const float raise = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          if (hc == 0)
            folds[x] = top >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                      : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint2 hi, lo;
            split_e4m3(v[k][p].x, v[k][p].y, raise, hi.x, lo.x);
            split_e4m3(v[k][p].z, v[k][p].w, raise, hi.y, lo.y);
            unsigned char* at = qbuf + x * 128 + (((4 * p + (hc >> 1)) ^ (x & 7)) << 4) + 8 * (hc & 1);
            *reinterpret_cast<uint2*>(at) = hi;
            *reinterpret_cast<uint2*>(at + kBpQBytes) = lo;
          }
        }
      }
      fence_proxy_async_smem();                     // before the tensor core reads them
      named_barrier(1, 128);                        // the rows and their factors are in place
      if (r == 0) mbar_arrive(hdr + kQReady);
    }
    const float row_fold = row_factor(folds[r]);    // scale_log2 q = row_fold (hi + lo)
    float m = -INFINITY, l = 0.f;
    bool failed = false;
    const float4* const scale_slots = reinterpret_cast<const float4*>(base + kBpScaleOff);
    for (int j = 0; j < nst; ++j) {
      if constexpr (kJitter) jitter_sleep(c_bp_jitter, warp, j);
      if (!__all_sync(kFullMask, mbar_wait_parked(hdr + kSFull + 8 * (j & 1), (j >> 1) & 1))) {
        failed = true;
        break;
      }
      tc_fence_after();
      const uint32_t sbuf = trow + kBpSCols * (j & 1);
      float sc[kBpKeys];
      {
        uint32_t s0[32], s1[32];
        tmem_ld32(sbuf, s0);
        tmem_ld32(sbuf + 32, s1);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          sc[c] = __uint_as_float(s0[c]);
          sc[32 + c] = __uint_as_float(s1[c]);
        }
      }
      float f[kBpKB], e[kBpKB], w[kBpKB];
      bool all_there = true;
      bool there[kBpKB];
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        const float4 v = scale_slots[(j % kBpScaleSlots) * kBpKB + b];
        f[b] = row_fold * v.x;
        e[b] = v.y;
        w[b] = v.z;
        there[b] = v.w != 0.f;
        all_there = all_there && there[b];
      }
      // causal mask and absent blocks -> -inf, exponents in two steps: only on a stage that needs it
      const bool far = fmaxf(fmax3(f[0], f[1], f[2]), f[3]) > kFarFactor;
      if (far || !all_there || kBpKeys * (j0 + j + 1) - 1 > pos0) {
        if (far) {
#pragma unroll
          for (int c = 0; c < kBpKeys; ++c) sc[c] = fmaf(sc[c], f[c / kBlockSize], e[c / kBlockSize]);
#pragma unroll
          for (int b = 0; b < kBpKB; ++b) {
            f[b] = 1.f;
            e[b] = 0.f;
          }
        }
        const int lim = p_r - kBpKeys * (j0 + j);
#pragma unroll
        for (int c = 0; c < kBpKeys; ++c)
          if (!there[c / kBlockSize] || c > lim) sc[c] = -INFINITY;
      }
      __syncwarp();                                 // rows differ in `far`; the tensor-memory accesses want the whole warp
      float mrow = -INFINITY;
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {             // 16 -> 6 -> 2 -> 1, then the block's scale
        const float* x = sc + kBlockSize * b;
        const float u0 = fmax3(x[0], x[1], x[2]), u1 = fmax3(x[3], x[4], x[5]), u2 = fmax3(x[6], x[7], x[8]);
        const float u3 = fmax3(x[9], x[10], x[11]), u4 = fmax3(x[12], x[13], x[14]);
        mrow = fmaxf(mrow, fmaf(fmax3(fmax3(u0, u1, u2), fmaxf(u3, u4), x[15]), f[b], e[b]));
      }
      const float mn = mrow - m > 15.f ? mrow - 7.f : m;
      const float sh = mn == -INFINITY ? 0.f : mn;
      const float alpha = (mn == m || m == -INFINITY) ? 1.f : ex2_ftz(m - sh);
      m = mn;
      uint32_t pw[kBpKeys / 2];
      l *= alpha;
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        const float es = e[b] - sh;
        const uint64_t f2 = pack_f32x2(f[b], f[b]), e2 = pack_f32x2(es, es);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < kBlockSize / 2; ++k) {
          const int c = kBlockSize * b + 2 * k;
          float x0, x1;
          unpack_f32x2(fma_f32x2(pack_f32x2(sc[c], sc[c + 1]), f2, e2), x0, x1);
          const float p0 = ex2_ftz(x0), p1 = ex2_ftz(x1);
          pw[c / 2] = pack_f16x2(p0, p1);
          sum[k & 1] = add_f32x2(sum[k & 1], pack_f32x2(p0, p1));
        }
        float s0, s1;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
        l = fmaf(s0 + s1, w[b], l);
      }
      tmem_st32(sbuf, pw);                          // P_j over S_j
      // O *= alpha where a row's shift moved (warp-collective), once P V of stage j - 1 is done
      if (j > 0 && __any_sync(kFullMask, alpha != 1.f)) {
        const int pj = j - 1;
        if (!__all_sync(kFullMask, mbar_wait_parked(hdr + kVFree + 8 * (pj % kBpVRing), (pj / kBpVRing) & 1))) {
          failed = true;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t ov[32];
          tmem_ld32(trow + kBpOCol + 32 * q4, ov);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
          tmem_st32(trow + kBpOCol + 32 * q4, ov);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(hdr + kPFull + 8 * (j & 1));
    }
    // A warp that gave up still takes part in the barriers below (its rows' values are undefined).
    const bool ok = !failed && __all_sync(kFullMask, mbar_wait_parked(hdr + kDone, 0));
    if (!ok && lane == 0) raise_flag(a.status, PA_FLAG_TIMEOUT);
    const int last_key = p_r - key0;
    const bool spoiled = nan_from[kHeadDim] <= last_key;   // the row sees a NaN that the converters took out of V
    if constexpr (kSplit) {
      // Every MMA of this CTA is done, so its stages are free; the others' partial rows come there.
      reinterpret_cast<float2*>(base + kBpMlOff)[r] = make_float2(m, l);
      tc_fence_before();
      cluster_sync();
      tc_fence_after();
      float top = m, total = 0.f;
      float2 ml[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ml[k] = k < ranks ? ld_cluster_f2(cluster_addr(stages + kBpMlOff + 8 * r, k)) : make_float2(-INFINITY, 0.f);
        top = fmaxf(top, ml[k].x);
      }
      const float sh = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int k = 0; k < 8; ++k) total = fmaf(ml[k].y, ml[k].x == -INFINITY ? 0.f : ex2_ftz(ml[k].x - sh), total);
      const float mine = m == -INFINITY ? 0.f : ex2_ftz(m - sh);
      const int dims = kHeadDim >> log_ranks;       // of a CTA: 64, 32 or 16
      // Partial rows: [source CTA][row][dims] floats; 16-byte chunk c of a row at c ^ turn, so that the
      // eight rows of a store or load instruction's phase lie on distinct banks.
      const int turn = ranks == 8 ? (r >> 1) & 3 : r & 7;
      const int xi = over_g(r);
      // warps without a query's row, and CTAs without stages, have nothing to send
#pragma unroll 1
      for (int q4 = nst > 0 && __any_sync(kFullMask, xi < rows_q) ? 0 : 4; q4 < 4; ++q4) {   // 32 dims of O at a time
        __syncwarp();                               // rows without a query skipped the stores below
        uint32_t ov[32];
        if (ok) {
          tmem_ld32(trow + kBpOCol + 32 * q4, ov);
          tmem_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const int dim = 32 * q4 + c, to = dim >> (7 - log_ranks);
          const bool any = m != -INFINITY;          // a row without keys in this CTA's stages has nothing in O
          float4 v;
          v.x = any ? __uint_as_float(ov[c]) * mine : 0.f;
          v.y = any ? __uint_as_float(ov[c + 1]) * mine : 0.f;
          v.z = any ? __uint_as_float(ov[c + 2]) * mine : 0.f;
          v.w = any ? __uint_as_float(ov[c + 3]) * mine : 0.f;
          const int at = (rank * kBpRows + r) * dims * 4 + ((((dim - to * dims) >> 2) ^ turn) << 4);
          if (xi < rows_q) st_cluster_f4(cluster_addr(stages + at, to), v);
        }
      }
      if (spoiled && xi < rows_q) {
#pragma unroll 1
        for (int dim = 0; dim < kHeadDim; ++dim) {
          if (nan_from[dim] > last_key) continue;
          const int to = dim >> (7 - log_ranks), d = dim - to * dims;
          st_cluster_f1(cluster_addr(stages + (rank * kBpRows + r) * dims * 4 + (((d >> 2) ^ turn) << 4) + 4 * (d & 3), to),
                        __uint_as_float(0x7fc00000u));
        }
      }
      folds[r] = total == 0.f ? 0.f : 1.f / total;  // read by the CTA's threads after the barrier
      cluster_sync();
    } else {
      tc_fence_after();
      // a row whose every key was skipped has l = 0: zeros
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        if (part) named_barrier(1, 128);            // the first half has been stored
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
          uint32_t ov[32];
          if (ok) {
            tmem_ld32(trow + kBpOCol + 64 * part + 32 * q2, ov);
            tmem_wait_ld();
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              o[u] = pack_bf16x2(__uint_as_float(ov[8 * k + 2 * u]) * inv, __uint_as_float(ov[8 * k + 2 * u + 1]) * inv);
            *reinterpret_cast<uint4*>(qbuf + r * 128 + (((4 * q2 + k) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        if (spoiled) {
#pragma unroll 1
          for (int d = 0; d < 64; ++d)
            if (nan_from[64 * part + d] <= last_key)
              *reinterpret_cast<uint16_t*>(qbuf + r * 128 + (((d >> 3) ^ (r & 7)) << 4) + 2 * (d & 7)) = 0x7fc0;
        }
        named_barrier(1, 128);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int x = hr + 16 * k;
          const long long at = global_row(x);
          if (at >= 0)
            reinterpret_cast<uint4*>(a.out + at)[8 * part + hc] =
                *reinterpret_cast<const uint4*>(qbuf + x * 128 + ((hc ^ (x & 7)) << 4));
        }
      }
    }
  }
  if constexpr (kSplit) {
    // This CTA's dims of every row: the sum over the CTAs that had stages, in rank order.
    const int dims = kHeadDim >> log_ranks, log_chunks = 5 - log_ranks, rows = rows_q * G;
    for (int u = threadIdx.x; u < rows << log_chunks; u += kBpThreads) {
      const int x = u >> log_chunks, c = u - (x << log_chunks), xi = over_g(x);
      const int turn = ranks == 8 ? (x >> 1) & 3 : x & 7;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < ranks; ++k) {
        if (first_stage(k + 1) == first_stage(k)) continue;
        const float4 v = *reinterpret_cast<const float4*>(base + (k * kBpRows + x) * dims * 4 + ((c ^ turn) << 4));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      const float inv = reinterpret_cast<const float*>(base + kBpFoldOff)[x];
      *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(q0 + i0 + xi) * a.num_q_heads + g * G + (x - xi * G)) * kHeadDim +
                                rank * dims + 4 * c) =
          make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kBpTmemCols);
  }
}

}  // namespace

cudaError_t set_prefill_block_jitter(const uint32_t (&hook)[2]) {
  jitter_on = hook[0] != 0;
  return cudaMemcpyToSymbol(c_bp_jitter, hook, sizeof hook);
}

cudaError_t launch_prefill_block(const PrefillArgs& a, cudaStream_t stream) {
  const int G = a.num_q_heads / a.num_kv_heads;
  if (G < 1 || G > 8) return cudaErrorInvalidValue;
  const int Tq = kBpRows / G;
  const long long rows = static_cast<long long>(a.num_blocks) * a.num_kv_heads * kBlockSize;
  CUtensorMap tm_k, tm_v;
  if (!cache_tensor_map(a.k_cache, rows, true, &tm_k) || !cache_tensor_map(a.v_cache, rows, true, &tm_v))
    return cudaErrorInvalidValue;
  {  // opt in to the shared-memory size once per device
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
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBpSmem);
        if (err == cudaSuccess)
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
      };
      opt_in(prefill_block_kernel<false, false>);
      opt_in(prefill_block_kernel<true, false>);
      opt_in(prefill_block_kernel<false, true>);
      opt_in(prefill_block_kernel<true, true>);
      if (err != cudaSuccess) return err;
      done[dev] = true;
    }
  }
  // Split the keys while the grid leaves SMs without a CTA and each part keeps kMinSplitStages stages.
  const long long tiles = (a.max_query_len - 1) / Tq + 1;
  const long long pairs = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  const int stages = (a.max_context_len - 1) / kBpKeys + 1;
  int ranks = 1;
  while (ranks < 8 && stages >= kSplitFrom && tiles * pairs * ranks * 2 <= kSplitCtas && stages >= 2 * ranks * kMinSplitStages) ranks *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ranks > 1 ? dim3(static_cast<unsigned>(ranks), static_cast<unsigned>(tiles), static_cast<unsigned>(pairs))
                          : dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(pairs));
  cfg.blockDim = dim3(static_cast<unsigned>(kBpThreads));
  cfg.dynamicSmemBytes = kBpSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  const bool jitter = jitter_on;
  auto kernel = ranks > 1 ? (jitter ? prefill_block_kernel<true, true> : prefill_block_kernel<true, false>)
                          : (jitter ? prefill_block_kernel<false, true> : prefill_block_kernel<false, false>);
  return cudaLaunchKernelEx(&cfg, kernel, tm_k, tm_v, a);
}

}  // namespace pa
