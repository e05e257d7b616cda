// Paged (chunked) prefill attention over the 4-bit cache, on the tcgen05 tensor cores.
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现", §2 Kernel层 (PagedAttention prefill kernel); "从零实现 LLM
// 推理引擎：深挖 vLLM 的六大核心优化", §3.1 and §3.3 Chunked Prefill; "nano-vllm：vLLM 极简实现与大模型推理
// 流程解析", §学习要点 (4-bit quantisation of the cache).
//
// The work is cut as in the other prefill kernels: CTA = (sequence, KV head, tile of floor(128 / G)
// queries), 128 matrix rows = (query, head) pairs, keys 64 at a time (four blocks), two CTAs per SM, the
// keys of few tiles over a long context split over a cluster.  An element of the cache has at most eight
// significant bits, so K and V go into the matrix products as bf16, exactly as the cache holds them, and
// what remains is attention over bf16 operands: x = scale_log2 q . K, p = 2^(x - m), out = sum p V / sum p.
//
// Warpgroups of a CTA (registers split with setmaxnreg):
//   0   softmax, one thread per row
//   1   warp 4 the MMAs
//   2   converters: a warp takes one of the stage's four records from global memory into registers, a stage
//       ahead, and widens it into the K and V operands (two and a half integer and bf16 instructions a
//       pair).  V rows past the context and of absent blocks are zeros; so is a V row whose scale is NaN
//       (0 * NaN would reach queries that do not see its token), and the rows that do see it become NaN when
//       out is written.
// Tensor memory per CTA (256 columns): S_j in columns 64 (j & 1) .. + 63, O in 128-255; a row's P_j (64 bf16,
// 32 columns) is written by its thread over the S_j it has read, and is the A operand of P V from there.  P is bf16, and l
// adds it unrounded: both operands of an MMA have one type, and V's elements reach from 2^-40 to 2^44, past f16.  That costs
// up to 2^-8 of a weight where f16 (the decode, whose V is codes) costs 2^-11: 0.0021 - 0.0023 of the largest value
// against 64 bits, for 0.0016 - 0.0017.
// q goes in after a power of two for each row that brings its largest magnitude to [128, 256), so that no
// product leaves fp32's range whatever the magnitudes of q and of the scales.
// Shared memory per CTA: q (32 KiB, the A operand of S; out leaves through its first half), two 16 KiB stages
// each of K and V, barriers: 98 KiB.  Every wait is bounded.
//
// What bounds it: the SM's path of shared and tensor memory, as in the kernel over E4M3 caches, with bf16 operands and both
// of them written by the converters.  Of a tile's 64 keys (128 bytes a cycle): operands in 256 cycles, S out of tensor
// memory and P into it 384, q as A operand 256, K and V as B operands 256, rescaling and the ends of a tile the rest: some
// 1,275 of the 1,637 cycles that two CTAs of an SM take for one tile each.  4 prompts of 2048 tokens, 12 / 2 heads: 70.5
// us (52 GFLOP, 0.73 PFLOP/s); 16 chunks of 256 over 1792: 72.5 (75 on some GPUs); 8 chunks of 5 over 6000, 28 / 4 heads,
// split: 27.2.
// Registers loaded only when their stage begins 79.4 / 95.7 / 30.1; K and V by three warps each 80 - 103; records brought
// to L2 ahead 73 / 76 / 28; softmax warps without a row left out: no change.

#include <atomic>
#include <mutex>

#include "int4_cache.cuh"
#include "int4_launch.h"
#include "umma_desc.h"

namespace pa {
namespace {

constexpr int kIpRows = 128;
constexpr int kIpKB = 4;                             // key blocks per stage
constexpr int kIpKeys = kIpKB * kBlockSize;          // 64
constexpr int kIpRing = 2;                           // stages of K and of V
constexpr int kIpHalf = kIpKeys * 128;               // 64 keys x 64 dims of K: 8 KiB
constexpr int kIpTile = kBlockSize * 128;            // 16 tokens x 64 dims of V: 2 KiB
constexpr int kIpStage = 2 * kIpHalf;                // K (or V) of a stage: 16 KiB
constexpr int kIpVOff = kIpRing * kIpStage;
constexpr int kIpQOff = kIpVOff + kIpRing * kIpStage;
constexpr int kIpQBytes = kIpRows * 128;             // 64 dims of the rows: 16 KiB
constexpr int kIpHdrOff = kIpQOff + 2 * kIpQBytes;
constexpr int kIpHeader = 256;
constexpr int kIpFoldOff = kIpHdrOff + kIpHeader;    // a float per row
constexpr int kIpMlOff = kIpFoldOff + kIpRows * 4;   // split: a row's (m, L)
constexpr int kIpNanOff = kIpMlOff + kIpRows * 8;    // the first key of this CTA whose V is NaN
constexpr int kIpSmem = kIpNanOff + 16 + 1024;       // + alignment of the first stage
static_assert(kIpRows * kHeadDim * 4 <= kIpQOff, "the partial rows of a split tile fit the stages");
static_assert(2 * (kIpSmem + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr int kIpThreads = 384;
// registers per thread at launch, and the split (their sums per warpgroup are equal)
constexpr int kIpRegsSoftmax = 128, kIpRegsIssue = 40, kIpRegsConvert = 72;
static_assert(kIpRegsSoftmax + kIpRegsIssue + kIpRegsConvert <= 3 * 80, "of the 80 a thread launched with");
// A tile's keys are split over 2, 4 or 8 CTAs as long as there are at most kSplitCtas CTAs (two per SM) and
// at least kMinSplitStages stages for each; not below kSplitFrom stages.
constexpr int kSplitCtas = 304, kMinSplitStages = 3, kSplitFrom = 10;
constexpr uint32_t kIpTmemCols = 256, kIpSCols = 64, kIpOCol = 128;   // S (and P) at 0 and 64

// header (byte offsets): mbarriers, one per ring slot, then the TMEM address
constexpr int kKFull = 0;                            // converters (a warp each: 4) -> MMA (S)
constexpr int kKFree = kKFull + 8 * kIpRing;         // MMA (S done) -> converters
constexpr int kVFull = kKFree + 8 * kIpRing;         // converters (4) -> MMA (P V)
constexpr int kVFree = kVFull + 8 * kIpRing;         // MMA (P V done) -> converters, MMA (S over P), softmax (O, when it rescales)
constexpr int kSFull = kVFree + 8 * kIpRing;         // [2] MMA (S done) -> softmax
constexpr int kPFull = kSFull + 16;                  // [2] softmax (a warp each: 4) -> MMA
constexpr int kDone = kPFull + 16;                   // MMA: its last MMAs finished; its own arrival passes on the converters'
constexpr int kQReady = kDone + 8;                   // softmax (one thread, all rows in place) -> MMA
constexpr int kTmemAt = kQReady + 8;
static_assert(kTmemAt + 4 <= kIpHeader, "header");

// Timing jitter, a test hook (pa_set_timing_jitter): a role sleeps below max_ns at each of its stages.  A
// kernel variant (kJitter), taken while the hook is set, so that the ordinary one has nothing of it in its stages.
__constant__ uint32_t c_ip_jitter[2];
std::atomic<bool> jitter_on{false};

template <bool kSplit, bool kJitter>
__global__ void __launch_bounds__(kIpThreads, 2)
prefill_int4_kernel(const PrefillArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads;
  const int G = a.num_q_heads / Hkv;
  const int Tq = kIpRows / G;
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
  if (q0 < 0 || n < 0 || q0 > a.num_tokens - n || n > a.max_query_len || ctx < n || ctx > a.max_context_len) {
    if (threadIdx.x == 0 && tile == 0 && g == 0) raise_flag(a.status, PA_FLAG_CONTEXT_LEN_OOB);
    return;
  }
  const int i0 = tile * Tq;
  if (i0 >= n) return;
  const int rows_q = min(Tq, n - i0);
  const int pos0 = ctx - n + i0;
  const int nblocks_all = (pos0 + rows_q - 1) / kBlockSize + 1;
  const int nst_all = (nblocks_all + kIpKB - 1) / kIpKB;
  // This CTA's stages j0 .. j0 + nst - 1 and its blocks, numbered from its first.
  auto first_stage = [&](int k) { return (nst_all * k) >> log_ranks; };   // nst_all < 2^26
  const int j0 = kSplit ? first_stage(rank) : 0;
  const int nst = kSplit ? first_stage(rank + 1) - j0 : nst_all;
  const int block0 = kIpKB * j0;
  const int nblocks = min(kIpKB * nst, nblocks_all - block0);

  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t stages = (raw + 1023u) & ~1023u;
  const uint32_t hdr = stages + kIpHdrOff;
  unsigned char* const base = smem_raw + (stages - raw);
  unsigned char* const hdr_gen = smem_raw + (hdr - raw);

  // Lane k holds the id of block 32 w + k of the current window w, and the next window's.
  const int32_t* bt_row = a.block_tables + static_cast<size_t>(s) * a.max_blocks + block0;
  auto load_id = [&](int w) { const int b = 32 * w + lane; return b < nblocks ? bt_row[b] : -1; };
  auto in_pool = [&](int id) { return id >= 0 && id < a.num_blocks; };
  int ids = load_id(0), ids_next = load_id(1);
  auto next_window = [&](int j) {  // at the first stage of a window
    if (j > 0 && ((kIpKB * j) & 31) == 0) {
      ids = ids_next;
      ids_next = load_id((kIpKB * j) / 32 + 1);
      return true;
    }
    return false;
  };
  // the stage's block of lane & 3 is inside the tile's keys and the pool
  auto stage_mask = [&](int j) {
    const int id = __shfl_sync(kFullMask, ids, ((kIpKB * j) & 31) + (lane & (kIpKB - 1)));
    return static_cast<int>(__ballot_sync(kFullMask, in_pool(id)) & ((1u << kIpKB) - 1));
  };
  int* const nan_from = reinterpret_cast<int*>(base + kIpNanOff);   // the first key whose V is NaN
  const int key0 = kIpKeys * j0;                    // this CTA's first key
  if (threadIdx.x == 0) {
    *nan_from = 0x7fffffff;
    for (int i = 0; i < kIpRing; ++i) {
      mbar_init(hdr + kKFull + 8 * i, 4);
      mbar_init(hdr + kKFree + 8 * i, 1);
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
    tmem_alloc(hdr + kTmemAt, kIpTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(hdr_gen + kTmemAt);

  if (warp >= 8) {
    // ---- converters: warp 8 + b takes block b of each stage --------------------------------------
    regs_dec<kIpRegsConvert>();
    const int cw = warp - 8;
    const int r8 = lane & 7, i = lane >> 3;         // tokens r8 and r8 + 8, 16-byte unit i of their codes
    const uint8_t* const cache = reinterpret_cast<const uint8_t*>(a.k_cache);
    // A stage's codes and scale words are asked for as soon as those of the stage before are widened.  (A block that is
    // not there is read as the pool's first; its keys are masked and its V is written as zeros.)
    uint4 k[2], v[2];
    uint2 ks[2];
    uint32_t vs[2];
    auto record = [&](int id) { return cache + (static_cast<size_t>(in_pool(id) ? id : 0) * Hkv + g) * kInt4Record; };
    auto load_k = [&](const uint8_t* rec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        k[h] = *reinterpret_cast<const uint4*>(rec + 512 * h + 64 * r8 + 16 * i);
        ks[h] = *reinterpret_cast<const uint2*>(rec + kInt4KScales + 64 * h + 8 * r8);
      }
    };
    auto load_v = [&](const uint8_t* rec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[h] = *reinterpret_cast<const uint4*>(rec + kInt4VCodes + 512 * h + 64 * r8 + 16 * i);
        vs[h] = *reinterpret_cast<const uint16_t*>(rec + kInt4VScales + 16 * h + 2 * r8);
      }
    };
    const int vu = i ^ ((r8 >> 1) & 3);             // the unit of V's dims that lies at i (token r8 + 8 as r8)
    // byte offsets of this lane's 16-byte chunks in a 128-byte row of an operand, swizzled
    const uint32_t k_at = (kBlockSize * cw + r8) * 128, k_even = (i ^ r8) << 4, k_odd = ((4 + i) ^ r8) << 4;
    const uint32_t v_at = (2 * cw + (vu >> 1)) * kIpTile + r8 * 128, v_chunk = 4 * (vu & 1);
    int id = __shfl_sync(kFullMask, ids, cw);
    {
      const uint8_t* rec = record(id);
      load_k(rec);
      load_v(rec);
    }
    bool failed = false;
    for (int j = 0; j < nst; ++j) {
      const int st = j % kIpRing;
      if constexpr (kJitter) jitter_sleep(c_ip_jitter, warp, j);
      const bool there = in_pool(id);
      if (!there && kIpKB * j + cw < nblocks && lane == 0) raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
      const uint8_t* next = nullptr;
      if (j + 1 < nst) {
        next_window(j + 1);
        id = __shfl_sync(kFullMask, ids, ((kIpKB * (j + 1)) & 31) + cw);
        next = record(id);
      }
      if (j >= kIpRing && !__all_sync(kFullMask, mbar_wait_parked(hdr + kKFree + 8 * st, ((j / kIpRing) - 1) & 1))) {
        failed = true;
        break;
      }
      {
        unsigned char* const ops = base + st * kIpStage + k_at;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {             // dims 32c + 8i .. + 7: chunk 4c + i of the token's row
            const uint32_t code = c == 0 ? k[h].x : c == 1 ? k[h].y : c == 2 ? k[h].z : k[h].w;
            uint32_t s2, z2;
            int4_unpack_scale(c < 2 ? ks[h].x : ks[h].y, c & 1, s2, z2);
            *reinterpret_cast<uint4*>(ops + (c >> 1) * kIpHalf + 1024 * h + ((c & 1) ? k_odd : k_even)) = int4_elements(code, s2, z2);
          }
        }
      }
      if (next) load_k(next);
      fence_proxy_async_smem();                     // before the tensor core reads them
      __syncwarp();
      if (lane == 0) mbar_arrive(hdr + kKFull + 8 * st);
      if (j >= kIpRing && !__all_sync(kFullMask, mbar_wait_parked(hdr + kVFree + 8 * st, ((j / kIpRing) - 1) & 1))) {
        failed = true;
        break;
      }
      {
        unsigned char* const ops = base + kIpVOff + st * kIpStage + v_at;
        // tokens of this lane's block that the context has
        const int inside = there ? ctx - key0 - kIpKeys * j - kBlockSize * cw : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s2, z2;
          int4_unpack_scale(vs[h], 0, s2, z2);
          if (8 * h + r8 >= inside || vs[h] > 0x7f8fu) {   // past the context, absent, or a scale of NaN
            if (8 * h + r8 < inside) atomicMin(nan_from, kIpKeys * j + kBlockSize * cw + 8 * h + r8);
            s2 = 0u;                                // c - z is finite: zeros
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {             // dims 32 vu + 8c .. + 7: chunk 4 (vu & 1) + c of the half's row
            const uint32_t code = c == 0 ? v[h].x : c == 1 ? v[h].y : c == 2 ? v[h].z : v[h].w;
            *reinterpret_cast<uint4*>(ops + 1024 * h + (((v_chunk + c) ^ r8) << 4)) = int4_elements(code, s2, z2);
          }
        }
        __syncwarp();
      }
      if (next) load_v(next);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(hdr + kVFull + 8 * st);
    }
    if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
    if constexpr (kSplit) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else if (warp >= 4) {
    regs_dec<kIpRegsIssue>();
    if (warp == 4) {
      // ---- MMA issuer --------------------------------------------------------------------------
      const uint32_t id_s = umma_idesc_bf16(kIpRows, kIpKeys, false, false);
      const uint32_t id_pv = umma_idesc_bf16(kIpRows, kHeadDim, false, true);
      const uint64_t k_desc0 = umma_smem_desc(stages, 16, 1024);
      const uint64_t q_desc = umma_smem_desc(stages + kIpQOff, 16, 1024);
      const uint64_t v_desc0 = umma_smem_desc(stages + kIpVOff, kIpTile, 1024);
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(kFullMask, mbar_wait_parked(bar, parity));
      };
      // Looks at barriers come off the chain from P_j to S_{j+2}: K_{j+2}'s while P_j V_j runs, V_{j+1}'s behind S_{j+2}.
      auto k_there = [&](int j) { return wait_all(hdr + kKFull + 8 * (j % kIpRing), (j / kIpRing) & 1); };
      auto v_there = [&](int j) { return wait_all(hdr + kVFull + 8 * (j % kIpRing), (j / kIpRing) & 1); };
      // one lane: S_j = Q K_j^T (its columns hold P_{j-2}, which P V has read)
      auto issue_s = [&](int j) {
        const int st = j % kIpRing;
        const uint64_t kd = k_desc0 + static_cast<uint64_t>((st * kIpStage) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)              // 16 dims each, four in each half of 64
          umma_bf16(tmem + kIpSCols * (j & 1), q_desc + static_cast<uint64_t>(((kk >> 2) * kIpQBytes + (kk & 3) * 32) >> 4),
                    kd + static_cast<uint64_t>(((kk >> 2) * kIpHalf + (kk & 3) * 32) >> 4), id_s, kk > 0);
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
        const int st = j % kIpRing;
        if constexpr (kJitter) jitter_sleep(c_ip_jitter, warp, j);
        if (!wait_all(hdr + kPFull + 8 * (j & 1), (j >> 1) & 1)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint64_t vd = v_desc0 + static_cast<uint64_t>((st * kIpStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kIpKB; ++i)
            umma_bf16_tmem_a(tmem + kIpOCol, tmem + kIpSCols * (j & 1) + 8 * i, vd + static_cast<uint64_t>((i * 2 * kIpTile) >> 4), id_pv, j > 0 || i > 0);
          umma_commit(hdr + kVFree + 8 * st);
        }
        __syncwarp();
        if (j + 1 == nst) break;
        if (j + 2 < nst) {
          // S_{j+2} is written over P_j: MMAs keep their order of issue only among those of one accumulator and
          // shape, so P_j V_j has to be done first (the slot's next phase is this warp's own P_{j+2} V_{j+2}).
          if (!k_there(j + 2) || !wait_all(hdr + kVFree + 8 * st, (j / kIpRing) & 1)) {
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
    regs_inc<kIpRegsSoftmax>();
    const int r = threadIdx.x;
    const int p_r = pos0 + over_g(r);
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // q comes in and out leaves 8 lanes a row, so that global memory sees whole 128-byte lines; a
    // 16-byte chunk c of row x of a 128-byte-wide buffer sits at c ^ (x % 8).
    unsigned char* const qbuf = base + kIpQOff;
    const int hr = r >> 3, hc = r & 7;              // rows hr + 16 k, chunk hc of the half
    auto global_row = [&](int x) {                  // matrix row x of q and out, -1 past the queries
      const int xi = over_g(x);
      return xi < rows_q ? (static_cast<long long>(q0 + i0 + xi) * a.num_q_heads + g * G + (x - xi * G)) * kHeadDim
                         : -1ll;
    };
    float* const folds = reinterpret_cast<float*>(base + kIpFoldOff);
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
          for (int p = 0; p < 2; ++p) {             // exact: only the exponent changes
            auto raised = [&](uint32_t u) { return pack_bf16x2(bf16lo(u) * raise, bf16hi(u) * raise); };
            *reinterpret_cast<uint4*>(qbuf + p * kIpQBytes + x * 128 + ((hc ^ (x & 7)) << 4)) =
                make_uint4(raised(v[k][p].x), raised(v[k][p].y), raised(v[k][p].z), raised(v[k][p].w));
          }
        }
      }
      fence_proxy_async_smem();                     // before the tensor core reads them
      named_barrier(1, 128);                        // the rows and their factors are in place
      if (r == 0) mbar_arrive(hdr + kQReady);
    }
    const float row_fold = row_factor(folds[r]);    // scale_log2 q = row_fold times the row as it went in
    float m = -INFINITY, l = 0.f;
    bool failed = false;
    for (int j = 0; j < nst; ++j) {
      if constexpr (kJitter) jitter_sleep(c_ip_jitter, warp, j);
      next_window(j);
      const int mask = stage_mask(j);
      if (!__all_sync(kFullMask, mbar_wait_parked(hdr + kSFull + 8 * (j & 1), (j >> 1) & 1))) {
        failed = true;
        break;
      }
      tc_fence_after();
      const uint32_t sbuf = trow + kIpSCols * (j & 1);
      float sc[kIpKeys];
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
      // causal mask and absent blocks -> -inf: only on a stage that needs it
      if (mask != (1 << kIpKB) - 1 || kIpKeys * (j0 + j + 1) - 1 > pos0) {
        const int lim = p_r - kIpKeys * (j0 + j);
#pragma unroll
        for (int c = 0; c < kIpKeys; ++c)
          if (!((mask >> (c / kBlockSize)) & 1) || c > lim) sc[c] = -INFINITY;
      }
      float mrow = -INFINITY;
#pragma unroll
      for (int c = 0; c < kIpKeys; c += 16) {       // 16 -> 6 -> 2 -> 1
        const float* x = sc + c;
        const float u0 = fmax3(x[0], x[1], x[2]), u1 = fmax3(x[3], x[4], x[5]), u2 = fmax3(x[6], x[7], x[8]);
        const float u3 = fmax3(x[9], x[10], x[11]), u4 = fmax3(x[12], x[13], x[14]);
        mrow = fmax3(mrow, fmax3(u0, u1, u2), fmax3(u3, u4, x[15]));
      }
      // An exponent is one FMA of raw score, factor and shift, whose own rounding is left in it: half a step of the
      // score.  Where scores are so far out that this matters they are scaled first.
      float f = row_fold;
      const float bs = mrow * f;
      if (fabsf(bs) > 0x1p24f && mrow != -INFINITY) {
#pragma unroll
        for (int c = 0; c < kIpKeys; ++c) sc[c] *= f;
        f = 1.f;
      }
      __syncwarp();                                 // rows differ in it; the tensor-memory accesses want the whole warp
      // The shift moves to the row maximum only when that exceeds it by more than 8: P stays at most 2^8 and O is
      // rarely rescaled.
      const float mn = bs > m + 8.f ? bs : m;
      const float sh = mn == -INFINITY ? 0.f : mn;
      const float alpha = (mn == m || m == -INFINITY) ? 1.f : ex2_ftz(m - sh);
      m = mn;
      uint32_t pw[kIpKeys / 2];
      const uint64_t f2 = pack_f32x2(f, f), e2 = pack_f32x2(-sh, -sh);
      uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int k = 0; k < kIpKeys / 2; ++k) {
        float x0, x1;
        unpack_f32x2(fma_f32x2(pack_f32x2(sc[2 * k], sc[2 * k + 1]), f2, e2), x0, x1);
        const float p0 = ex2_ftz(x0), p1 = ex2_ftz(x1);
        pw[k] = pack_bf16x2(p0, p1);
        sum[k & 3] = add_f32x2(sum[k & 3], pack_f32x2(p0, p1));
      }
      {
        float s0, s1;
        unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), s0, s1);
        l = fmaf(l, alpha, s0 + s1);
      }
      tmem_st32(sbuf, pw);                          // P_j over S_j
      // O *= alpha where a row's shift moved (warp-collective), once P V of stage j - 1 is done
      if (j > 0 && __any_sync(kFullMask, alpha != 1.f)) {
        const int pj = j - 1;
        if (!__all_sync(kFullMask, mbar_wait_parked(hdr + kVFree + 8 * (pj % kIpRing), (pj / kIpRing) & 1))) {
          failed = true;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t ov[32];
          tmem_ld32(trow + kIpOCol + 32 * q4, ov);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
          tmem_st32(trow + kIpOCol + 32 * q4, ov);
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
    if (*nan_from <= last_key) l = __uint_as_float(0x7fc00000u);   // the row sees a V of NaN, which the converters left out
    if constexpr (kSplit) {
      // Every MMA of this CTA is done, so its stages are free; the others' partial rows come there.
      reinterpret_cast<float2*>(base + kIpMlOff)[r] = make_float2(m, l);
      tc_fence_before();
      cluster_sync();
      tc_fence_after();
      float top = m, total = 0.f;
      float2 ml[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ml[k] = k < ranks ? ld_cluster_f2(cluster_addr(stages + kIpMlOff + 8 * r, k)) : make_float2(-INFINITY, 0.f);
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
          tmem_ld32(trow + kIpOCol + 32 * q4, ov);
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
          const int at = (rank * kIpRows + r) * dims * 4 + ((((dim - to * dims) >> 2) ^ turn) << 4);
          if (xi < rows_q) st_cluster_f4(cluster_addr(stages + at, to), v);
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
            tmem_ld32(trow + kIpOCol + 64 * part + 32 * q2, ov);
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
    for (int u = threadIdx.x; u < rows << log_chunks; u += kIpThreads) {
      const int x = u >> log_chunks, c = u - (x << log_chunks), xi = over_g(x);
      const int turn = ranks == 8 ? (x >> 1) & 3 : x & 7;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < ranks; ++k) {
        if (first_stage(k + 1) == first_stage(k)) continue;
        const float4 v = *reinterpret_cast<const float4*>(base + (k * kIpRows + x) * dims * 4 + ((c ^ turn) << 4));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      const float inv = reinterpret_cast<const float*>(base + kIpFoldOff)[x];
      *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(q0 + i0 + xi) * a.num_q_heads + g * G + (x - xi * G)) * kHeadDim +
                                rank * dims + 4 * c) =
          make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kIpTmemCols);
  }
}

}  // namespace

cudaError_t set_prefill_int4_jitter(const uint32_t (&hook)[2]) {
  jitter_on = hook[0] != 0;
  return cudaMemcpyToSymbol(c_ip_jitter, hook, sizeof hook);
}

cudaError_t launch_prefill_int4(const PrefillArgs& a, cudaStream_t stream) {
  const int G = a.num_q_heads / a.num_kv_heads;
  if (G < 1 || G > 8) return cudaErrorInvalidValue;
  const int Tq = kIpRows / G;
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
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kIpSmem);
        if (err == cudaSuccess)
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
      };
      opt_in(prefill_int4_kernel<false, false>);
      opt_in(prefill_int4_kernel<true, false>);
      opt_in(prefill_int4_kernel<false, true>);
      opt_in(prefill_int4_kernel<true, true>);
      if (err != cudaSuccess) return err;
      done[dev] = true;
    }
  }
  // Split the keys while the grid leaves SMs without a CTA and each part keeps kMinSplitStages stages.
  const long long tiles = (a.max_query_len - 1) / Tq + 1;
  const long long pairs = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  const int stages = (a.max_context_len - 1) / kIpKeys + 1;
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
  cfg.blockDim = dim3(static_cast<unsigned>(kIpThreads));
  cfg.dynamicSmemBytes = kIpSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  const bool jitter = jitter_on;
  auto kernel = ranks > 1 ? (jitter ? prefill_int4_kernel<true, true> : prefill_int4_kernel<true, false>)
                          : (jitter ? prefill_int4_kernel<false, true> : prefill_int4_kernel<false, false>);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace pa
