// Paged (chunked) prefill attention over block-scaled E4M3 caches, on the tcgen05 tensor cores.
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现", §2 Kernel层 (PagedAttention prefill kernel); "从零实现 LLM
// 推理引擎：深挖 vLLM 的六大核心优化", §3.1 and §3.3 Chunked Prefill; "nano-vllm：vLLM 极简实现与大模型推理
// 流程解析", §学习要点 (8-bit quantisation of the cache).
//
// The work is cut as in the bf16 prefill: CTA = (sequence, KV head, tile of floor(128 / G)
// queries), 128 matrix rows = (query, head) pairs, keys 64 at a time (four blocks), two CTAs per
// SM.  E4M3 codes widen exactly to f16, so they enter the matrix products unscaled and the
// scales k_b, v_b of key t's block act on the scores:
//   x_t = scale_log2 k_b (q . Kcode_t) + log2 v_b,   p_t = 2^(x_t - m),
//   O = sum p_t Vcode_t,   L = sum p_t / v_b,   out = O / L.
// Both sums carry 2^m, and v_b cancels in the second.  The shift m follows the largest
// contribution p_t lazily, from 7 below it (the largest p_t is 2^7 when the shift is set and at
// most 2^15 before it moves), so P fits f16 whatever the scales and tokens far below the largest
// are still normal f16 values.
// Inside a block k_b and v_b are constants: the row maximum is taken per block on the raw
// products (k_b > 0) and then scaled, each exponent's argument stays one FMA, and L costs one FMA
// a block.
//
// Warpgroups of a CTA (registers split with setmaxnreg):
//   0   softmax, one thread per row
//   1   warp 4 K tiles and warp 6 V tiles by TMA (one 2 KiB box a block), warp 5 the MMAs
//   2   converters: 128 threads widen a stage's K codes, then its V codes, from the TMA's ring
//       into the f16 operand ring, 16 codes a load, in the layouts that the MMAs read (K-major
//       K as two 64-dim halves, MN-major V as two halves a block, 128-byte swizzle).  V rows past
//       the context, and V of absent blocks, are written as zeros.
// Tensor memory per CTA (256 columns): Q as f16 pairs 0-63, S 64-127, O 128-255.
// Shared memory per CTA (113 KB): two 32 KiB f16 stages, two 16 KiB code stages, the 16 KiB P
// buffer, barriers.  Every wait is bounded.

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
constexpr int kBpRing = 2;                           // stages of codes, and of f16 operands
constexpr int kBpHalf = kBlockSize * 128;            // 16 rows x 64 f16, and a block's codes: 2 KiB
constexpr int kBpCodes = kBpKB * kBpHalf;            // codes of K (or V) of a stage: 8 KiB
constexpr int kBpKHalf = kBpKB * kBpHalf;            // one f16 K half of a stage: 8 KiB
constexpr int kBpVOff = 2 * kBpKHalf;                // f16 V after the K halves
constexpr int kBpStage = 2 * kBpVOff;                // 32 KiB
constexpr int kBpCodeOff = kBpRing * kBpStage;       // code stages: [K | V]
constexpr int kBpCodeStage = 2 * kBpCodes;           // 16 KiB
constexpr int kBpPOff = kBpCodeOff + kBpRing * kBpCodeStage;
constexpr int kBpPBytes = kBpRows * kBpKeys * 2;     // 16 KiB
constexpr int kBpHdrOff = kBpPOff + kBpPBytes;
constexpr int kBpHeader = 256;
// As in the bf16 kernel: the header sits in the padding before the first 1024-byte boundary when
// it fits there, else after the P buffer; either way the layout ends within kBpSmem.
constexpr int kBpSmem = kBpHdrOff + kBpHeader + 768;
static_assert(2 * (kBpSmem + 1024) <= 228 * 1024, "two CTAs per SM");
static_assert(1008 + kBpHdrOff <= kBpSmem && kBpHeader - 1 + kBpHdrOff + kBpHeader <= kBpSmem, "layout");
constexpr int kBpThreads = 384;
// registers per thread at launch, and the split (their sums per warpgroup are equal)
constexpr int kBpRegsSoftmax = 120, kBpRegsIssue = 56, kBpRegsConvert = 64;
static_assert(kBpRegsSoftmax + kBpRegsIssue + kBpRegsConvert <= 3 * 80, "of the 80 a thread launched with");
constexpr uint32_t kBpTmemCols = 256, kBpQCol = 0, kBpSCol = 64, kBpOCol = 128;

// header (byte offsets)
constexpr int kCodesKFull = 0;     // [2] K TMA -> converters
constexpr int kCodesVFull = 16;    // [2] V TMA -> converters
constexpr int kCodesKFree = 32;    // [2] converters (128) -> K TMA
constexpr int kCodesVFree = 48;    // [2] converters (128) -> V TMA
constexpr int kKFull = 64;         // [2] converters (128) -> MMA (S)
constexpr int kVFull = 80;         // [2] converters (128) -> MMA (P V)
constexpr int kKFree = 96;         // [2] MMA (S done) -> converters
constexpr int kVFree = 112;        // [2] MMA (P V done) -> converters, softmax (P buffer, O)
constexpr int kSFull = 128;        // MMA (S done) -> softmax
constexpr int kSFree = 136;        // softmax (128) -> MMA
constexpr int kPFull = 144;        // [2] softmax (128) -> MMA
constexpr int kDone = 160;         // MMA: its last MMAs finished
constexpr int kQReady = 168;       // softmax (128) -> MMA
constexpr int kTmemAt = 176;
static_assert(kTmemAt + 4 <= kBpHeader, "header");

__global__ void __launch_bounds__(kBpThreads, 2)
prefill_block_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const PrefillArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads;
  const int G = a.num_q_heads / Hkv;
  const int Tq = kBpRows / G;
  // linear order of the CTAs: the same query tile of every (sequence, KV head), latest tile first
  const unsigned long long pairs = gridDim.y;
  const unsigned long long lin = static_cast<unsigned long long>(blockIdx.y) * gridDim.x + blockIdx.x;
  const int sg = static_cast<int>(lin % pairs);
  const int tile = static_cast<int>(gridDim.x) - 1 - static_cast<int>(lin / pairs);
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
  const int nblocks = (pos0 + rows_q - 1) / kBlockSize + 1;
  const int nst = (nblocks + kBpKB - 1) / kBpKB;

  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t stages = (raw + 1023u) & ~1023u;
  const uint32_t pad = stages - raw;
  const uint32_t hdr = pad >= static_cast<uint32_t>(kBpHeader) ? stages - kBpHeader : stages + kBpHdrOff;
  unsigned char* const base = smem_raw + pad;
  unsigned char* const hdr_gen = smem_raw + (hdr - raw);

  // Lane k holds the id of block 32 w + k of the current window w, and the next window's.
  const int32_t* bt_row = a.block_tables + static_cast<size_t>(s) * a.max_blocks;
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBpRing; ++i) {
      mbar_init(hdr + kCodesKFull + 8 * i, 1);
      mbar_init(hdr + kCodesVFull + 8 * i, 1);
      mbar_init(hdr + kCodesKFree + 8 * i, 128);
      mbar_init(hdr + kCodesVFree + 8 * i, 128);
      mbar_init(hdr + kKFull + 8 * i, 128);
      mbar_init(hdr + kVFull + 8 * i, 128);
      mbar_init(hdr + kKFree + 8 * i, 1);
      mbar_init(hdr + kVFree + 8 * i, 1);
      mbar_init(hdr + kPFull + 8 * i, 128);
    }
    mbar_init(hdr + kSFull, 1);
    mbar_init(hdr + kSFree, 128);
    mbar_init(hdr + kDone, 1);
    mbar_init(hdr + kQReady, 128);
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
    // ---- converters ------------------------------------------------------------------------
    regs_dec<kBpRegsConvert>();
    const int t = threadIdx.x - 256;                // 0..127
    const int c = t & 7;                            // 16-code chunk of a row: dims 16c .. 16c + 15
    const int r8 = t >> 3;                          // row 0..15 of a block
    const int half = c >> 2;
    const int valid_last = ctx - kBlockSize * ((ctx - 1) / kBlockSize);
    const int last_blk = (ctx - 1) / kBlockSize;
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
    // the codes have landed and (after the ring's first round) their operand slot is free: the
    // whole warp goes on or gives up
    auto wait_both = [&](uint32_t full, uint32_t slot_free, uint32_t ph, bool used) {
      bool ok = mbar_wait_bounded(full, ph);
      if (ok && used) ok = mbar_wait_bounded(slot_free, ph ^ 1u);
      return __all_sync(kFullMask, ok) != 0;
    };
    bool failed = false;
    for (int j = 0; j < nst; ++j) {
      const int st = j % kBpRing;
      const uint32_t ph = (j / kBpRing) & 1;
      next_window(j);
      const int mask = stage_mask(j);
      // K: rows of absent blocks keep what the slot held (their scores are masked)
      if (!wait_both(hdr + kCodesKFull + 8 * st, hdr + kKFree + 8 * st, ph, j >= kBpRing)) {
        failed = true;
        break;
      }
      unsigned char* const codes = base + kBpCodeOff + st * kBpCodeStage;
      unsigned char* const ops = base + st * kBpStage;
      uint4 w[kBpKB];
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) w[b] = *reinterpret_cast<const uint4*>(codes + b * kBpHalf + in_off);
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        uint4 lo, hi;
        widen(w[b], lo, hi);
        unsigned char* dst = ops + half * kBpKHalf + b * kBpHalf;
        *reinterpret_cast<uint4*>(dst + out0) = half ? hi : lo;
        *reinterpret_cast<uint4*>(dst + out1) = half ? lo : hi;
      }
      mbar_arrive(hdr + kCodesKFree + 8 * st);
      fence_proxy_async_smem();                     // before the tensor core reads them
      mbar_arrive(hdr + kKFull + 8 * st);
      // V: zeros for absent blocks and rows past the context
      if (!wait_both(hdr + kCodesVFull + 8 * st, hdr + kVFree + 8 * st, ph, j >= kBpRing)) {
        failed = true;
        break;
      }
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        w[b] = *reinterpret_cast<const uint4*>(codes + kBpCodes + b * kBpHalf + in_off);
        const bool live = ((mask >> b) & 1) && (kBpKB * j + b != last_blk || r8 < valid_last);
        if (!live) w[b] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        uint4 lo, hi;
        widen(w[b], lo, hi);
        unsigned char* dst = ops + kBpVOff + b * 2 * kBpHalf + half * kBpHalf;
        *reinterpret_cast<uint4*>(dst + out0) = half ? hi : lo;
        *reinterpret_cast<uint4*>(dst + out1) = half ? lo : hi;
      }
      mbar_arrive(hdr + kCodesVFree + 8 * st);
      fence_proxy_async_smem();
      mbar_arrive(hdr + kVFull + 8 * st);
    }
    if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
  } else if (warp >= 4) {
    regs_dec<kBpRegsIssue>();
    if (warp == 4 || warp == 6) {
      // ---- TMA producers: warp 4 K, warp 6 V; lanes 0-3 the stage's blocks -------------------
      const bool is_k = warp == 4;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      if (lane == 0) prefetch_tensor_map(tm);
      const uint32_t full = hdr + (is_k ? kCodesKFull : kCodesVFull);
      const uint32_t free_ = hdr + (is_k ? kCodesKFree : kCodesVFree);
      int issued = 0;
      bool failed = false;
      for (int j = 0; j < nst; ++j) {
        const int st = j % kBpRing;
        next_window(j);
        const int mask = stage_mask(j);
        const int blk = __shfl_sync(kFullMask, ids, ((kBpKB * j) & 31) + (lane & (kBpKB - 1)));
        bool ok = true;
        if (lane == 0 && j >= kBpRing) ok = mbar_wait_bounded(free_ + 8 * st, ((j / kBpRing) - 1) & 1);
        if (!__shfl_sync(kFullMask, ok, 0)) {
          failed = true;
          break;
        }
        const uint32_t bar = full + 8 * st;
        if (lane == 0) {
          if (mask) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(mask)) * kBpHalf);
          else mbar_arrive(bar);
        }
        __syncwarp();
        if (is_k && lane < kBpKB && kBpKB * j + lane < nblocks && !((mask >> lane) & 1))
          raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
        if (lane < kBpKB && ((mask >> lane) & 1)) {
          const uint32_t dst = stages + kBpCodeOff + st * kBpCodeStage + (is_k ? 0 : kBpCodes) + lane * kBpHalf;
          tma_load_2d(dst, tm, 0, (blk * Hkv + g) * kBlockSize, bar);
        }
        issued = j + 1;
      }
      if (lane == 0) {
        if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
        // let the copies still in flight land before the CTA exits
        for (int j = max(0, issued - kBpRing); j < issued; ++j)
          mbar_wait_bounded(full + 8 * (j % kBpRing), (j / kBpRing) & 1, 10000000ull);
      }
    } else if (warp == 5) {
      // ---- MMA issuer --------------------------------------------------------------------------
      const uint32_t id_s = umma_idesc_f16(kBpRows, kBpKeys, false, false);
      const uint32_t id_pv = umma_idesc_f16(kBpRows, kHeadDim, false, true);
      const uint64_t k_desc0 = umma_smem_desc(stages, 16, 1024);
      const uint64_t p_desc = umma_smem_desc(stages + kBpPOff, 16, 1024);
      const uint64_t v_desc0 = umma_smem_desc(stages + kBpVOff, kBpHalf, 1024);
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(kFullMask, mbar_wait_bounded(bar, parity));
      };
      // S_j = Q K_j^T once K_j is widened and the softmax has loaded S_{j-1}
      auto issue_s = [&](int j) {
        const int st = j % kBpRing;
        if (!wait_all(hdr + kKFull + 8 * st, (j / kBpRing) & 1)) return false;
        if (j > 0 && !wait_all(hdr + kSFree, (j - 1) & 1)) return false;
        tc_fence_after();
        const uint64_t kd = k_desc0 + static_cast<uint64_t>((st * kBpStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_tmem_a(tmem + kBpSCol, tmem + kBpQCol + 8 * kk,
                             kd + static_cast<uint64_t>(((kk >> 2) * kBpKHalf + (kk & 3) * 32) >> 4), id_s, kk > 0);
          umma_commit(hdr + kSFull);
          umma_commit(hdr + kKFree + 8 * st);
        }
        __syncwarp();
        return true;
      };
      bool failed = !wait_all(hdr + kQReady, 0);
      if (!failed) {
        tc_fence_after();
        failed = !issue_s(0);
      }
      for (int j = 0; j < nst && !failed; ++j) {
        if (j + 1 < nst && !issue_s(j + 1)) {
          failed = true;
          break;
        }
        const int st = j % kBpRing;
        if (!wait_all(hdr + kPFull + 8 * (j & 1), (j >> 1) & 1) || !wait_all(hdr + kVFull + 8 * st, (j / kBpRing) & 1)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint64_t vd = v_desc0 + static_cast<uint64_t>((st * kBpStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kBpKB; ++i)
            umma_bf16(tmem + kBpOCol, p_desc + static_cast<uint64_t>((32 * i) >> 4),
                      vd + static_cast<uint64_t>((i * 2 * kBpHalf) >> 4), id_pv, j > 0 || i > 0);
          umma_commit(hdr + kVFree + 8 * st);
        }
        __syncwarp();
      }
      if (lane == 0) {
        if (failed) raise_flag(a.status, PA_FLAG_TIMEOUT);
        umma_commit(hdr + kDone);
        mbar_wait_bounded(hdr + kDone, 0);
      }
      __syncwarp();
    }
  } else {
    // ---- Q into TMEM, then the softmax: thread = row r of the tile ------------------------------
    regs_inc<kBpRegsSoftmax>();
    const int r = threadIdx.x;
    const int i = r / G, h = r - (r / G) * G;
    const int p_r = pos0 + i;
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(q0 + i0 + (i < rows_q ? i : 0)) * a.num_q_heads + g * G + h) * kHeadDim);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint32_t qv[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = i < rows_q ? src[8 * part + c] : make_uint4(0u, 0u, 0u, 0u);
          qv[4 * c] = bf16x2_to_f16x2(v.x);
          qv[4 * c + 1] = bf16x2_to_f16x2(v.y);
          qv[4 * c + 2] = bf16x2_to_f16x2(v.z);
          qv[4 * c + 3] = bf16x2_to_f16x2(v.w);
        }
        tmem_st32(trow + kBpQCol + 32 * part, qv);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(hdr + kQReady);
    }
    // Scales of the lane's block of the window: factor on q . Kcode, lift of the exponent, weight in L
    float fold = 0.f, lift = 0.f, weigh = 0.f, fold_next = 0.f, lift_next = 0.f, weigh_next = 0.f;
    auto load_scales = [&](int id, float& f, float& e, float& w) {
      const float2 kv = in_pool(id) ? a.kv_scale[static_cast<size_t>(id) * Hkv + g] : make_float2(1.f, 1.f);
      f = a.scale_log2 * kv.x;
      e = log2_of(kv.y);
      w = __frcp_rn(kv.y);
    };
    load_scales(ids, fold, lift, weigh);
    load_scales(ids_next, fold_next, lift_next, weigh_next);
    float m = -INFINITY, l = 0.f;
    bool failed = false;
    const uint32_t sbuf = trow + kBpSCol;
    for (int j = 0; j < nst; ++j) {
      if (next_window(j)) {
        fold = fold_next;
        lift = lift_next;
        weigh = weigh_next;
        load_scales(ids_next, fold_next, lift_next, weigh_next);
      }
      const int mask = stage_mask(j);
      float f[kBpKB], e[kBpKB], w[kBpKB];
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {
        const int src = ((kBpKB * j) & 31) + b;
        f[b] = __shfl_sync(kFullMask, fold, src);
        e[b] = __shfl_sync(kFullMask, lift, src);
        w[b] = __shfl_sync(kFullMask, weigh, src);
      }
      if (!__all_sync(kFullMask, mbar_wait_bounded(hdr + kSFull, j & 1))) {
        failed = true;
        break;
      }
      tc_fence_after();
      float sc[kBpKeys];
      {
        uint32_t sv[32];
        tmem_ld32(sbuf, sv);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) sc[c] = __uint_as_float(sv[c]);
        tmem_ld32(sbuf + 32, sv);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) sc[32 + c] = __uint_as_float(sv[c]);
      }
      tc_fence_before();
      mbar_arrive(hdr + kSFree);
      // causal mask and absent blocks -> -inf, only on a stage that needs it
      if (mask != (1 << kBpKB) - 1 || kBpKeys * (j + 1) - 1 > pos0) {
        const int lim = p_r - kBpKeys * j;
#pragma unroll
        for (int c = 0; c < kBpKeys; ++c)
          if (!((mask >> (c / kBlockSize)) & 1) || c > lim) sc[c] = -INFINITY;
      }
      float mrow = -INFINITY;
#pragma unroll
      for (int b = 0; b < kBpKB; ++b) {             // 16 -> 6 -> 2 -> 1, then the block's scale
        const float* x = sc + kBlockSize * b;
        const float u0 = fmax3(x[0], x[1], x[2]), u1 = fmax3(x[3], x[4], x[5]), u2 = fmax3(x[6], x[7], x[8]);
        const float u3 = fmax3(x[9], x[10], x[11]), u4 = fmax3(x[12], x[13], x[14]);
        mrow = fmaxf(mrow, fmaf(fmax3(fmax3(u0, u1, u2), fmaxf(u3, u4), x[15]), f[b], e[b]));
      }
      const float mn = mrow > m + 15.f ? mrow - 7.f : m;
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
      // P V of stage j - 1 must be done before P_j overwrites its buffer and before O is rescaled
      if (j > 0) {
        const int pj = j - 1;
        if (!__all_sync(kFullMask, mbar_wait_bounded(hdr + kVFree + 8 * (pj % kBpRing), (pj / kBpRing) & 1))) {
          failed = true;
          break;
        }
        tc_fence_after();
      }
      if (j > 0 && __any_sync(kFullMask, alpha != 1.f)) {
#pragma unroll 1
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t ov[32];
          tmem_ld32(trow + kBpOCol + 32 * q4, ov);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
          tmem_st32(trow + kBpOCol + 32 * q4, ov);
        }
        tmem_wait_st();
      }
      {
        unsigned char* prow = base + kBpPOff + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) =
              make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(hdr + kPFull + 8 * (j & 1));
    }
    if (failed) {
      if (lane == 0) raise_flag(a.status, PA_FLAG_TIMEOUT);
    } else if (__all_sync(kFullMask, mbar_wait_bounded(hdr + kDone, 0))) {
      tc_fence_after();
      // a row whose every key was skipped has l = 0: zeros
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool store = i < rows_q;
      uint4* dst = reinterpret_cast<uint4*>(
          a.out + (static_cast<size_t>(q0 + i0 + (store ? i : 0)) * a.num_q_heads + g * G + h) * kHeadDim);
#pragma unroll 1
      for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t ov[32];
        tmem_ld32(trow + kBpOCol + 32 * q4, ov);
        tmem_wait_ld();
        if (store) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              o[u] = pack_bf16x2(__uint_as_float(ov[8 * k + 2 * u]) * inv, __uint_as_float(ov[8 * k + 2 * u + 1]) * inv);
            dst[4 * q4 + k] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    } else if (lane == 0) {
      raise_flag(a.status, PA_FLAG_TIMEOUT);
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
      err = cudaFuncSetAttribute(prefill_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBpSmem);
      if (err != cudaSuccess) return err;
      err = cudaFuncSetAttribute(prefill_block_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
      if (err != cudaSuccess) return err;
      done[dev] = true;
    }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.max_query_len + Tq - 1) / Tq),
                     static_cast<unsigned>(a.num_seqs * a.num_kv_heads));
  cfg.blockDim = dim3(static_cast<unsigned>(kBpThreads));
  cfg.dynamicSmemBytes = kBpSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_block_kernel, tm_k, tm_v, a);
}

}  // namespace pa
