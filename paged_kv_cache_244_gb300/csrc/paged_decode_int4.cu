// Single-token paged GQA decode attention over the 4-bit cache, for sm_103a, with the fused step (RoPE
// form + quantising store of the new token).
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现": §2 Kernel层 (PagedAttention decode kernel), §H200上的详细对比
// (Flash Decode); "从零实现 LLM 推理引擎：深挖 vLLM 的六大核心优化", §3.1 Paged KV Cache; "nano-vllm：vLLM
// 极简实现与大模型推理流程解析", §学习要点 (4-bit quantisation of the cache).
//
// The work is cut as in the other decode kernels (pa_device.cuh): one axis of (sequence, KV head, block),
// an equal contiguous range for each warp of a persistent grid, pieces of split segments merged by a kernel
// after it.  The mathematics, with K element (t, d) =
// s_tg (c_td - z_tg) for d in group g of 32 dims, V element s_t (c_td - z_t), and head column h:
//
//   score   x_th = sum_g s_tg sum_{d in g} q_hd c_td - sum_g s_tg z_tg Q_hg,   Q_hg = sum_{d in g} q_hd
//   weight  e_th = scale_log2 x_th + log2 s_t,   p_th = 2^(e_th - m_h)
//   output  out_hd = (sum_t p_th c_td - sum_t p_th z_t) / L_h,   L_h = sum_t p_th / s_t
//
// Codes enter the matrix instructions with no conversion: a pair masked out of a shifted word is a pair of small
// f16 values, c 2^-21 or c 2^-17, exact (below 2^-13 an f16 pattern is its integer times 2^-24), and the products
// with a normal q or p are normal fp32 numbers.  Eight codes cost six integer instructions.  (Masked as they lie, at
// 2^-24 and 2^-20, they cost five, but the instruction aligns a subnormal operand by its exponent field, and the last
// bits of what is added to a large product were lost: 2^-13 of it.)  The factor of 16 between the two kinds of
// pair is taken out of q for K, and out of the accumulators for V at the end.  The two sums over zero points are
// matrix instructions as well:
//   - sum_g s_tg z_tg Q_hg is one bf16 instruction a block: s z is exact in bf16, and each Q_hg goes in as
//     three bf16 numbers that add up to it.
//   - sum_t p_th z_t is one f16 instruction a block whose A operand has the zero points in every row, so each
//     lane gets the sum for its own head columns, over the same rounded p as the codes' sums.
// V's scale acts on the exponent and cancels in L, so p stays within f16 whatever the scales: the shift m is
// set 7 below the largest contribution and moves when one passes it by more than 15.  L adds the unrounded p.
// Where a shift passes 2^10, log2 s would be rounded away next to the score, and the piece forms e_th as
// (scale_log2 x_th - base) + log2 s_t from there on (kFarShift).
//
// A job is up to two neighbouring blocks of a piece in one stage of the warp's ring.  A record is one run of memory, so
// each of a stage's few runs (two records, q of a piece's first job, the step's rows) is one bulk copy.  Where 16
// tokens are 2.2 KB, what a job costs whatever its size counts as much as its products: walking the range, table
// look-ups, flags and copies took a warp 120 instructions a block, of 366 in all.  So one warp of the CTA
// does it for all the others, a lane for each: a pass of its loop emits the next job of every consumer that has a
// free stage.
//
// What bounds it: us replayed from a graph, 64 sequences of 64-4096 tokens.  12 / 2 heads (39 MB) 17.6; 32 / 8 heads (156
// MB, 23.0 at the copy rate) 42.1, the fused step 48.0; one sequence of 2048 tokens 6.9, latency.  Of the 42.1, 32.5 lie
// between the first CTA's lengths and the last one's last job: 0.9 for the prefix, 3.3 for ids and the first record, 25.7
// for the loop (medians of the CTAs; 27.9 the longest); the merge takes 1.9, and the rest are the two kernels' hand-overs
// and ends.  The whole call without its products takes 33.0, without copies and feeder 34.6 (2 of it to fill the
// stages once): each is most of the 42.1, and they overlap in part.  Of some 310 instructions a record and kernel 147 go
// to the ALU, one in two cycles (80 masks and shifts for the operands, the scales, the softmax), and the one feeder is
// never idle: 77 - 80 cycles a bulk copy of one record.  Neither pipe nor DRAM is full; copies of all KV heads' records
// of a block (they are adjacent) would take fewer, with another way to cut the work, and are not built.
// Tried (32 / 8 heads, against 42.0): each warp feeding itself 44.6; the feeder
// describing jobs and each warp asking for its own copies 47.5, by cp.async 48.1; cp.async by 1, 2, 3 or 4 feeders 60,
// 46.0, 43.4, 44.0; two feeders for bulk copies 43.2; block ids asked for a job ahead 45.0; 7, 13 or 15 consumers 48.4,
// 44.1, 43.0 (the last with 128 registers); the right shift as a product's upper half 44.8; jobs of four blocks 46.7.
// The step's 6 us over the decode: quantising and storing 2, rotating q 1.5, its rows 1.2, fewer stages the rest.

#include <mutex>
#include <type_traits>

#include "int4_cache.cuh"
#include "int4_launch.h"

namespace pa {
namespace {

constexpr int kDiConsumers = 11;                     // warps of a CTA that have ranges; one more feeds them
constexpr int kDiJob = 2;                            // blocks of a job at most
// A stage: its job's descriptor, records, q rows of G heads, and for the step cos/sin (R <= 128 floats), k and v.
constexpr int kDiRecOff = 32;
constexpr int kDiQOff = kDiRecOff + kDiJob * kInt4Record;
__host__ __device__ constexpr int di_stage(int G, bool step) {
  return kDiQOff + G * kHeadDim * 2 + (step ? kHeadDim * 4 + 2 * kHeadDim * 2 : 0);
}
constexpr int kDiMaxRing = 8;                        // stages of a warp
constexpr int kDiSmemMax = 226 * 1024;               // beside the static part of build_prefix
// Shared memory: per consumer and stage a barrier that the copies complete and one that the consumer does, a word set
// when a wait has run out, the prefix, the stages.
constexpr int kDiBarOff = 0;
constexpr int kDiFailOff = kDiConsumers * kDiMaxRing * 16;
constexpr int kDiPrefixOff = kDiFailOff + 16;
// The largest call's step has two stages for every consumer, so all calls have the same ones, with and without the step: both
// cut sequences alike and give the same bits.
static_assert((kDiSmemMax - kDiPrefixOff - prefix_bytes(kMaxDecodeSeqs)) / di_stage(8, true) >= 2 * kDiConsumers, "stages");

// More job flags: two blocks, and which of them are there (valid tokens of the last one at bits 8-12).
constexpr uint32_t kTwo = 1u << 13, kHas0 = 1u << 14, kHas1 = 1u << 15;

// A shift below every score (they are finite, and below 2^123): weights of no key so far are 0, not NaN.
constexpr float kNoShift = -3.402823466e38f;

// Shifts up to this size (in the exponent, so scores up to 710 or so) keep log2 s to 2^-14 where it is added to a score.
// Past it the addition would round the scales of V away (by 2^-4 at 2^20, whole at 2^26) while L still divides by them, so
// a piece goes on with each head's scores counted from its largest one, which leaves near ones exact.
constexpr float kFarShift = 0x1p10f;

// Pairs of codes as f16: of a word's neighbouring pairs shifted by 3, the first c 2^-21 and the second c 2^-17.
constexpr uint32_t kPairA = 0x00780078u, kPairB = 0x07800780u;

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
// Whether phase `parity` of the barrier is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D = A B of f16 (bf16) operands: the accumulator begins at zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <bool kStep>
__global__ void __launch_bounds__((kDiConsumers + 1) * 32, 1) decode_int4_kernel(const DecodeArgs a, const int pool) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  int* prefix = reinterpret_cast<int*>(smem_raw + kDiPrefixOff);
  unsigned char* last_rows = smem_raw + kDiPrefixOff + (((a.num_seqs + 1) * 4 + 15) & ~15);
  const uint32_t tile_base = raw + kDiPrefixOff + prefix_bytes(a.num_seqs);
  // With early metadata the lengths and block table are read, and the work resolved, before the
  // preceding kernel has finished; copies and writes wait for it (below).
  const bool early = a.early_metadata != 0;
  if (!early) pdl_wait_prior_grid();
  pdl_allow_next_grid();

  const int S = a.num_seqs;
  const int Hkv = a.num_kv_heads;
  const int G = a.num_q_heads / Hkv;
  constexpr int warps = kDiConsumers;
  const int stage_bytes = di_stage(G, kStep);
  const int cos_off = kDiQOff + G * kHeadDim * 2;    // (step)
  for (int i = threadIdx.x; i < warps * kDiMaxRing * 2; i += (warps + 1) * 32) mbar_init(raw + kDiBarOff + 8 * i, 1);
  volatile int* const fail = reinterpret_cast<volatile int*>(smem_raw + kDiFailOff);
  if (threadIdx.x == 0) *fail = 0;
  fence_mbar_init();
  build_prefix<kDiConsumers + 1>(a, prefix, last_rows);   // (a barrier of the CTA behind the above)
  const long long T = static_cast<long long>(Hkv) * prefix[S];
  const Ranges R = make_ranges(T, a);
  // Range v goes to consumer v / grid of CTA v % grid; the CTA's stages are shared out among its consumers
  // that have a range, the first of them taking one more where they do not divide.
  const int active = min(warps, max(0, (R.V - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                                           static_cast<int>(gridDim.x)));
  const int who = warp < warps ? warp : lane;        // consumer: this warp, or the one that this lane feeds
  if (active == 0 || (warp < warps && warp >= active)) {
    if (early) pdl_wait_prior_grid();
    return;
  }
  const int my_v = static_cast<int>(blockIdx.x) + who * static_cast<int>(gridDim.x);
  const int n_st = min(pool / active + (who < pool % active ? 1 : 0), kDiMaxRing);
  const uint32_t ring = tile_base + (who * (pool / active) + min(who, pool % active)) * stage_bytes;
  const uint32_t ring_end = ring + n_st * stage_bytes;
  const uint32_t full_bars = raw + kDiBarOff + who * kDiMaxRing * 16;   // the stage's other barrier 8 bytes behind

  if (warp == warps) {
    // ---------------------------------------------------------------- feeder ----------
    const uint8_t* const cache = reinterpret_cast<const uint8_t*>(a.k_cache);
    const bool mine = lane < active;
    const long long x0 = mine ? R.begin(my_v) : 0;
    const int len = mine ? static_cast<int>(R.begin(my_v + 1) - x0) : 0;
    // The next job: block `rel` of the range is block j of ns of (sequence s, KV head g).
    int rel = 0, s = 0, g = 0, j = 0, ns = 1, id0 = -1, id1 = -1;
    uint32_t fl = 0;
    const int chunk = a.chunk_blocks;
    // flags of the job at hand, its block ids asked for
    auto look = [&] {
      const int part = chunk ? j / chunk : 0;
      const bool p_first = chunk && j == part * chunk;
      auto ends = [&](int d) { return rel + d == len - 1 || j + d == ns - 1 || (chunk && j + d == part * chunk + chunk - 1); };
      const bool two = !ends(0);                     // a piece ends at the range's end at the latest
      const bool whole = rel >= j && rel - j + ns <= len && (chunk == 0 || ns <= chunk);
      const bool tail = j + (two ? 1 : 0) == ns - 1; // the job reaches the sequence's last block
      fl = ((rel == 0 || j == 0 || p_first) ? kFirst : 0u) | (ends(two ? 1 : 0) ? kLast : 0u) | (whole ? kWhole : 0u) |
           ((rel == 0 && j > 0 && p_first) ? kGap : 0u) | (two ? kTwo : 0u) | (tail ? kNew : 0u);
      fl |= static_cast<uint32_t>(tail ? last_rows[s] : kBlockSize) << 8;
      const int32_t* ids = a.block_tables + static_cast<size_t>(s) * a.max_blocks + j;
      id0 = ids[0];
      if (two) id1 = ids[1];
    };
    if (mine) {
      int lo = 0, hi = S;                            // largest s with Hkv * N_s <= x0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(Hkv) * prefix[mid] <= x0) lo = mid;
        else hi = mid;
      }
      s = lo;
      ns = prefix[s + 1] - prefix[s];
      const int off = static_cast<int>(x0 - static_cast<long long>(Hkv) * prefix[s]);
      g = off / ns;
      j = off - g * ns;
      look();
    }
    if (early) pdl_wait_prior_grid();
    uint32_t at = ring, bar = full_bars, phase = 1;  // parity of the stage's last release
    int fills = 0;
    uint64_t since = 0;                              // of waiting with nothing to do
    while (__any_sync(kFullMask, rel < len)) {
      bool ready = rel < len;
      if (ready && fills >= n_st) ready = mbar_test(bar + 8, phase);
      if (!__any_sync(kFullMask, ready)) {
        if (__any_sync(kFullMask, *fail != 0)) break;   // together: the loop's votes want every lane
        const uint64_t now = global_ns();
        if (since == 0) since = now;
        if (__any_sync(kFullMask, now - since > kWaitLimitNs)) {
          if (lane == 0) raise_flag(a.status, PA_FLAG_TIMEOUT);
          break;
        }
        __nanosleep(32);
        continue;
      }
      since = 0;
      if (ready) {
        const bool two = (fl & kTwo) != 0;
        const bool here0 = id0 >= 0 && id0 < a.num_blocks, here1 = two && id1 >= 0 && id1 < a.num_blocks;
        const int row0 = here0 ? id0 * Hkv + g : 0, row1 = here1 ? id1 * Hkv + g : 0;
        const int seg = s * Hkv + g;
        const int part = chunk ? j / chunk : 0;
        // Fused step: a position without a cos/sin row leaves the token out -- q unrotated, nothing stored.
        const int pos = (ns - 1) * kBlockSize + last_rows[s] - 1;
        const bool rope = kStep && pos < a.max_pos;
        const bool fresh = rope && (fl & kNew) && (two ? here1 : here0);    // the new token's record is here
        const bool turns = rope && ((fl & kFirst) || fresh);
        if (kStep && (fl & kNew) && !rope) raise_flag(a.status, PA_FLAG_POSITION_OOB);
        if (!here0 || (two && !here1)) raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
        const uint32_t flags = (fl & ~kNew) | (fresh ? kNew : 0u) | (rope ? kRope : 0u) | (here0 ? kHas0 : 0u) | (here1 ? kHas1 : 0u);
        *reinterpret_cast<int4*>(smem_raw + (at - raw)) =
            make_int4(seg, static_cast<int>(flags), static_cast<int>(piece_slot(my_v, seg, part, a.max_parts)), two ? row1 : row0);
        uint32_t bytes = (static_cast<uint32_t>(here0) + static_cast<uint32_t>(here1)) * kInt4Record;
        if (fl & kFirst) bytes += G * kHeadDim * 2;
        if (kStep) bytes += (turns ? a.rotary_dim * 4 : 0) + (fresh ? 2 * kHeadDim * 2 : 0);
        if (bytes) mbar_arrive_expect_tx(bar, bytes);
        else mbar_arrive(bar);
        if (fl & kFirst) bulk_copy_g2s(at + kDiQOff, a.q + static_cast<size_t>(seg) * G * kHeadDim, G * kHeadDim * 2, bar);
        if (kStep && turns)
          bulk_copy_g2s(at + cos_off, a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim, a.rotary_dim * 4, bar);
        if (kStep && fresh) {
          bulk_copy_g2s(at + cos_off + kHeadDim * 4, a.k_new + static_cast<size_t>(seg) * kHeadDim, kHeadDim * 2, bar);
          bulk_copy_g2s(at + cos_off + kHeadDim * 6, a.v_new + static_cast<size_t>(seg) * kHeadDim, kHeadDim * 2, bar);
        }
        if (here0) bulk_copy_g2s(at + kDiRecOff, cache + static_cast<size_t>(row0) * kInt4Record, kInt4Record, bar);
        if (here1) bulk_copy_g2s(at + kDiRecOff + kInt4Record, cache + static_cast<size_t>(row1) * kInt4Record, kInt4Record, bar);
        ++fills;
        at += stage_bytes;
        bar += 16;
        if (at == ring_end) {
          at = ring;
          bar = full_bars;
          phase ^= 1u;
        }
        rel += two ? 2 : 1;
        j += two ? 2 : 1;
        if (rel < len) {
          if (j == ns) {
            j = 0;
            if (++g == Hkv) {
              g = 0;
              do ++s;
              while (prefix[s + 1] == prefix[s]);    // blocks are left, so a later sequence has some
              ns = prefix[s + 1] - prefix[s];
            }
          }
          look();
        }
      }
      __syncwarp();
    }
    // let the copies still in flight land before the CTA exits (they have, in a normal run, but for the last ones)
    for (int k = max(0, fills - n_st); k < fills; ++k) mbar_wait_bounded(full_bars + 16 * (k % n_st), (k / n_st) & 1);
    return;
  }
  if (early) pdl_wait_prior_grid();
  const int gq = lane >> 2;  // fragment row group
  const int cq = lane & 3;   // fragment column pair

  // ---------------------------------------------------------------- consumer state --
  // V rows of this lane's ldmatrix addresses: token r + 8 (i & 1), 16-byte unit u of its row at u ^ (r / 2 % 4)
  const int mi = lane >> 3, r8 = lane & 7;
  const uint32_t v_row = static_cast<uint32_t>(kInt4VCodes + 64 * (r8 + 8 * (mi & 1)));
  const int v_unit = mi >> 1, v_turn = (r8 >> 1) & 3;
  uint32_t qb[8][2];                      // B operand: dims 32c + 8cq .. + 7 of head gq, k permuted as the codes are
  uint32_t qsum[2];                       // B operand: -Q of group cq of head gq as three bf16 numbers
  float kf0 = 0.f, kf1 = 0.f;             // what turns x of head columns 2cq, 2cq + 1 into the exponent
  float m0 = kNoShift, m1 = kNoShift;     // softmax shifts of those columns, from their bases:
  float base0 = 0.f, base1 = 0.f;         // 0, or with `far` the largest score so far
  bool far = false;                       // of the piece, the same in every lane
  float l0 = 0.f, l1 = 0.f;               // this lane's share of L
  float o[8][4];                          // sums of p c: [2u + i] = rows gq, gq + 8: code pairs 2i, 2i + 1 of unit u
  float z[4];                             // sums of p z (two and two alike)

  // The new token (row `row` of the stage's record at `rec`, in the cache record `tile_row`) is rotated and
  // quantised into both.
  auto store_new = [&](unsigned char* stage, unsigned char* rec, int row, int tile_row) {
    const float* cs = reinterpret_cast<const float*>(stage + cos_off);
    uint32_t* kn = reinterpret_cast<uint32_t*>(stage + cos_off + kHeadDim * 4);
    const int rot = a.rotary_dim;
    // Lane l < R/4 turns two words (dim pairs) of the row: of the half layout words l and l + R/4, of the
    // interleaved one 2l and 2l + 1.
    if (lane < rot / 4) {
      const int wa = a.interleaved ? 2 * lane : lane, wb = a.interleaved ? 2 * lane + 1 : lane + rot / 4;
      uint32_t kx = kn[wa], ky = kn[wb];
      const float2 co = reinterpret_cast<const float2*>(cs)[lane];
      const float2 si = reinterpret_cast<const float2*>(cs + rot / 2)[lane];
      if (a.interleaved) int4_rotate<true>(kx, ky, co, si);
      else int4_rotate<false>(kx, ky, co, si);
      kn[wa] = kx;
      kn[wb] = ky;
    }
    __syncwarp();
    // half-lanes: 0-15 the chunks of 8 dims of k, 16-31 those of v
    const int ch = lane & 15;
    const bool is_k = lane < 16;
    const uint4 w = reinterpret_cast<const uint4*>(kn)[lane];
    bool wild = false;
    uint32_t e = int4_extremes(w, wild);
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) {
      const uint32_t other = __shfl_xor_sync(kFullMask, e, x);
      if (x < 4 || !is_k) e = __vmaxu2(e, other);
    }
    const Int4Scale qs = int4_scale(e);
    const uint32_t code = int4_word(w, qs, wild);
    uint8_t* const dst = reinterpret_cast<uint8_t*>(a.k_store) + static_cast<size_t>(tile_row) * kInt4Record;
    const int at = is_k ? int4_k_word(row, ch) : int4_v_word(row, ch);
    *reinterpret_cast<uint32_t*>(rec + at) = code;
    *reinterpret_cast<uint32_t*>(dst + at) = code;
    const int sat = is_k ? kInt4KScales + 8 * row + 2 * (ch >> 2) : kInt4VScales + 2 * row;
    if (is_k ? (ch & 3) == 0 : ch == 0) {
      *reinterpret_cast<uint16_t*>(rec + sat) = static_cast<uint16_t>(qs.word);
      *reinterpret_cast<uint16_t*>(dst + sat) = static_cast<uint16_t>(qs.word);
    }
    __syncwarp();
  };

  // q rows of the piece: rotated (step), scaled and rounded to f16.
  auto load_q = [&](const unsigned char* stage, uint32_t fl) {
    const uint4* qrow = reinterpret_cast<const uint4*>(stage + kDiQOff + (gq < G ? gq : 0) * kHeadDim * 2);
    uint32_t w[4][4];                     // dims 32c + 8cq + 2j, + 1
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = gq < G ? qrow[4 * c + cq] : make_uint4(0u, 0u, 0u, 0u);
      w[c][0] = v.x;
      w[c][1] = v.y;
      w[c][2] = v.z;
      w[c][3] = v.w;
    }
    if (kStep && (fl & kRope)) {
      const int rot = a.rotary_dim, half = rot / 2;
      const float* cs = reinterpret_cast<const float*>(stage + cos_off);
      if (!a.interleaved && rot == kHeadDim) {       // partners 64 dims away, in the same lane
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = 32 * c + 8 * cq + 2 * j;
            rope_rotate_pairs(w[c][j], w[c + 2][j], *reinterpret_cast<const float2*>(cs + d),
                              *reinterpret_cast<const float2*>(cs + 64 + d));
          }
        }
      } else {
        // dims below R turn: within neighbouring words when interleaved, else with the dims R/2 away, read
        // from the row (R/2 is a multiple of 8: a lane's eight dims lie on one side)
        const uint32_t* row = reinterpret_cast<const uint32_t*>(qrow);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int d = 32 * c + 8 * cq;
          if (d >= rot || gq >= G) continue;
          if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              rope_rotate_interleaved(w[c][j], w[c][j + 1], *reinterpret_cast<const float2*>(cs + d / 2 + j),
                                      *reinterpret_cast<const float2*>(cs + half + d / 2 + j));
          } else {
            const int i = d < half ? d : d - half;   // angle of the first dim
            const int other_dim = d < half ? d + half : i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t other = row[other_dim / 2 + j];
              const float2 co = *reinterpret_cast<const float2*>(cs + i + 2 * j);
              const float2 si = *reinterpret_cast<const float2*>(cs + half + i + 2 * j);
              if (d < half) rope_rotate_pairs(w[c][j], other, co, si);
              else rope_rotate_pairs(other, w[c][j], co, si);
            }
          }
        }
      }
    }
    __syncwarp();
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[c][j] & 0x7fff7fffu);
    top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, 2));
    top = max(top & 0xffffu, top >> 16);             // the head's largest magnitude
    // to [128, 256); below 2^-119 not as far: multiples of 2^-133 become multiples of 2^-7, exact all the same
    const int e = min(7 + 127 - static_cast<int>(top >> 7), 126);
    const float raise = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    // Pairs j = 0 and 2 meet codes of 2^-21 and go in 16 times larger, pairs 1 and 3 codes of 2^-17.
    float part[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = (j & 1) ? 1.f : 16.f;
        const uint32_t h = pack_f16x2(bf16lo(w[c][j]) * raise * f, bf16hi(w[c][j]) * raise * f);
        qb[2 * c + (j >> 1)][j & 1] = h;
        s = fmaf(f16lo(h) + f16hi(h), 1.f / f, s);
      }
      part[c] = s;
    }
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      part[c] += __shfl_xor_sync(kFullMask, part[c], 1);
      part[c] += __shfl_xor_sync(kFullMask, part[c], 2);
      if (c == cq) mine = part[c];
    }
    mine *= -0x1p-17f;
    const uint32_t hi = pack_bf16x2(mine, 0.f);
    const float rest = mine - bf16lo(hi);
    const uint32_t mid = pack_bf16x2(rest, 0.f);
    qsum[0] = hi | (mid << 16);
    qsum[1] = pack_bf16x2(rest - bf16lo(mid), 0.f);
    // x is 2^-17 raise of the product of q and K; an infinity or a NaN in q makes the head's scores NaN
    const float fold = top >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                      : row_factor(a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23)) * 0x1p17f;
    kf0 = __shfl_sync(kFullMask, fold, 8 * cq);
    kf1 = __shfl_sync(kFullMask, fold, 8 * cq + 4);
  };

  auto consume = [&](uint32_t at) -> int {
    unsigned char* const stage = smem_raw + (at - raw);
    const int4 d = *reinterpret_cast<const int4*>(stage);
    const uint32_t fl = static_cast<uint32_t>(d.y);
    const uint32_t kt = at + kDiRecOff;
    if (fl & kFirst) {
      load_q(stage, fl);
      m0 = m1 = kNoShift;
      base0 = base1 = 0.f;
      far = false;
      l0 = l1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      z[0] = z[1] = z[2] = z[3] = 0.f;
      if ((fl & kGap) && lane < G)                   // mark the skipped slot before this piece empty
        a.ws_ml[(static_cast<size_t>(d.z) - 1) * G + lane] = make_float2(-INFINITY, 0.f);
      __syncwarp();                                  // some lanes have stored; what follows wants the whole warp
    }
    const bool two = (fl & kTwo) != 0;
    const int valid = static_cast<int>((fl >> 8) & 0x1fu);   // rows of the job's last block
    if (kStep && (fl & kNew)) store_new(stage, stage + kDiRecOff + (two ? kInt4Record : 0), valid - 1, d.w);

    // Exponents before the shift: [i][0] = (token gq of block i, head 2cq), [1] = (gq, 2cq + 1), [2] = (gq + 8,
    // 2cq), [3] = (gq + 8, 2cq + 1); and 1 / s of V of tokens gq, gq + 8.
    float y[kDiJob][4], iv[kDiJob][2];
    float ev[kDiJob][2];                             // log2 s of V of tokens gq, gq + 8 (used with `far`)
    auto scores = [&](int i, auto apart) {           // apart: y without log2 s of V
      const uint32_t rec = kt + i * kInt4Record;
      const uint4 wa = lds128(rec + 64 * gq + 16 * cq), wb = lds128(rec + 64 * gq + 512 + 16 * cq);
      const uint2 sa = lds64(rec + kInt4KScales + 8 * gq), sb = lds64(rec + kInt4KScales + 64 + 8 * gq);
      const uint32_t ga = lds16(rec + kInt4KScales + 8 * gq + 2 * cq), gb = lds16(rec + kInt4KScales + 64 + 8 * gq + 2 * cq);
      const float va = int4_scale_of(lds16(rec + kInt4VScales + 2 * gq));
      const float vb = int4_scale_of(lds16(rec + kInt4VScales + 16 + 2 * gq));
      float x[4];
      {  // - sum_g s z Q: A rows = tokens, this lane's four k indices all stand for group cq
        const uint32_t w = __byte_perm(ga, gb, 0x5410);
        const uint32_t sz = mul_bf16x2(w & 0xfff0fff0u, sub_bf16x2((w & kPairLo) | 0x43004300u, 0x43004300u));
        const uint32_t ra = __byte_perm(sz, sz, 0x1010), rb = __byte_perm(sz, sz, 0x3232);
        mma_bf16_first(x, ra, rb, ra, rb, qsum[0], qsum[1]);
      }
      auto group = [&](int c, uint32_t u, uint32_t v, float fu, float fv) {
        float acc[4];
        const uint32_t u0 = u << 3, v0 = v << 3, u1 = u >> 5, v1 = v >> 5;
        mma_f16_first(acc, u0 & kPairA, v0 & kPairA, u0 & kPairB, v0 & kPairB, qb[2 * c][0], qb[2 * c][1]);
        mma_f16_16816(acc, u1 & kPairA, v1 & kPairA, u1 & kPairB, v1 & kPairB, qb[2 * c + 1][0], qb[2 * c + 1][1]);
        x[0] = fmaf(fu, acc[0], x[0]);
        x[1] = fmaf(fu, acc[1], x[1]);
        x[2] = fmaf(fv, acc[2], x[2]);
        x[3] = fmaf(fv, acc[3], x[3]);
      };
      group(0, wa.x, wb.x, int4_scale_of(sa.x), int4_scale_of(sb.x));
      group(1, wa.y, wb.y, __uint_as_float(sa.x & 0xfff00000u), __uint_as_float(sb.x & 0xfff00000u));
      group(2, wa.z, wb.z, int4_scale_of(sa.y), int4_scale_of(sb.y));
      group(3, wa.w, wb.w, __uint_as_float(sa.y & 0xfff00000u), __uint_as_float(sb.y & 0xfff00000u));
      // 2^-65 more: nothing to a scale of 2^-40 or more, and a slot of zeros (a cleared cache that nothing was stored in)
      // counts in L like any token of its score, with codes of zero
      const float sva = va + 0x1p-65f, svb = vb + 0x1p-65f;
      const float ea = lg2(sva), eb = lg2(svb);
      if constexpr (decltype(apart)::value) {
        y[i][0] = __fmul_rn(x[0], kf0);
        y[i][1] = __fmul_rn(x[1], kf1);
        y[i][2] = __fmul_rn(x[2], kf0);
        y[i][3] = __fmul_rn(x[3], kf1);
        ev[i][0] = ea;
        ev[i][1] = eb;
      } else {
        y[i][0] = fmaf(x[0], kf0, ea);
        y[i][1] = fmaf(x[1], kf1, ea);
        y[i][2] = fmaf(x[2], kf0, eb);
        y[i][3] = fmaf(x[3], kf1, eb);
      }
      iv[i][0] = rcp_ftz(sva);
      iv[i][1] = rcp_ftz(svb);
    };
    // Most jobs are two whole blocks: theirs is a path without a branch, whose blocks interleave.
    const bool full = (fl & (kTwo | kHas0 | kHas1)) == (kTwo | kHas0 | kHas1) && valid == kBlockSize;
    auto each_block = [&](auto apart) {
#pragma unroll
      for (int i = 0; i < kDiJob; ++i) {
        y[i][0] = y[i][1] = y[i][2] = y[i][3] = -INFINITY;
        iv[i][0] = iv[i][1] = 0.f;
        if (i == 1 && !two) continue;
        scores(i, apart);
        // tokens past the context, and absent blocks, may hold anything
        const int n = !(fl & (i ? kHas1 : kHas0)) ? 0 : i == 1 || !two ? valid : kBlockSize;
        if (gq >= n) y[i][0] = y[i][1] = -INFINITY, iv[i][0] = 0.f;
        if (gq + 8 >= n) y[i][2] = y[i][3] = -INFINITY, iv[i][1] = 0.f;
      }
      __syncwarp();
    };
    float top0, top1;
    auto tops = [&] {                                // of this lane's tokens
      top0 = top1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < kDiJob; ++i) {
        top0 = fmax3(top0, y[i][0], y[i][2]);
        top1 = fmax3(top1, y[i][1], y[i][3]);
      }
    };
    auto over_tokens = [&] {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        top0 = fmaxf(top0, __shfl_xor_sync(kFullMask, top0, x));
        top1 = fmaxf(top1, __shfl_xor_sync(kFullMask, top1, x));
      }
    };
    if (!far) {
      if (full) {
#pragma unroll
        for (int i = 0; i < kDiJob; ++i) scores(i, std::false_type{});
      } else {
        each_block(std::false_type{});
      }
      tops();
    }
    const bool near = !far && !__any_sync(kFullMask, top0 - m0 > 15.f || top1 - m1 > 15.f);
    if (!near) {
      // A shift may have to move (at a piece's first job from kNoShift): the maxima over the tokens, and what
      // was summed so far scaled to the new shifts.
      if (!far) {
        over_tokens();
        far = __any_sync(kFullMask, (top0 - m0 > 15.f && fabsf(top0) > kFarShift) || (top1 - m1 > 15.f && fabsf(top1) > kFarShift));
        if (far) {                                   // what there is so far is counted from its shift
          if (m0 != kNoShift) base0 = m0, m0 = 0.f;
          if (m1 != kNoShift) base1 = m1, m1 = 0.f;
        }
      }
      if (far) {
        // Scores by themselves, rounded; their differences to the base are exact where they matter, and log2 s is added
        // to those.  A base moves up to the largest score, so that one is at most 0 from it and a shift some
        // 90 at most; without keys so far it is set to it.
        each_block(std::true_type{});
        tops();
        over_tokens();
        auto rebase = [](float top, float& base, float& m) {
          const float to = m == kNoShift ? (top == -INFINITY ? base : top) : fmaxf(base, top);
          if (m != kNoShift) m -= to - base;
          base = to;
        };
        rebase(top0, base0, m0);
        rebase(top1, base1, m1);
#pragma unroll
        for (int i = 0; i < kDiJob; ++i) {
          if (i == 1 && !two) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (y[i][c] != -INFINITY) y[i][c] = y[i][c] - ((c & 1) ? base1 : base0) + ev[i][c >> 1];
        }
        __syncwarp();
        tops();
        over_tokens();
      }
      const float mn0 = top0 - m0 > 15.f ? top0 - 7.f : m0, mn1 = top1 - m1 > 15.f ? top1 - 7.f : m1;
      const float al0 = mn0 == m0 ? 1.f : ex2_ftz(m0 - mn0), al1 = mn1 == m1 ? 1.f : ex2_ftz(m1 - mn1);
      m0 = mn0;
      m1 = mn1;
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] *= al0;
        o[i][1] *= al1;
        o[i][2] *= al0;
        o[i][3] *= al1;
      }
      z[0] *= al0;
      z[1] *= al1;
      z[2] *= al0;
      z[3] *= al1;
    }
    auto values = [&](int i) {
      const uint32_t rec = kt + i * kInt4Record;
      const float p0 = ex2_ftz(y[i][0] - m0), p1 = ex2_ftz(y[i][1] - m1);
      const float p2 = ex2_ftz(y[i][2] - m0), p3 = ex2_ftz(y[i][3] - m1);
      l0 = fmaf(p0, iv[i][0], fmaf(p2, iv[i][1], l0));
      l1 = fmaf(p1, iv[i][0], fmaf(p3, iv[i][1], l1));
      // B operand P^T: tokens 2cq, 2cq + 1 (+ 8) of head gq
      const uint32_t b0 = movmatrix_trans(pack_f16x2(p0, p1)), b1 = movmatrix_trans(pack_f16x2(p2, p3));
      const uint32_t za = (lds32(rec + kInt4VScales + 4 * cq) << 7) & kPairB;
      const uint32_t zb = (lds32(rec + kInt4VScales + 16 + 4 * cq) << 7) & kPairB;
      mma_f16_16816(z, za, za, zb, zb, b0, b1);
      // The transposing ldmatrix takes four codes for an element: lane (gq, cq) gets tokens 2cq and 2cq + 1 of
      // eight bytes' dims in the halves of a word, so that a masked pair is a pair along the tokens.
#pragma unroll
      for (int u = 0; u < 4; u += 2) {
        uint32_t w[4];
        ldsm_x4_trans(rec + v_row + (((u + v_unit) ^ v_turn) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u0 = w[2 * h] << 3, v0 = w[2 * h + 1] << 3, u1 = w[2 * h] >> 5, v1 = w[2 * h + 1] >> 5;
          mma_f16_16816(o[2 * (u + h)], u0 & kPairA, u0 & kPairB, v0 & kPairA, v0 & kPairB, b0, b1);
          mma_f16_16816(o[2 * (u + h) + 1], u1 & kPairA, u1 & kPairB, v1 & kPairA, v1 & kPairB, b0, b1);
        }
      }
    };
    if (full) {
#pragma unroll
      for (int i = 0; i < kDiJob; ++i) values(i);
    } else {
#pragma unroll
      for (int i = 0; i < kDiJob; ++i)
        if (i == 0 || two) values(i);
    }
    if (fl & kLast) {
      float L0 = l0, L1 = l1;                        // the 8 lanes sharing cq hold disjoint tokens
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        L0 += __shfl_xor_sync(kFullMask, L0, x);
        L1 += __shfl_xor_sync(kFullMask, L1, x);
      }
      const bool piece_whole = (fl & kWhole) != 0;
      // a sequence whose every block is out of range has L = 0 and gives zeros
      float f0 = piece_whole ? (L0 == 0.f ? 0.f : 1.f / L0) : 1.f, f1 = piece_whole ? (L1 == 0.f ? 0.f : 1.f / L1) : 1.f;
      if (far && !piece_whole) {
        // the merge's shift is one number: the base, and the rest goes into the sums (2^m, |m| of some 90 at most)
        if (m0 != kNoShift) f0 = ex2_ftz(m0), m0 = base0;
        if (m1 != kNoShift) f1 = ex2_ftz(m1), m1 = base1;
        L0 *= f0;
        L1 *= f1;
      }
      const size_t row = (piece_whole ? static_cast<size_t>(d.x) : static_cast<size_t>(d.z)) * G + 2 * cq;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // Column gq of the unit's eight has dims 8 (gq / 2) + gq % 2 + 2j, j = 0 .. 3.  Neighbouring columns
          // exchange two of them each and hold four dims in a row: 32u + 4gq .. + 3.
          const float zh = z[h], f = (h ? f1 : f0) * 0x1p17f;
          const float v0 = fmaf(o[2 * u][h], 16.f, -zh) * f, v1 = (o[2 * u][2 + h] - zh) * f;
          const float v2 = fmaf(o[2 * u + 1][h], 16.f, -zh) * f, v3 = (o[2 * u + 1][2 + h] - zh) * f;
          const bool odd = gq & 1;
          const float g0 = __shfl_xor_sync(kFullMask, odd ? v0 : v2, 4), g1 = __shfl_xor_sync(kFullMask, odd ? v1 : v3, 4);
          const float4 v = odd ? make_float4(g0, v2, g1, v3) : make_float4(v0, g0, v1, g1);
          if (2 * cq + h >= G) continue;
          if (piece_whole)
            *reinterpret_cast<uint2*>(a.out + (row + h) * kHeadDim + 32 * u + 4 * gq) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          else
            *reinterpret_cast<float4*>(a.ws_o + (row + h) * kHeadDim + 32 * u + 4 * gq) = v;
        }
      }
      if (!piece_whole && gq == 0) {
        if (2 * cq < G) a.ws_ml[row] = make_float2(m0, L0);
        if (2 * cq + 1 < G) a.ws_ml[row + 1] = make_float2(m1, L1);
      }
    }
    return two ? 2 : 1;
  };

  // ---------------------------------------------------------------- pipeline --------
  // The k-th use of a stage completes phase k & 1 of its barriers.
  uint32_t at = ring, bar = full_bars, phase = 0;
  for (int left = static_cast<int>(R.begin(my_v + 1) - R.begin(my_v)); left > 0;) {
    if (!__all_sync(kFullMask, *fail == 0 && mbar_wait_parked(bar, phase))) {
      if (lane == 0) {
        raise_flag(a.status, PA_FLAG_TIMEOUT);
        *fail = 1;
      }
      break;
    }
    left -= consume(at);
    fence_proxy_async_smem();   // what this warp read and wrote in the stage before the copies that follow
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + 8);
    at += stage_bytes;
    bar += 16;
    if (at == ring_end) {
      at = ring;
      bar = full_bars;
      phase ^= 1u;
    }
  }
}

// CTAs of the persistent grid: one per SM, capped to kMaxDecodeWarps ranges (looked up once per
// device, with the shared-memory opt-in of both variants).
cudaError_t int4_ctas(int* ctas) {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!cached[dev]) {
    auto opt_in = [&](auto kernel) {
      if (err == cudaSuccess)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDiSmemMax);
    };
    opt_in(decode_int4_kernel<false>);
    opt_in(decode_int4_kernel<true>);
    int sms = 0;
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    cached[dev] = min(sms, kMaxDecodeWarps / kDiConsumers);
  }
  *ctas = cached[dev];
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeArgs& args, cudaStream_t stream) {
  DecodeArgs a = args;
  const bool step = a.k_new != nullptr;
  int max_ctas = 0;
  cudaError_t err = int4_ctas(&max_ctas);
  if (err != cudaSuccess) return err;
  // Stages: what fits.
  const int G = a.num_q_heads / a.num_kv_heads;
  const int fixed = kDiPrefixOff + prefix_bytes(a.num_seqs);
  const int stage = di_stage(G, step);
  const int pool = (kDiSmemMax - fixed) / stage;
  // no more CTAs than there can be ranges (they are dealt to the CTAs one at a time)
  const long long jobs = static_cast<long long>(a.num_seqs) * a.num_kv_heads *
                         ((a.max_context_len + kBlockSize - 1) / kBlockSize);
  const long long ctas = min(static_cast<long long>(max_ctas), (jobs + kMinRangeBlocks - 1) / kMinRangeBlocks);
  a.num_warps = static_cast<int>(ctas) * kDiConsumers;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>((kDiConsumers + 1) * 32));
  cfg.dynamicSmemBytes = fixed + pool * stage;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, step ? decode_int4_kernel<true> : decode_int4_kernel<false>, a, pool);
  if (err != cudaSuccess) return err;
  return launch_block_merge(a, cfg);
}

}  // namespace pa
