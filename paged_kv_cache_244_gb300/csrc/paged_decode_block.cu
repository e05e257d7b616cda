// Single-token paged GQA decode attention over block-scaled E4M3 caches, for sm_103a, with the
// fused step (RoPE form + quantising store of the new token).
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现": §2 Kernel层 (PagedAttention decode kernel), §H200上的详细对比
// (Flash Decode); "从零实现 LLM 推理引擎：深挖 vLLM 的六大核心优化", §3.1 Paged KV Cache; "nano-vllm：vLLM
// 极简实现与大模型推理流程解析", §学习要点 (8-bit quantisation of the cache).
//
// The work is cut as in the decode over bf16 caches (pa_device.cuh): one axis of (sequence, KV
// head, block), an equal contiguous range for each warp of a persistent grid, pieces of split
// segments merged by a kernel after it.  A warp serves the G <= 8 query heads of its KV head
// and is its own producer and consumer.  What differs:
//
//   Jobs of two blocks.  A 2 KiB tile of codes is little work beside what a job costs whatever its
//   size (looking up, arming the barrier, issuing copies, waiting, testing the softmax's shift), so
//   a job takes two neighbouring blocks of its piece where it can: 8 KiB a stage.
//   q in f16 after a power of two that brings a head's largest magnitude to [128, 256), so that no
//   magnitude of q is out of f16's range: q = row_fold q', exact down to 2^-22 of the largest.  (The
//   E4M3 product of mma.sync takes K codes unwidened and q as a sum of two E4M3 vectors; it ran as
//   f16 products and conversions here, 400 instructions a tile against 300 for this form.)
//   Tiles by cp.async.  A stage is four scattered 2 KiB tiles.  TMA boxes of that size leave an SM
//   one in about 100 cycles whatever issues them, 20 bytes a cycle where HBM brings 23: issuing a
//   job's four took its warp 700 cycles (64 sequences of 64-4096 tokens, 32 / 8 heads: 64 us).  A
//   warp's 16-byte cp.async moves 512 bytes an instruction, each lane swizzling its own address.  A
//   warp waits for its own copies only, so there is no barrier: one commit group a job.  q of a
//   piece's first job, and the new token's rows and cos/sin row, come with its tiles, ahead of them
//   in the group: with 20 MB of tiles in flight on the GPU a load that follows them takes 4 us (read
//   by the lanes when a piece began, q held the first tiles of a lone call back by 5 us).
//   Scales on the scores.  With k_b, v_b the scales of token t's block:
//     x_t = scale_log2 k_b (q . Kcode_t) + log2 v_b,   p_t = 2^(x_t - m),
//     O = sum p_t Vcode_t,   L = sum p_t / v_b,   out = O / L.
//   Both sums carry 2^m, and v_b cancels in the second; pieces merge as any others do.  V codes
//   widen exactly to f16.  The shift m is set 7 below the largest contribution and moves when one
//   passes it by more than 15, so P lies within f16 whatever the scales, and whether it has to move
//   is one vote a job: the maximum over the tokens is formed only then.  L adds the unrounded fp32
//   p_t: a block of tiny V scale (an attention sink) may carry most of the weight with a p_t below
//   f16.
//
// What bounds it: 64 sequences of 64-4096 tokens, us replayed from a graph.  12 / 2 heads (66 MB): 18.4,
// of which some 2.5 before the first tile (lengths, table, tile: dependent cold reads), some 10 streaming at the
// copy rate, 2.4 between the first SM done and the last, the rest launch and merge; a kernel that only
// gathers the same tiles takes 13.7.  Fused step with 32 / 8 heads (276 MB): 50.6, 5.5 TB/s (gather 43.8).
// One sequence of 2048 tokens: 6.2, latency (an empty kernel: 1.9).
//
// Per stage: [K tile 0 | K tile 1 | V tile 0 | V tile 1 | q rows | (step) cos/sin row, k row, v row];
// 16-byte chunk c of row r of a tile (16 x 128 codes) lies at c ^ (r % 8) of its row.

#include <mutex>

#include "int4_launch.h"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kBdWarps = 12;                         // of a CTA at most (registers)
constexpr int kBdTile = kTileBytes / 2;              // 16 x 128 codes: 2 KiB
constexpr int kBdVOff = 2 * kBdTile;                 // V tiles after the two K tiles
constexpr int kBdQOff = 4 * kBdTile;
// A stage: tiles, q rows of G heads, and for the step cos/sin (R <= 128 floats), k and v.
__host__ __device__ inline int bd_stage(int G, bool step) {
  return kBdQOff + G * kHeadDim * 2 + (step ? kHeadDim * 4 + 2 * kHeadDim * 2 : 0);
}
constexpr int kBdMaxStages = 32;                     // of a CTA
constexpr int kBdMaxRing = 8;                        // of a warp
constexpr int kBdSmemMax = 226 * 1024;               // beside the static part of build_prefix

// Shared memory: int4 descriptors and float2 x 2 scales of every stage, the prefix, the stages.
constexpr int kBdScaleOff = kBdMaxStages * 16;
constexpr int kBdPrefixOff = kBdScaleOff + kBdMaxStages * 16;

// Codes are read evict-first (kOnce) from a pool of more than this, and with early metadata: tiles read once a
// call leave lengths, tables, partial results and the neighbouring kernels' data in L2.  Normal / evict-first,
// us: 64 sequences of 64-4096 tokens with 12 / 2 heads (66 MB) 19.0 / 18.3, the fused step with 32 / 8 heads
// (276 MB) 51.8 / 50.7; as one of several layers with a matrix product of 64 MB of weights between (its
// 12 us included) 31.5 / 30.8 and 65.4 / 63.9.  One sequence of 2048 tokens (1 MB) 6.07 / 6.18.  Against it: 32
// sequences that share all of a 16,384-token prefix (67 MB) 117.9 / 126.1, a prefix of 2048 tokens 17.6 / 17.6.
constexpr long long kOncePool = 32ll << 20;

// More job flags: which of the two blocks are there.
constexpr uint32_t kTwo = 1u << 13, kHas0 = 1u << 14, kHas1 = 1u << 15;

template <bool kStep, bool kOnce>
__global__ void __launch_bounds__(kBdWarps * 32, 1)
decode_block_kernel(const DecodeArgs a, const int pool) {
  extern __shared__ unsigned char smem_raw[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  int* prefix = reinterpret_cast<int*>(smem_raw + kBdPrefixOff);
  unsigned char* last_rows = smem_raw + kBdPrefixOff + (((a.num_seqs + 1) * 4 + 15) & ~15);
  const uint32_t tile_base = (raw + kBdPrefixOff + prefix_bytes(a.num_seqs) + 1023u) & ~1023u;
  // With early metadata the lengths and block table are read, and the work resolved, before the
  // preceding kernel has finished; copies and writes wait for it (below).
  const bool early = a.early_metadata != 0;
  if (!early) pdl_wait_prior_grid();
  pdl_allow_next_grid();

  const int S = a.num_seqs;
  const int Hkv = a.num_kv_heads;
  const int G = a.num_q_heads / Hkv;
  const int warps = static_cast<int>(blockDim.x >> 5);
  const int stage_bytes = bd_stage(G, kStep);
  const int cos_off = kBdQOff + G * kHeadDim * 2;    // (step)
  build_prefix<kBdWarps>(a, prefix, last_rows, blockDim.x);
  const long long T = static_cast<long long>(Hkv) * prefix[S];
  const Ranges R = make_ranges(T, a);
  // Range v goes to warp v / grid of CTA v % grid; the CTA's stages are shared out among its warps
  // that have a range, the first of them taking one more where they do not divide.
  const int my_v = static_cast<int>(blockIdx.x) + warp * static_cast<int>(gridDim.x);
  if (my_v >= R.V) {
    if (early) pdl_wait_prior_grid();
    return;
  }
  const int active = min(warps, (R.V - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                                       static_cast<int>(gridDim.x));
  const int share = pool / active + (warp < pool % active ? 1 : 0);
  const int st0 = warp * (pool / active) + min(warp, pool % active);
  const int n_st = min(share, kBdMaxRing);
  int4* descs = reinterpret_cast<int4*>(smem_raw) + st0;
  float4* scales = reinterpret_cast<float4*>(smem_raw + kBdScaleOff) + st0;  // (k0, v0, k1, v1)
  const uint32_t tiles = tile_base + st0 * stage_bytes;
  const int gq = lane >> 2;  // fragment row group
  const int cq = lane & 3;   // fragment column pair
  const int mi = lane >> 3;  // ldmatrix: matrix this lane addresses
  const int r = lane & 7;    // ldmatrix: row of that matrix
  const long long x0 = R.begin(my_v), x1 = R.begin(my_v + 1);

  // ---- lookahead: window = up to 32 consecutive blocks of the range, lane j resolves block j ----
  struct Window {
    long long x;
    int n;
    int blk, seg, fl, slot, pos;
  };
  auto resolve = [&](Window& W) {
    W.blk = -1;
    W.seg = W.fl = W.slot = W.pos = 0;
    if (lane >= W.n) return;
    const long long p = W.x + lane;
    int lo = 0, hi = S;                              // largest s with Hkv * N_s <= p
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<long long>(Hkv) * prefix[mid] <= p) lo = mid;
      else hi = mid;
    }
    const int s = lo;
    const int ns = prefix[s + 1] - prefix[s];
    const int off = static_cast<int>(p - static_cast<long long>(Hkv) * prefix[s]);
    const int g = off / ns;
    const int j = off - g * ns;
    const long long Xi = static_cast<long long>(Hkv) * prefix[s] + static_cast<long long>(g) * ns;
    W.blk = a.block_tables[static_cast<size_t>(s) * a.max_blocks + j];
    W.seg = s * Hkv + g;
    const int tail = last_rows[s];
    const int valid = j == ns - 1 ? tail : kBlockSize;
    const int chunk = a.chunk_blocks;
    const int part = chunk ? j / chunk : 0;
    const bool p_first = chunk && j == part * chunk;
    const bool p_last = chunk && j == part * chunk + chunk - 1;
    uint32_t flags = ((p == x0 || j == 0 || p_first) ? kFirst : 0u) |
                     ((p == x1 - 1 || j == ns - 1 || p_last) ? kLast : 0u) |
                     ((Xi >= x0 && Xi + ns <= x1 && (chunk == 0 || ns <= chunk)) ? kWhole : 0u) |
                     ((p == x0 && j > 0 && p_first) ? kGap : 0u);
    if (kStep) {
      W.pos = (ns - 1) * kBlockSize + tail - 1;      // position of the sequence's new token
      if (j == ns - 1) flags |= kNew;
      if (W.pos < a.max_pos) flags |= kRope;
    }
    W.fl = static_cast<int>(flags | (static_cast<uint32_t>(valid) << 8) | (static_cast<uint32_t>(g) << 16));
    W.slot = static_cast<int>(piece_slot(my_v, W.seg, part, a.max_parts));
  };
  auto next_of = [&](const Window& W, Window& N) {
    N.x = W.x + W.n;
    N.n = static_cast<int>(min(32ll, x1 - N.x));
  };
  Window cur, nxt;
  cur.x = x0;
  cur.n = static_cast<int>(min(32ll, x1 - x0));
  resolve(cur);
  next_of(cur, nxt);   // resolved behind the first jobs: a ring takes at most 16 of a window's 32 blocks
  static_assert(2 * kBdMaxRing < 32, "the first window outlasts the first jobs");
  int pk = 0;  // next block of `cur`
  uint64_t once = 0;
  if constexpr (kOnce) once = l2_evict_first_policy();
  // This lane's 16-byte chunks of a tile: chunk lane + 32 i, row (lane / 8) + 4 i, to its swizzled place.
  const uint32_t row0 = lane >> 3;
  const uint32_t to_even = row0 * 128 + (((lane & 7) ^ row0) << 4);          // i = 0, 2: row % 8 = lane / 8
  const uint32_t to_odd = row0 * 128 + (((lane & 7) ^ (row0 + 4)) << 4);     // i = 1, 3: + 4
  auto copy_tile = [&](uint32_t dst, const void* cache, int tile_row) {
    const char* src = static_cast<const char*>(cache) + static_cast<size_t>(tile_row) * kBdTile + lane * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t to = dst + i * 512 + ((i & 1) ? to_odd : to_even);
      if constexpr (kOnce) cp_async16_hint(to, src + i * 512, once);
      else cp_async16(to, src + i * 512);
    }
  };

  // Emit the next job into stage st, as one commit group; false when the range is used up.
  auto produce = [&](int st) -> bool {
    if (pk == cur.n) {
      if (nxt.n == 0) return false;
      cur = nxt;
      pk = 0;
      next_of(cur, nxt);
      resolve(nxt);
    }
    const int fl0 = __shfl_sync(kFullMask, cur.fl, pk);
    const bool two = !(fl0 & kLast) && pk + 1 < cur.n;
    const int blk0 = __shfl_sync(kFullMask, cur.blk, pk);
    const int fl1 = __shfl_sync(kFullMask, cur.fl, pk + (two ? 1 : 0));
    const int blk1 = __shfl_sync(kFullMask, cur.blk, pk + (two ? 1 : 0));
    const int seg = __shfl_sync(kFullMask, cur.seg, pk);
    const int slot = __shfl_sync(kFullMask, cur.slot, pk);
    const int pos = kStep ? __shfl_sync(kFullMask, cur.pos, pk) : 0;
    pk += two ? 2 : 1;
    const bool here0 = blk0 >= 0 && blk0 < a.num_blocks, here1 = two && blk1 >= 0 && blk1 < a.num_blocks;
    const int g = fl0 >> 16;
    const int row0 = blk0 * Hkv + g, row1 = blk1 * Hkv + g;   // (block, KV head) tiles
    const uint32_t dst = tiles + st * stage_bytes;
    // Fused step: a position without a cos/sin row leaves the token out -- q unrotated, nothing stored.
    const bool rope = kStep && (fl0 & kRope);
    const bool fresh = rope && (fl1 & kNew) && (two ? here1 : here0);       // the new token's tile is here
    if (fl0 & kFirst) {
      const char* q = reinterpret_cast<const char*>(a.q + static_cast<size_t>(seg) * G * kHeadDim);
      for (int c = lane; c < G * 16; c += 32) cp_async16(dst + kBdQOff + 16 * c, q + 16 * c);
    }
    if (kStep && rope && ((fl0 & kFirst) || fresh) && lane < a.rotary_dim / 4)
      cp_async16(dst + cos_off + 16 * lane, a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + 4 * lane);
    if (kStep && fresh) {
      const __nv_bfloat16* row = (lane < 16 ? a.k_new : a.v_new) + static_cast<size_t>(seg) * kHeadDim;
      cp_async16(dst + cos_off + kHeadDim * 4 + 16 * lane, row + 8 * (lane & 15));
    }
    if (here0) {
      copy_tile(dst, a.k_cache, row0);
      copy_tile(dst + kBdVOff, a.v_cache, row0);
    }
    if (here1) {
      copy_tile(dst + kBdTile, a.k_cache, row1);
      copy_tile(dst + kBdVOff + kBdTile, a.v_cache, row1);
    }
    if (lane < 2 && (lane ? here1 : here0)) cp_async8(smem_addr(scales + st) + lane * 8, a.kv_scale + (lane ? row1 : row0));
    cp_async_commit();
    if (lane == 0) {
      if (!here0 || (two && !here1)) raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
      if (kStep && (fl1 & kNew) && !rope) raise_flag(a.status, PA_FLAG_POSITION_OOB);
      // flags of the job: the first block's kFirst and kGap, the last one's kLast, kNew and rows
      const uint32_t fl = (static_cast<uint32_t>(fl0) & (kFirst | kGap | kWhole | kRope)) |
                          (static_cast<uint32_t>(fl1) & (kLast | 0x1f00u)) | (fresh ? kNew : 0u) |
                          (two ? kTwo : 0u) | (here0 ? kHas0 : 0u) | (here1 ? kHas1 : 0u);
      descs[st] = make_int4(seg, static_cast<int>(fl), slot, two ? row1 : row0);
    }
    return true;
  };

  // ---------------------------------------------------------------- consumer state --
  const uint32_t k_row = static_cast<uint32_t>((r + 8 * (mi & 1)) * 128);   // ldmatrix rows 0-7 / 8-15
  const int k_col = mi >> 1;                                                 // chunk 2c / 2c + 1
  uint32_t qb[8][2];                      // B operand: dims 16c + 4cq .. + 3 of head gq (k permuted, below)
  float kf0 = 0.f, kf1 = 0.f;             // softmax scale * row_fold of head columns 2cq, 2cq + 1
  float m0 = -INFINITY, m1 = -INFINITY;   // softmax shifts of those columns
  float l0 = 0.f, l1 = 0.f;               // this lane's share of L
  float o[8][4];                          // O^T: dims 16mt + 2gq (+1), heads 2cq, 2cq + 1

  // The new token (row `row` of tile `which` of the stage, whose cache tile is `tile_row`) is rotated
  // and coded into the staged tile and the cache.  Row 0 begins the block; otherwise a scale that
  // has to grow codes the whole tile anew, and the tile is written back.  Returns the scales after.
  auto store_new = [&](unsigned char* stage, int which, float2 held, int row, int tile_row) -> float2 {
    const float* cs = reinterpret_cast<const float*>(stage + cos_off);
    const uint32_t* kn = reinterpret_cast<const uint32_t*>(cs + kHeadDim);
    const uint32_t* vn = kn + kHeadDim / 2;
    const int rot = a.rotary_dim;
    // Lane l holds two words (dim pairs) of the row: of the half layout words l and l + R/4 for
    // l < R/4, otherwise words 2l and 2l + 1; the first R/4 lanes rotate theirs.
    const bool turns = lane < rot / 4;
    const int wa = turns && !a.interleaved ? lane : 2 * lane;
    const int wb = turns && !a.interleaved ? lane + rot / 4 : 2 * lane + 1;
    uint32_t kx = kn[wa], ky = kn[wb];
    if (turns) {
      const float2 co = reinterpret_cast<const float2*>(cs)[lane];
      const float2 si = reinterpret_cast<const float2*>(cs + rot / 2)[lane];
      if (a.interleaved) rope_rotate_interleaved(kx, ky, co, si);
      else rope_rotate_pairs(kx, ky, co, si);
    }
    const uint32_t vx = vn[wa], vy = vn[wb];
    const uint32_t km = __vmaxu2(finite_magnitudes(kx), finite_magnitudes(ky));
    const uint32_t vm = __vmaxu2(finite_magnitudes(vx), finite_magnitudes(vy));
    const uint32_t ktop = __reduce_max_sync(kFullMask, max(km & 0xffffu, km >> 16));
    const uint32_t vtop = __reduce_max_sync(kFullMask, max(vm & 0xffffu, vm >> 16));
    const bool begins = row == 0;
    const float2 now = make_float2(e4m3_grow_scale(held.x, e4m3_scale_for(ktop), begins),
                                   e4m3_grow_scale(held.y, e4m3_scale_for(vtop), begins));
    // byte 2w of the row, through the 128-byte swizzle
    auto at = [&](int w) { return row * 128 + (((w >> 3) ^ (row & 7)) << 4) + 2 * (w & 7); };
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      const float old = kv ? held.y : held.x, s = kv ? now.y : now.x;
      const float inv = __frcp_rn(s);
      const uint16_t cx = e4m3x2_of(kv ? vx : kx, inv), cy = e4m3x2_of(kv ? vy : ky, inv);
      unsigned char* tile = stage + kv * kBdVOff + which * kBdTile;
      uint8_t* cache = reinterpret_cast<uint8_t*>(kv ? a.v_store : a.k_store) + static_cast<size_t>(tile_row) * kBdTile;
      const bool grown = !begins && s != old;
      if (grown) {
        const float f = __fdiv_rn(old, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* w = reinterpret_cast<uint4*>(tile) + lane + 32 * i;
          *w = e4m3x16_rescale(*w, f);
        }
        __syncwarp();
      }
      *reinterpret_cast<uint16_t*>(tile + at(wa)) = cx;
      *reinterpret_cast<uint16_t*>(tile + at(wb)) = cy;
      if (grown) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = lane + 32 * i, rr = c >> 3;  // 16-byte chunk c of the tile
          reinterpret_cast<uint4*>(cache)[rr * 8 + ((c & 7) ^ (rr & 7))] = reinterpret_cast<const uint4*>(tile)[c];
        }
      } else {
        uint16_t* dst = reinterpret_cast<uint16_t*>(cache + row * kHeadDim);
        dst[wa] = cx;
        dst[wb] = cy;
      }
    }
    if (lane == 0) a.kv_scale_store[tile_row] = now;
    __syncwarp();
    return now;
  };

  // q rows of the piece: rotated (step), scaled and rounded to f16.
  auto load_q = [&](const unsigned char* stage, uint32_t fl) {
    const uint2* qrow = reinterpret_cast<const uint2*>(stage + kBdQOff + (gq < G ? gq : 0) * kHeadDim * 2);
    uint2 w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = gq < G ? qrow[4 * c + cq] : make_uint2(0u, 0u);
    if (kStep && (fl & kRope)) {
      const int rot = a.rotary_dim, half = rot / 2;
      const float* cs = reinterpret_cast<const float*>(stage + cos_off);
      if (!a.interleaved && rot == kHeadDim) {       // partners 64 dims away, in the same lane
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int dd = 16 * c + 4 * cq;
          rope_rotate_pairs(w[c].x, w[c + 4].x, *reinterpret_cast<const float2*>(cs + dd),
                            *reinterpret_cast<const float2*>(cs + 64 + dd));
          rope_rotate_pairs(w[c].y, w[c + 4].y, *reinterpret_cast<const float2*>(cs + dd + 2),
                            *reinterpret_cast<const float2*>(cs + 66 + dd));
        }
      } else {
        // dims d .. d + 3 (d = 16c + 4cq) rotate if d < R: within the word pair when interleaved, else
        // with the dims R/2 away, read from its row
        const uint32_t* row = reinterpret_cast<const uint32_t*>(qrow);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int d = 16 * c + 4 * cq;
          if (d >= rot || gq >= G) continue;
          if (a.interleaved) {
            rope_rotate_interleaved(w[c].x, w[c].y, *reinterpret_cast<const float2*>(cs + d / 2),
                                    *reinterpret_cast<const float2*>(cs + half + d / 2));
          } else {
            const int i = d < half ? d : d - half;   // angle of the first dim
            const int other_dim = d < half ? d + half : i;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t own = e ? w[c].y : w[c].x, other = row[other_dim / 2 + e];
              const float2 co = *reinterpret_cast<const float2*>(cs + i + 2 * e);
              const float2 si = *reinterpret_cast<const float2*>(cs + half + i + 2 * e);
              if (d < half) rope_rotate_pairs(own, other, co, si);
              else rope_rotate_pairs(other, own, co, si);
              (e ? w[c].y : w[c].x) = own;
            }
          }
        }
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) top = __vmaxu2(top, __vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu));
    top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, 2));
    top = max(top & 0xffffu, top >> 16);             // the head's largest magnitude
    // to [128, 256); below 2^-119 not as far: multiples of 2^-133 become multiples of 2^-7, exact all the same
    const int e = min(7 + 127 - static_cast<int>(top >> 7), 126);
    const float raise = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      qb[c][0] = pack_f16x2(bf16lo(w[c].x) * raise, bf16hi(w[c].x) * raise);
      qb[c][1] = pack_f16x2(bf16lo(w[c].y) * raise, bf16hi(w[c].y) * raise);
    }
    // an infinity or a NaN makes the head's scores NaN
    const float fold = top >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                      : row_factor(a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23));
    kf0 = __shfl_sync(kFullMask, fold, 8 * cq);
    kf1 = __shfl_sync(kFullMask, fold, 8 * cq + 4);
  };

  auto consume = [&](int st) {
    const int4 d = descs[st];
    const uint32_t fl = static_cast<uint32_t>(d.y);
    const uint32_t kt = tiles + st * stage_bytes;
    unsigned char* const stage = smem_raw + (kt - raw);
    if (fl & kFirst) {
      load_q(stage, fl);
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
      if ((fl & kGap) && lane < G)                   // mark the skipped slot before this piece empty
        a.ws_ml[(static_cast<size_t>(d.z) - 1) * G + lane] = make_float2(-INFINITY, 0.f);
      __syncwarp();                                  // some lanes have stored; what follows wants the whole warp
    }
    const bool two = (fl & kTwo) != 0;
    float4 sv = scales[st];
    if (!(fl & kHas0)) sv.x = sv.y = 1.f;            // absent tiles: the slot holds anything
    if (!(fl & kHas1)) sv.z = sv.w = 1.f;
    const int valid = static_cast<int>((fl >> 8) & 0x1fu);   // rows of the job's last block
    if (kStep && (fl & kNew)) {
      const float2 now = store_new(stage, two ? 1 : 0, two ? make_float2(sv.z, sv.w) : make_float2(sv.x, sv.y),
                                   valid - 1, d.w);
      if (two) {
        sv.z = now.x;
        sv.w = now.y;
      } else {
        sv.x = now.x;
        sv.y = now.y;
      }
    }
    // S^T = Kcode q^T of both tiles, even and odd steps of k in chains of their own (the MMAs issue in
    // order).  ldmatrix reads the codes as 16-bit pairs, so lane (gq, cq) of matrix (rows 8h .. 8h + 7,
    // 16-byte chunk c) gets dims 16c + 4cq .. + 3 of token 8h + gq: widened to two f16 pairs they are
    // the A fragments of k indices (2cq, 2cq + 1) and (2cq + 8, 2cq + 9), the same permutation of the 16
    // dims as in qb.
    float s[2][4], t[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = t[0][i] = t[1][i] = 0.f;
    auto scores = [&](int i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w0, w1, w2, w3, lo0, hi0, lo1, hi1;
        ldsm_x4(kt + i * kBdTile + k_row + (((2 * c + k_col) ^ r) << 4), w0, w1, w2, w3);
        e4m3x4_to_f16x2x2(w0, lo0, hi0);
        e4m3x4_to_f16x2x2(w1, lo1, hi1);
        mma_f16_16816(s[i], lo0, lo1, hi0, hi1, qb[2 * c][0], qb[2 * c][1]);
        e4m3x4_to_f16x2x2(w2, lo0, hi0);
        e4m3x4_to_f16x2x2(w3, lo1, hi1);
        mma_f16_16816(t[i], lo0, lo1, hi0, hi1, qb[2 * c + 1][0], qb[2 * c + 1][1]);
      }
    };
    scores(0);
    if (two) scores(1);
    // [0] = (token gq, head 2cq), [1] = (gq, 2cq + 1), [2] = (gq + 8, 2cq), [3] = (gq + 8, 2cq + 1)
    const uint32_t all = two ? (kHas0 | kHas1) : kHas0;
    const bool whole_tiles = two && (fl & all) == all && valid == kBlockSize;
    const int n0 = (fl & kHas0) ? (two ? kBlockSize : valid) : 0;   // live tokens of each tile
    const int n1 = (fl & kHas1) ? valid : 0;
    float f00 = kf0 * sv.x, f01 = kf1 * sv.x, f10 = kf0 * sv.z, f11 = kf1 * sv.z;
    float e0 = log2_of(sv.y), e1 = log2_of(sv.w);
    float y[2][4];
    if (fmaxf(fmax3(f00, f01, f10), f11) > kFarFactor) {   // exponents in two steps
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[0][i] = fmaf(s[0][i] + t[0][i], (i & 1) ? f01 : f00, e0);
        s[1][i] = fmaf(s[1][i] + t[1][i], (i & 1) ? f11 : f10, e1);
        t[0][i] = t[1][i] = 0.f;
      }
      f00 = f01 = f10 = f11 = 1.f;
      e0 = e1 = 0.f;
    }
    __syncwarp();                                    // heads differ in it; the matrix instructions want the whole warp
    auto exponents = [&](float sh0, float sh1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[0][i] = fmaf(s[0][i] + t[0][i], (i & 1) ? f01 : f00, e0 - ((i & 1) ? sh1 : sh0));
        y[1][i] = fmaf(s[1][i] + t[1][i], (i & 1) ? f11 : f10, e1 - ((i & 1) ? sh1 : sh0));
      }
      if (!whole_tiles) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = gq + (i >> 1) * 8;
          if (tok >= n0) y[0][i] = -INFINITY;
          if (tok >= n1) y[1][i] = -INFINITY;
        }
      }
    };
    exponents(m0, m1);
    const float top = fmaxf(fmax3(fmaxf(y[0][0], y[0][1]), y[0][2], y[0][3]), fmax3(fmaxf(y[1][0], y[1][1]), y[1][2], y[1][3]));
    if (__any_sync(kFullMask, top > 15.f)) {
      // A shift has to move (at a piece's first job from -infinity): the maxima over the 32 tokens,
      // and what was summed so far scaled to the new shifts.
      exponents(0.f, 0.f);
      float b0 = fmaxf(fmaxf(y[0][0], y[0][2]), fmaxf(y[1][0], y[1][2]));
      float b1 = fmaxf(fmaxf(y[0][1], y[0][3]), fmaxf(y[1][1], y[1][3]));
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        b0 = fmaxf(b0, __shfl_xor_sync(kFullMask, b0, x));
        b1 = fmaxf(b1, __shfl_xor_sync(kFullMask, b1, x));
      }
      const float mn0 = b0 - m0 > 15.f ? b0 - 7.f : m0, mn1 = b1 - m1 > 15.f ? b1 - 7.f : m1;
      const float al0 = mn0 == m0 ? 1.f : ex2_ftz(m0 - mn0), al1 = mn1 == m1 ? 1.f : ex2_ftz(m1 - mn1);
      m0 = mn0;
      m1 = mn1;
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        o[mt][0] *= al0;
        o[mt][1] *= al1;
        o[mt][2] *= al0;
        o[mt][3] *= al1;
      }
      exponents(m0, m1);
    }
    uint32_t pb[2][2];                               // B operand P^T: tokens 2cq, 2cq + 1 (+8) of head gq
    const float iv0 = rcp_ftz(sv.y), iv1 = rcp_ftz(sv.w);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p0 = ex2_ftz(y[i][0]), p1 = ex2_ftz(y[i][1]), p2 = ex2_ftz(y[i][2]), p3 = ex2_ftz(y[i][3]);
      const float iv = i ? iv1 : iv0;
      l0 = fmaf(p0 + p2, iv, l0);
      l1 = fmaf(p1 + p3, iv, l1);
      pb[i][0] = movmatrix_trans(pack_f16x2(p0, p1));
      pb[i][1] = movmatrix_trans(pack_f16x2(p2, p3));
    }
    // O^T += V^T P^T.  The transposing ldmatrix of the V tile gives lane (gq, cq) the bytes
    // V[2cq][2gq], V[2cq][2gq+1], V[2cq+1][2gq], V[2cq+1][2gq+1] of one 16-dim chunk: regrouped by
    // dim and widened they are the A fragments of rows gq (dim 2gq) and gq + 8 (dim 2gq + 1).
    auto pv = [&](int i, uint32_t mask_lo, uint32_t mask_hi) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w0, w1, w2, w3;
        ldsm_x4_trans(kt + kBdVOff + i * kBdTile + k_row + (((2 * c + k_col) ^ r) << 4), w0, w1, w2, w3);
        uint32_t x0, y0, x1, y1;
        e4m3x4_pairs_to_f16(w0, x0, y0);
        e4m3x4_pairs_to_f16(w1, x1, y1);
        mma_f16_16816(o[2 * c], x0 & mask_lo, y0 & mask_lo, x1 & mask_hi, y1 & mask_hi, pb[i][0], pb[i][1]);
        e4m3x4_pairs_to_f16(w2, x0, y0);
        e4m3x4_pairs_to_f16(w3, x1, y1);
        mma_f16_16816(o[2 * c + 1], x0 & mask_lo, y0 & mask_lo, x1 & mask_hi, y1 & mask_hi, pb[i][0], pb[i][1]);
      }
    };
    if (whole_tiles) {
      pv(0, 0xffffffffu, 0xffffffffu);
      pv(1, 0xffffffffu, 0xffffffffu);
    } else {
      // rows past the context, and absent tiles, may hold anything (even NaN): zeros in the operand
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = i ? n1 : n0;
        if (n == 0) continue;
        pv(i, (2 * cq < n ? 0x0000ffffu : 0u) | (2 * cq + 1 < n ? 0xffff0000u : 0u),
           (2 * cq + 8 < n ? 0x0000ffffu : 0u) | (2 * cq + 9 < n ? 0xffff0000u : 0u));
      }
    }
    if (fl & kLast) {
      float L0 = l0, L1 = l1;                        // the 8 lanes sharing cq hold disjoint tokens
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        L0 += __shfl_xor_sync(kFullMask, L0, x);
        L1 += __shfl_xor_sync(kFullMask, L1, x);
      }
      const bool h0 = 2 * cq < G, h1 = 2 * cq + 1 < G;
      if (fl & kWhole) {
        // a sequence whose every block is out of range has L = 0 and gives zeros
        const float i0 = L0 == 0.f ? 0.f : 1.f / L0, i1 = L1 == 0.f ? 0.f : 1.f / L1;
        uint32_t* orow0 = reinterpret_cast<uint32_t*>(a.out + (static_cast<size_t>(d.x) * G + 2 * cq) * kHeadDim);
        uint32_t* orow1 = orow0 + kHeadDim / 2;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          if (h0) orow0[8 * mt + gq] = pack_bf16x2(o[mt][0] * i0, o[mt][2] * i0);
          if (h1) orow1[8 * mt + gq] = pack_bf16x2(o[mt][1] * i1, o[mt][3] * i1);
        }
      } else {
        const size_t row0 = static_cast<size_t>(d.z) * G + 2 * cq;
        float2* w0 = reinterpret_cast<float2*>(a.ws_o + row0 * kHeadDim) + gq;
        float2* w1 = w0 + kHeadDim / 2;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          if (h0) w0[8 * mt] = make_float2(o[mt][0], o[mt][2]);
          if (h1) w1[8 * mt] = make_float2(o[mt][1], o[mt][3]);
        }
        if (gq == 0) {
          if (h0) a.ws_ml[row0] = make_float2(m0, L0);
          if (h1) a.ws_ml[row0 + 1] = make_float2(m1, L1);
        }
      }
    }
  };

  // ---------------------------------------------------------------- pipeline --------
  int ahead = 0;           // jobs emitted and not yet consumed
  int pst = 0, cst = 0;
  bool more = true;
  if (early) pdl_wait_prior_grid();
  while (more && ahead < n_st) {
    more = produce(pst);
    if (more) {
      ++ahead;
      if (++pst == n_st) pst = 0;
    }
  }
  resolve(nxt);
  __syncwarp();
  while (ahead > 0) {
    cp_async_wait_but(ahead - 1);      // the oldest job's copies; the warp barrier shows them to every lane
    __syncwarp();
    consume(cst);
    --ahead;
    if (++cst == n_st) cst = 0;
    __syncwarp();
    if (more) {
      more = produce(pst);
      if (more) {
        ++ahead;
        if (++pst == n_st) pst = 0;
      }
    }
    __syncwarp();
  }
}

// Merge of the pieces of split segments: kGroups warps take one (sequence, query head), a lane four of its
// dims, a warp a contiguous share of the pieces with all rows of 8 or 16 pieces asked for at once; the warps'
// (M, L, acc) are joined in order.  out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) L_p; a gap (shift
// -inf, sum 0) weighs nothing and its row, never written, is not used.  A piece whose shift stayed at -inf
// over a sum that is not 0 met NaN only, and passes it on.
//
// The partition kernel's registers fill an SM, so the merge runs after it and its own length counts: the
// dependent round trips (lengths, (m, L) and rows) and the instructions of warps with few pieces each.  Four
// warps a pair: six CTAs an SM take the 768 pairs of 64 sequences with 12 heads in one wave (call 19.5 us;
// 19.9 with the 64 registers that eight want, 20.9 where the compiler chooses).
constexpr int kMergeCta = 4;        // warps of a CTA at least
// Warps of a pair, 16, 4 or 1, by the number of pairs: the fewer there are the more pieces each has, and the
// more warps the GPU has room for.  Contexts of 2000-2900 tokens, us of the whole call with 16 / 4 / 1:
// 96 pairs 9.3 / 11.7 / 16.3, 192: 11.0 / 12.3 / 16.4, 384: 15.4 / 13.5 / 15.7, 768: 22.8 / 17.0 / 18.3,
// 1200: 38.3 / 30.3 / 28.6, 2048: 74.2 / 61.2 / 58.3.  (Even contexts: one sequence far longer than the others has
// pieces that this does not see; 60,000 tokens among 199 sequences of 64, 8 / 1 heads: 89.6 us, 11.3 where the same
// tokens lie in equal sequences.)
constexpr int kWidePairs = 304, kMidPairs = 1024;

template <int kGroups>
__global__ void __launch_bounds__((kGroups > kMergeCta ? kGroups : kMergeCta) * 32, kGroups == kMergeCta ? 6 : 1)
decode_block_merge_kernel(const DecodeArgs a) {
  constexpr int kPairs = kGroups > kMergeCta ? 1 : kMergeCta / kGroups;   // of a CTA
  constexpr int kMergeRows = kGroups > 1 ? 8 : 16;                        // pieces of a round trip
  __shared__ float4 s_acc[kGroups > 1 ? kPairs * kGroups : 1][32];
  __shared__ float2 s_ml[kGroups > 1 ? kPairs * kGroups : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp % kGroups;
  const int S = a.num_seqs, Hq = a.num_q_heads, Hkv = a.num_kv_heads;
  const int w = blockIdx.x * kPairs + warp / kGroups;                     // (sequence, query head)
  const int G = Hq / Hkv;
  const int s = w / Hq, h = w - s * Hq, g = h / G;
  int before = 0, total = 0, ns = 0;
  if (w < S * Hq) {
    for (int t = lane; t < S; t += 32) {
      const int n = (clamp_len(a.context_lens[t], a.max_context_len) + kBlockSize - 1) / kBlockSize;
      total += n;
      if (t < s) before += n;
    }
    ns = (clamp_len(a.context_lens[s], a.max_context_len) + kBlockSize - 1) / kBlockSize;
    before = __reduce_add_sync(kFullMask, before);
    total = __reduce_add_sync(kFullMask, total);
  }
  uint2* const orow = reinterpret_cast<uint2*>(a.out + static_cast<size_t>(w) * kHeadDim) + lane;
  int k0 = 0, k1 = 0, npieces = 0;
  const float2* ml = nullptr;
  const float4* rows = nullptr;
  if (ns > 0) {
    const Ranges R = make_ranges(static_cast<long long>(Hkv) * total, a);
    const long long Xi = static_cast<long long>(Hkv) * before + static_cast<long long>(g) * ns;
    const int v_first = R.owner(Xi), v_last = R.owner(Xi + ns - 1);
    npieces = v_last - v_first + (a.chunk_blocks ? (ns - 1) / a.chunk_blocks : 0) + 1;
    const size_t row = static_cast<size_t>(piece_slot(v_first, s * Hkv + g, 0, a.max_parts)) * G + (h - g * G);
    ml = a.ws_ml + row;
    rows = reinterpret_cast<const float4*>(a.ws_o + row * kHeadDim) + lane;
    k0 = static_cast<int>(static_cast<long long>(grp) * npieces / kGroups);
    k1 = static_cast<int>(static_cast<long long>(grp + 1) * npieces / kGroups);
  }
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  // one piece: written directly by the partition kernel
  const bool merges = npieces > 1;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = k0; merges && base < k1; base += kMergeRows) {
    const int n = min(kMergeRows, k1 - base);
    const float2 mine = lane < n ? ml[(base + lane) * static_cast<size_t>(G)] : make_float2(-INFINITY, 0.f);
    float4 r[kMergeRows];
#pragma unroll
    for (int c = 0; c < kMergeRows; c += 4) {
      if (c < n) {
#pragma unroll
        for (int u = c; u < c + 4; ++u)
          if (u < n) r[u] = rows[static_cast<size_t>(base + u) * G * (kHeadDim / 4)];
      }
    }
    float Mb = mine.x;
#pragma unroll
    for (int x = kMergeRows / 2; x > 0; x >>= 1) Mb = fmaxf(Mb, __shfl_xor_sync(kFullMask, Mb, x));
    Mb = __shfl_sync(kFullMask, Mb, 0);
    const float Mn = fmaxf(M, Mb);
    const float rescale = M == -INFINITY ? 1.f : exp2f(M - Mn);           // 1: nothing but zeros or NaN so far
    M = Mn;
    const float wmine = mine.x == -INFINITY ? (mine.y == 0.f ? 0.f : mine.y) : exp2f(mine.x - M);
    float lb = wmine * mine.y;
#pragma unroll
    for (int x = kMergeRows / 2; x > 0; x >>= 1) lb += __shfl_xor_sync(kFullMask, lb, x);
    L = fmaf(L, rescale, __shfl_sync(kFullMask, lb, 0));
    acc.x *= rescale;
    acc.y *= rescale;
    acc.z *= rescale;
    acc.w *= rescale;
#pragma unroll
    for (int c = 0; c < kMergeRows; c += 4) {
      if (c < n) {
#pragma unroll
        for (int u = c; u < c + 4; ++u) {
          const float wu = __shfl_sync(kFullMask, wmine, u);              // 0 past the last piece
          if (wu != 0.f) {
            acc.x = fmaf(wu, r[u].x, acc.x);
            acc.y = fmaf(wu, r[u].y, acc.y);
            acc.z = fmaf(wu, r[u].z, acc.z);
            acc.w = fmaf(wu, r[u].w, acc.w);
          }
        }
      }
    }
  }
  if constexpr (kGroups > 1) {
    s_acc[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    if (grp != 0) return;
    // lane q weighs group q (one without pieces, or with gaps alone, has L = 0); the sum in their order
    const float2 o = lane < kGroups ? s_ml[warp + lane] : make_float2(-INFINITY, 0.f);
    M = o.x;
#pragma unroll
    for (int x = kGroups / 2; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, x));
    M = __shfl_sync(kFullMask, M, 0);
    const float mine = o.x == -INFINITY ? (o.y == 0.f ? 0.f : o.y) : exp2f(o.x - M);
    L = mine * o.y;
#pragma unroll
    for (int x = kGroups / 2; x > 0; x >>= 1) L += __shfl_xor_sync(kFullMask, L, x);
    L = __shfl_sync(kFullMask, L, 0);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const float wq = __shfl_sync(kFullMask, mine, q);
      const float4 v = s_acc[warp + q][lane];
      acc.x = fmaf(wq, v.x, acc.x);
      acc.y = fmaf(wq, v.y, acc.y);
      acc.z = fmaf(wq, v.z, acc.z);
      acc.w = fmaf(wq, v.w, acc.w);
    }
  }
  if (w >= S * Hq || (ns > 0 && !merges)) return;
  // no context, or a sequence whose every block is out of range: zeros
  const float i = L == 0.f ? 0.f : 1.f / L;
  *orow = make_uint2(pack_bf16x2(acc.x * i, acc.y * i), pack_bf16x2(acc.z * i, acc.w * i));
}

// CTAs of the persistent grid: one per SM, capped to kMaxDecodeWarps warps (looked up once per
// device, with the shared-memory opt-in of every variant).
cudaError_t block_ctas(int* ctas) {
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
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBdSmemMax);
    };
    opt_in(decode_block_kernel<false, false>);
    opt_in(decode_block_kernel<true, false>);
    opt_in(decode_block_kernel<true, true>);
    opt_in(decode_block_kernel<false, true>);
    int sms = 0;
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    cached[dev] = min(sms, kMaxDecodeWarps / kBdWarps);
  }
  *ctas = cached[dev];
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode_block(const DecodeArgs& args, cudaStream_t stream) {
  DecodeArgs a = args;
  const bool step = a.k_new != nullptr;
  int max_ctas = 0;
  cudaError_t err = block_ctas(&max_ctas);
  if (err != cudaSuccess) return err;
  // Stages: what fits (24 of 9 KiB without the step and 4 query heads a group, 20 of 10.5 KiB with it and
  // 6; fewer beside the prefix of thousands of sequences).  Warps: two of the step's stages each, 12 at
  // most, with and without the step, so that both cut sequences alike and give the same bits (64 sequences of
  // 64-4096 tokens, 6 heads a group: 10 warps and 11 within 1%).
  const int G = a.num_q_heads / a.num_kv_heads;
  const int fixed = kBdPrefixOff + prefix_bytes(a.num_seqs) + 1024;
  const int stage = bd_stage(G, step);
  const int pool = min(kBdMaxStages, (kBdSmemMax - fixed) / stage);
  const int warps = min(kBdWarps, (kBdSmemMax - fixed) / bd_stage(G, true) / 2);
  // no more CTAs than there can be ranges (they are dealt to the CTAs one at a time)
  const long long jobs = static_cast<long long>(a.num_seqs) * a.num_kv_heads *
                         ((a.max_context_len + kBlockSize - 1) / kBlockSize);
  const long long ctas = min(static_cast<long long>(max_ctas), (jobs + kMinRangeBlocks - 1) / kMinRangeBlocks);
  a.num_warps = static_cast<int>(ctas) * warps;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(warps * 32));
  cfg.dynamicSmemBytes = fixed + pool * stage;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long pool_bytes = static_cast<long long>(a.num_blocks) * a.num_kv_heads * 2 * kBdTile;
  const bool once = a.early_metadata || pool_bytes > kOncePool;
  auto kernel = step ? (once ? decode_block_kernel<true, true> : decode_block_kernel<true, false>)
                     : (once ? decode_block_kernel<false, true> : decode_block_kernel<false, false>);
  err = cudaLaunchKernelEx(&cfg, kernel, a, pool);
  if (err != cudaSuccess) return err;
  return launch_block_merge(a, cfg);
}

cudaError_t launch_block_merge(const DecodeArgs& a, cudaLaunchConfig_t cfg) {
  const long long pairs = static_cast<long long>(a.num_seqs) * a.num_q_heads;
  const int groups = pairs <= kWidePairs ? 16 : pairs <= kMidPairs ? 4 : 1;
  const int per_cta = groups > kMergeCta ? groups : kMergeCta;
  cfg.gridDim = dim3(static_cast<unsigned>((pairs * groups + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(static_cast<unsigned>(per_cta * 32));
  cfg.dynamicSmemBytes = 0;
  auto merge = groups == 16 ? decode_block_merge_kernel<16>
               : groups == 4 ? decode_block_merge_kernel<4> : decode_block_merge_kernel<1>;
  return cudaLaunchKernelEx(&cfg, merge, a);
}

}  // namespace pa
