// The fused RoPE + quantising store into the 4-bit cache, and reading cached rows back, for sm_103a.
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现", §1 模型实现层 (RoPE) and §2 Kernel层 (RoPE fused with
// the KV cache store); "从零实现 LLM 推理引擎：深挖 vLLM 的六大核心优化", §3.1 (16-token blocks);
// "nano-vllm：vLLM 极简实现与大模型推理流程解析", §学习要点 (4-bit quantisation).
//
// A token's scales are its own, so a row is quantised by the lanes that hold it and touches nothing of
// its block's other tokens: the store is the bf16 store of a RoPE form (eight lanes a head vector, four
// vectors a pass) with a few bytes out in the place of a row.
//
// Bound: rows in, q and codes out.  23,738 rows of 32 / 8 heads (525 MB with a cos/sin row each; 77 us at the copy rate)
// take 85.2 us, 6.16 TB/s.  The row's arithmetic (3,000 warp instructions a token, extremes and codes most of them) fills 70%
// of the issue slots, so a warp's next rows have to be on their way meanwhile: by cp.async, six passes ahead.  (Rows of two
// passes asked for at once and waited for 95.7; their registers loaded again as soon as a pass is done 112, as the compiler
// then waits for them before the next; three to eight passes ahead 84.5 - 86.5.)  256 rows of 12 / 2 heads: 2.8 us, an
// empty kernel's 1.9 and the load latencies.  18 warps an SM, so that none spills: 16, 20 - 24, 32 warps 86.5, 85.6 - 90.7,
// 91.7.  CTAs of two warps, as a token that is done makes room for the next (of 8: 2% more, and 3.1 for 256 rows); warps
// that go through tokens in a fixed order 99 - 113.

#include "int4_cache.cuh"
#include "int4_launch.h"
#include "rope_form.cuh"

namespace pa {
namespace {

constexpr int kStoreWarps = 2;

template <bool kInterleaved>
__device__ __forceinline__ void int4_rotate_chunks(uint4& x, uint4& y, const Angles& a) {
  const float2 c[4] = {{a.c0.x, a.c0.y}, {a.c0.z, a.c0.w}, {a.c1.x, a.c1.y}, {a.c1.z, a.c1.w}};
  const float2 s[4] = {{a.s0.x, a.s0.y}, {a.s0.z, a.s0.w}, {a.s1.x, a.s1.y}, {a.s1.z, a.s1.w}};
  uint32_t lo[4] = {x.x, x.y, x.z, x.w}, hi[4] = {y.x, y.y, y.z, y.w};
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {                   // word pairs (x.x, x.y), (x.z, x.w), (y.x, y.y), (y.z, y.w)
      const uint32_t u = i == 0 ? x.x : i == 1 ? x.z : i == 2 ? y.x : y.z, v = i == 0 ? x.y : i == 1 ? x.w : i == 2 ? y.y : y.w;
      lo[i] = __byte_perm(u, v, 0x5410);
      hi[i] = __byte_perm(u, v, 0x7632);
    }
  }
  uint32_t p[4], q[4], border = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = lo[i];
    q[i] = hi[i];
    int4_rotate_pairs(p[i], q[i], c[i], s[i], border);
  }
  if (at_border(border)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) int4_rotate_exactly(lo[i], hi[i], c[i], s[i], p[i], q[i]);
  }
  if constexpr (kInterleaved) {
    x = make_uint4(__byte_perm(p[0], q[0], 0x5410), __byte_perm(p[0], q[0], 0x7632), __byte_perm(p[1], q[1], 0x5410),
                   __byte_perm(p[1], q[1], 0x7632));
    y = make_uint4(__byte_perm(p[2], q[2], 0x5410), __byte_perm(p[2], q[2], 0x7632), __byte_perm(p[3], q[3], 0x5410),
                   __byte_perm(p[3], q[3], 0x7632));
  } else {
    x = make_uint4(p[0], p[1], p[2], p[3]);
    y = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// One warp, one token: its pairs of passes of four head vectors part, part + parts, ..: queries rotated into q_out, keys
// (rotated) and values quantised into the token's slot.  Rows come by cp.async, kStoreAhead passes ahead, and every lane
// reads the chunks that it asked for.
constexpr int kStoreAhead = 6;
static_assert(kStoreAhead <= 8, "groups that a wait can name");

template <bool kInterleaved>
__global__ void __launch_bounds__(kStoreWarps * 32, 18 / kStoreWarps) rope_int4_store_kernel(const RopeFormArgs a) {
  __shared__ uint4 s_extremes[kStoreWarps][4][4];   // of a pass's vectors, a word for each 8 dims
  __shared__ uint4 s_rows[kStoreWarps][kStoreAhead][2][32];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kStoreWarps + warp;
  if (t >= a.num_tokens) return;
  const int j = lane & 7, sub = lane >> 3;
  const int R = a.rotary_dim;
  const int Hq = a.num_q_heads, Hkv = a.num_kv_heads;
  const int all = Hq + 2 * Hkv;
  int ca, cb;
  lane_chunks<kInterleaved>(j, R, ca, cb);
  const int part = static_cast<int>(blockIdx.y), parts = static_cast<int>(gridDim.y);
  auto first_of = [&](int n) { return 8 * (part + (n >> 1) * parts) + 4 * (n & 1); };   // vector of the n-th pass
  const uint32_t rows = smem_addr(s_rows[warp]) + 16 * lane;
  auto ask = [&](int n, int slot) {
    const int i = first_of(n) + sub;
    if (i < all) {
      const __nv_bfloat16* src;
      if (i < Hq) src = a.q + (static_cast<size_t>(t) * Hq + i) * kHeadDim;
      else if (i < Hq + Hkv) src = a.k + (static_cast<size_t>(t) * Hkv + (i - Hq)) * kHeadDim;
      else src = a.v + (static_cast<size_t>(t) * Hkv + (i - Hq - Hkv)) * kHeadDim;
      cp_async16(rows + 1024 * slot, reinterpret_cast<const uint4*>(src) + ca);
      cp_async16(rows + 1024 * slot + 512, reinterpret_cast<const uint4*>(src) + cb);
    }
    cp_async_commit();
  };
  const int pos = a.positions[t];
  const int64_t slot = a.slot_mapping[t];
#pragma unroll
  for (int n = 0; n < kStoreAhead; ++n) ask(n, n);
  const bool has_pos = pos >= 0 && pos < a.max_pos;
  if (!has_pos && lane == 0) raise_flag(a.status, PA_FLAG_POSITION_OOB);
  bool store = has_pos && slot >= 0;
  if (store && slot >= static_cast<int64_t>(a.num_blocks) * kBlockSize) {
    if (lane == 0) raise_flag(a.status, PA_FLAG_SLOT_OOB);
    store = false;
  }
  if (!has_pos && a.q == a.q_out) {                 // left as it is
    cp_async_wait_but(0);
    return;
  }
  const int64_t blk = store ? slot / kBlockSize : 0;
  const int off = store ? static_cast<int>(slot - blk * kBlockSize) : 0;
  uint8_t* const records = static_cast<uint8_t*>(a.k_cache) + static_cast<size_t>(blk) * Hkv * kInt4Record;
  const bool turns = has_pos && j < (R >> 4);
  Angles ang = {};
  if (turns) ang = load_angles(a.cos_sin, pos, R, j);
  const int items = store ? all : Hq;
  int at = 0;
  // (a pass's place is asked for again when it is done, by the lanes that read it)
  for (int n = 0; first_of(n) < items; ask(n + kStoreAhead, at), ++n, at = at + 1 == kStoreAhead ? 0 : at + 1) {
    const int base = first_of(n), i = base + sub;
    cp_async_wait_but(kStoreAhead - 1);
    __syncwarp();
    uint4 x = s_rows[warp][at][0][lane], y = s_rows[warp][at][1][lane];
    if (i < Hq) {
      if (turns) rotate_chunks<kInterleaved>(x, y, ang);
      uint4* dst = reinterpret_cast<uint4*>(a.q_out + (static_cast<size_t>(t) * Hq + i) * kHeadDim);
      dst[ca] = x;
      dst[cb] = y;
    }
    if (base + 3 < Hq || items == Hq) continue;     // the same for the whole warp
    // keys and values (lanes of a query, or past the last vector, go along)
    const bool is_k = i < Hq + Hkv, mine = i >= Hq && i < all;
    if (turns && mine && is_k) int4_rotate_chunks<kInterleaved>(x, y, ang);
    __syncwarp();
    bool wild = false;
    uint32_t ex = int4_extremes(x, wild), ey = int4_extremes(y, wild);
    uint32_t* const words = reinterpret_cast<uint32_t*>(s_extremes[warp][sub]);
    words[ca] = ex;
    words[cb] = ey;
    __syncwarp();
    if (is_k) {
      const uint4 ga = s_extremes[warp][sub][ca >> 2], gb = s_extremes[warp][sub][cb >> 2];
      ex = __vmaxu2(__vmaxu2(ga.x, ga.y), __vmaxu2(ga.z, ga.w));
      ey = __vmaxu2(__vmaxu2(gb.x, gb.y), __vmaxu2(gb.z, gb.w));
    }
    __syncwarp();                                 // before the next pass writes the words
    ex = is_k ? ex : __vmaxu2(ex, ey);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const uint32_t other = __shfl_xor_sync(kFullMask, ex, o);
      if (!is_k) ex = __vmaxu2(ex, other);
    }
    if (!mine) continue;
    const Int4Scale qa = int4_scale(ex);
    const Int4Scale qb = is_k ? int4_scale(ey) : qa;
    uint8_t* const rec = records + static_cast<size_t>(is_k ? i - Hq : i - Hq - Hkv) * kInt4Record;
    const uint32_t wa = int4_word(x, qa, wild), wb = int4_word(y, qb, wild);
    if (is_k) {
      *reinterpret_cast<uint32_t*>(rec + int4_k_word(off, ca)) = wa;
      *reinterpret_cast<uint32_t*>(rec + int4_k_word(off, cb)) = wb;
      uint16_t* const scales = reinterpret_cast<uint16_t*>(rec + kInt4KScales + 8 * off);
      if ((ca & 3) == 0) scales[ca >> 2] = static_cast<uint16_t>(qa.word);
      if ((cb & 3) == 0) scales[cb >> 2] = static_cast<uint16_t>(qb.word);
    } else {
      *reinterpret_cast<uint32_t*>(rec + int4_v_word(off, ca)) = wa;
      *reinterpret_cast<uint32_t*>(rec + int4_v_word(off, cb)) = wb;
      if (j == 0) *reinterpret_cast<uint16_t*>(rec + kInt4VScales + 2 * off) = static_cast<uint16_t>(qa.word);
    }
  }
  cp_async_wait_but(0);
}

// ---- reading back ------------------------------------------------------------------------------
// A warp takes one record: half a warp a token, a lane the word of 8 dims, K and V of the 16 tokens with
// all loads ahead of the stores.  Each store instruction writes two rows of 256 bytes.  64 prefixes, 99,801 rows of 8 heads
// (519 MB): 80.4 us, 6.46 TB/s, 0.95 of the copy rate; one of 2,000 rows, 2 heads: 2.3 us, latency (CTAs of 8 warps: 80.6
// and 2.9).  The grid is one of num_seqs times the bound's records: CTAs past a sequence's rows load two words and leave,
// a nanosecond each, so a bound of 131,072 for those 64 costs 2.1 ms, and one of 16,384 rows among 255 of 64 1.05 ms.
__global__ void __launch_bounds__(kInt4ReadWarps * 32) read_int4_kernel(const ReadInt4Args a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads;
  const int s = blockIdx.y;
  const int r0 = a.row_start[s], n = a.row_start[s + 1] - r0;
  const int first = a.first ? a.first[s] : 0;
  if (r0 < 0 || n < 0 || n > a.max_rows || r0 > a.num_rows - n || first < 0 ||
      first > a.max_blocks * kBlockSize - n) {
    if (threadIdx.x == 0 && blockIdx.x == 0) raise_flag(a.status, PA_FLAG_CONTEXT_LEN_OOB);
    return;
  }
  if (n == 0) return;
  const int b0 = first / kBlockSize, nb = (first + n - 1) / kBlockSize - b0 + 1;
  const long long unit = static_cast<long long>(blockIdx.x) * kInt4ReadWarps + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(nb) * Hkv) return;
  const int b = static_cast<int>(unit / Hkv), g = static_cast<int>(unit - static_cast<long long>(b) * Hkv);
  const int blk = a.block_tables[static_cast<size_t>(s) * a.max_blocks + b0 + b];
  if (blk < 0 || blk >= a.num_blocks) {
    if (lane == 0) raise_flag(a.status, PA_FLAG_BLOCK_ID_OOB);
    return;
  }
  const uint8_t* const rec = a.cache + (static_cast<size_t>(blk) * Hkv + g) * kInt4Record;
  const int ch = lane & 15, odd = lane >> 4;
  uint32_t kw[8], vw[8], ks[8], vs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = 2 * i + odd;
    kw[i] = *reinterpret_cast<const uint32_t*>(rec + int4_k_word(t, ch));
    vw[i] = *reinterpret_cast<const uint32_t*>(rec + int4_v_word(t, ch));
    ks[i] = *reinterpret_cast<const uint16_t*>(rec + kInt4KScales + 8 * t + 2 * (ch >> 2));
    vs[i] = *reinterpret_cast<const uint16_t*>(rec + kInt4VScales + 2 * t);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = kBlockSize * (b0 + b) + 2 * i + odd - first;
    if (row < 0 || row >= n) continue;
    const size_t at = ((static_cast<size_t>(r0) + row) * Hkv + g) * (kHeadDim / 8) + ch;
    uint32_t s2, z2;
    int4_unpack_scale(ks[i], 0, s2, z2);
    reinterpret_cast<uint4*>(a.k_out)[at] = int4_elements(kw[i], s2, z2);
    int4_unpack_scale(vs[i], 0, s2, z2);
    reinterpret_cast<uint4*>(a.v_out)[at] = int4_elements(vw[i], s2, z2);
  }
}

cudaLaunchConfig_t chained(dim3 grid, unsigned threads, cudaLaunchAttribute* attr, cudaStream_t stream) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_rope_int4_store(const RopeFormArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const unsigned token_ctas = static_cast<unsigned>((static_cast<long long>(a.num_tokens) + kStoreWarps - 1) / kStoreWarps);
  // Where tokens are few, each group of a token's vectors has a warp of its own, up to 16 warps an SM.
  const int groups = (a.num_q_heads + 2 * a.num_kv_heads + 7) / 8;
  constexpr unsigned kRoom = 2432 / kStoreWarps;
  const int room = static_cast<int>(kRoom / (token_ctas > kRoom ? kRoom : token_ctas));
  cudaLaunchConfig_t cfg = chained(dim3(token_ctas, groups < room ? groups : room), kStoreWarps * 32, &attr, stream);
  return a.interleaved ? cudaLaunchKernelEx(&cfg, rope_int4_store_kernel<true>, a)
                       : cudaLaunchKernelEx(&cfg, rope_int4_store_kernel<false>, a);
}

cudaError_t launch_read_int4(const ReadInt4Args& a, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  // a sequence's rows may begin and end inside a block
  const long long units = ((static_cast<long long>(a.max_rows) + kBlockSize - 2) / kBlockSize + 1) * a.num_kv_heads;
  cudaLaunchConfig_t cfg = chained(dim3(static_cast<unsigned>((units + kInt4ReadWarps - 1) / kInt4ReadWarps), a.num_seqs),
                                   kInt4ReadWarps * 32, &attr, stream);
  return cudaLaunchKernelEx(&cfg, read_int4_kernel, a);
}

}  // namespace pa
