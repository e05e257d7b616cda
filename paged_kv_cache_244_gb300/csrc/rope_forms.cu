// RoPE tables, and the fused RoPE + KV-cache store with a RoPE form, for sm_103a.
//
// "Pico-vLLM：从零手写的工业级LLM推理引擎实现", §1 模型实现层 (RoPE) and §2 Kernel层 (RoPE fused with
// the KV cache store); "从零实现 LLM 推理引擎：深挖 vLLM 的六大核心优化", §3.1 (16-token blocks);
// "nano-vllm：vLLM 极简实现与大模型推理流程解析", §学习要点 (8-bit quantisation of the cache).

#include "pa_device.cuh"
#include "pa_launch.h"
#include "rope_form.cuh"

namespace pa {
namespace {

// Bytes bound the large calls: 17,363 rows of 32 + 8 + 8 heads with 96 dims rotated (434 MB) take 65 us,
// 6.7 TB/s, the copy rate.  The loads' latency bounds the small ones: 64 rows take 2.6 us.
constexpr int kFormWarps = 8;

// One warp, one token: the Hq query heads into q_out (rotated), and unless kQOnly the Hkv keys
// (rotated) and values into their cache slot, four vectors a pass, kGroup passes loaded before
// any is stored (the shape of the whole-head half-layout store, and its two group sizes).  With
// parts > 1 the warp takes the groups part, part + parts, .. only: where tokens are few, each group
// of a token has a warp of its own and all loads are in flight at once.
template <bool kInterleaved, int kGroup, bool kQOnly>
__device__ __forceinline__ void form_token(const RopeFormArgs& a, int t, int part = 0, int parts = 1) {
  const int lane = threadIdx.x & 31;
  const int j = lane & 7, sub = lane >> 3;
  const int R = a.rotary_dim;
  const int Hq = a.num_q_heads, Hkv = a.num_kv_heads;
  const int all = kQOnly ? Hq : Hq + 2 * Hkv;
  int ca, cb;
  lane_chunks<kInterleaved>(j, R, ca, cb);
  uint4 x[kGroup], y[kGroup];
  auto load_group = [&](int base) {
#pragma unroll
    for (int p = 0; p < kGroup; ++p) {
      const int i = base + 4 * p + sub;
      x[p] = y[p] = make_uint4(0u, 0u, 0u, 0u);
      if (i >= all) continue;
      const __nv_bfloat16* src;
      if (i < Hq) src = a.q + (static_cast<size_t>(t) * Hq + i) * kHeadDim;
      else if (i < Hq + Hkv) src = a.k + (static_cast<size_t>(t) * Hkv + (i - Hq)) * kHeadDim;
      else src = a.v + (static_cast<size_t>(t) * Hkv + (i - Hq - Hkv)) * kHeadDim;
      x[p] = reinterpret_cast<const uint4*>(src)[ca];
      y[p] = reinterpret_cast<const uint4*>(src)[cb];
    }
  };
  const int pos = a.positions[t];
  const int64_t slot = kQOnly ? -1 : a.slot_mapping[t];
  const int first = 4 * kGroup * part, step = 4 * kGroup * parts;
  load_group(first);
  const bool has_pos = pos >= 0 && pos < a.max_pos;
  if (!has_pos && lane == 0) raise_flag(a.status, PA_FLAG_POSITION_OOB);
  bool store = !kQOnly && has_pos && slot >= 0;
  if (store && slot >= static_cast<int64_t>(a.num_blocks) * kBlockSize) {
    if (lane == 0) raise_flag(a.status, PA_FLAG_SLOT_OOB);
    store = false;
  }
  if (!has_pos && a.q == a.q_out) return;  // left as it is
  const int64_t blk = store ? slot / kBlockSize : 0;
  const int off = store ? static_cast<int>(slot - blk * kBlockSize) : 0;
  const bool turns = has_pos && j < (R >> 4);
  Angles ang = {};
  if (turns) ang = load_angles(a.cos_sin, pos, R, j);
  const int items = store ? all : Hq;
  for (int base = first; base < items; base += step) {
    if (base != first) load_group(base);
#pragma unroll
    for (int p = 0; p < kGroup; ++p) {
      const int i = base + 4 * p + sub;
      if (i >= items) continue;
      if (turns && i < Hq + Hkv) rotate_chunks<kInterleaved>(x[p], y[p], ang);
      uint4* dst;
      if (i < Hq) {
        dst = reinterpret_cast<uint4*>(a.q_out + (static_cast<size_t>(t) * Hq + i) * kHeadDim);
      } else {
        const bool is_k = i < Hq + Hkv;
        const int g = is_k ? i - Hq : i - Hq - Hkv;
        const size_t row = (static_cast<size_t>(blk) * Hkv + g) * kBlockSize + off;
        dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_k ? a.k_cache : a.v_cache) + row * kHeadDim);
      }
      dst[ca] = x[p];
      dst[cb] = y[p];
    }
  }
}

template <bool kInterleaved, int kGroup>
__global__ void __launch_bounds__(kFormWarps * 32, kGroup == 2 ? 4 : 1) rope_form_store_kernel(const RopeFormArgs a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int t = blockIdx.x * kFormWarps + static_cast<int>(threadIdx.x >> 5);
  if (t >= a.num_tokens) return;
  form_token<kInterleaved, kGroup, false>(a, t, blockIdx.y, gridDim.y);
}

// ---- the store into block-scaled E4M3 caches -----------------------------------------------
// A block's scale depends on all the rows the call puts into it, so the unit of work is a run:
// the rows of one block, which follow one another with at most kGap - 1 padding rows between
// two.  A CTA takes a window of rows, lists the runs that begin in it, and its warps take (run,
// KV head, K or V) units: the run's up to 16 rows are loaded at once (4 KiB a warp), K rotated,
// the magnitudes reduced over the warp, and the codes written.  CTAs behind them rotate q.
// Bytes bound it.  8,270 rows of 16 ragged prompts, 32 / 8 heads (191 MB): 33.4 us, 5.7 TB/s, with four CTAs of
// 64 registers (24 to 32 bytes spilled) an SM and q two passes at a time (three CTAs of 80 registers, four passes:
// 34.5 us; q's CTAs first: 39.5; loads marked as streaming: 35.0).
constexpr int kGap = 16;                       // a row that follows one of its block within kGap rows is in its run
constexpr int kRunWindow = 64;                 // most rows of a window
constexpr int kRunTail = kGap * kBlockSize;    // rows past the window that its last run may take

template <bool kInterleaved>
__global__ void __launch_bounds__(kFormWarps * 32, 4) rope_block_store_kernel(const RopeFormArgs a, const int window,
                                                                             const int kv_ctas, const int q_parts) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= kv_ctas) {
    const int unit = static_cast<int>(blockIdx.x) - kv_ctas;
    const int t = unit / q_parts * kFormWarps + warp;
    if (t < a.num_tokens) form_token<kInterleaved, 2, true>(a, t, unit % q_parts, q_parts);
    return;
  }
  __shared__ int blocks[kGap + kRunWindow + kRunTail];       // block of a row, -1: not stored
  __shared__ unsigned char offs[kGap + kRunWindow + kRunTail];
  __shared__ int run_block[kRunWindow];
  __shared__ short run_rows[kRunWindow][kBlockSize];         // row (from the window's first) of each slot, -1: none
  __shared__ int num_runs;
  const int T = a.num_tokens, R = a.rotary_dim, Hkv = a.num_kv_heads;
  const int w0 = static_cast<int>(blockIdx.x) * window;
  if (threadIdx.x == 0) num_runs = 0;
  for (int i = threadIdx.x; i < kGap + window + kRunTail; i += kFormWarps * 32) {
    const long long t = static_cast<long long>(w0) - kGap + i;
    int b = -1, o = 0;
    if (t >= 0 && t < T) {
      const int64_t slot = a.slot_mapping[t];
      const int pos = a.positions[t];
      if (slot >= 0 && pos >= 0 && pos < a.max_pos) {
        if (slot < static_cast<int64_t>(a.num_blocks) * kBlockSize) {
          b = static_cast<int>(slot / kBlockSize);
          o = static_cast<int>(slot % kBlockSize);
        } else if (i >= kGap && i < kGap + window) {
          raise_flag(a.status, PA_FLAG_SLOT_OOB);
        }
      }
    }
    blocks[i] = b;
    offs[i] = static_cast<unsigned char>(o);
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < window) {
    const int i = kGap + threadIdx.x;
    const int b = blocks[i];
    bool head = b >= 0;
    for (int d = 1; head && d <= kGap; ++d) {
      if (blocks[i - d] < 0) continue;
      head = blocks[i - d] != b;
      break;
    }
    if (head) {
      const int n = atomicAdd(&num_runs, 1);   // the order of the list changes nothing: runs are apart
      run_block[n] = b;
#pragma unroll
      for (int o = 0; o < kBlockSize; ++o) run_rows[n][o] = -1;
      for (int k = i, last = i; k < kGap + window + kRunTail && k - last <= kGap; ++k) {
        if (blocks[k] < 0) continue;
        if (blocks[k] != b) break;
        run_rows[n][offs[k]] = static_cast<short>(k - kGap);
        last = k;
      }
    }
  }
  __syncthreads();

  const int j = lane & 7, sub = lane >> 3;
  int ca, cb;
  lane_chunks<kInterleaved>(j, R, ca, cb);
  const int units = num_runs * 2 * Hkv;
  for (int u = warp; u < units; u += kFormWarps) {
    const int n = u / (2 * Hkv), item = u - n * 2 * Hkv;
    const bool is_k = item < Hkv;
    const int g = is_k ? item : item - Hkv;
    const int blk = run_block[n];
    const size_t tile = static_cast<size_t>(blk) * Hkv + g;
    float* scale = reinterpret_cast<float*>(a.kv_scale + tile) + (is_k ? 0 : 1);
    const float old = *scale;
    const __nv_bfloat16* src = is_k ? a.k : a.v;
    uint4 x[4], y[4];
    int rows[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {             // slot 4p + sub of the block
      rows[p] = run_rows[n][4 * p + sub];
      x[p] = y[p] = make_uint4(0u, 0u, 0u, 0u);
      if (rows[p] < 0) continue;
      const uint4* v = reinterpret_cast<const uint4*>(src + (static_cast<size_t>(w0 + rows[p]) * Hkv + g) * kHeadDim);
      x[p] = v[ca];
      y[p] = v[cb];
    }
    if (is_k && j < (R >> 4)) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (rows[p] >= 0)
          rotate_chunks<kInterleaved>(x[p], y[p], load_angles(a.cos_sin, a.positions[w0 + rows[p]], R, j));
    }
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(finite_magnitudes(x[p].x), finite_magnitudes(x[p].y)),
                                   __vmaxu2(finite_magnitudes(x[p].z), finite_magnitudes(x[p].w))));
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(finite_magnitudes(y[p].x), finite_magnitudes(y[p].y)),
                                   __vmaxu2(finite_magnitudes(y[p].z), finite_magnitudes(y[p].w))));
    }
    const uint32_t amax = __reduce_max_sync(kFullMask, max(top & 0xffffu, top >> 16));
    const bool fresh = run_rows[n][0] >= 0;
    const float now = e4m3_grow_scale(old, e4m3_scale_for(amax), fresh);
    const float inv = __frcp_rn(now);
    uint8_t* codes = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) + tile * kBlockSize * kHeadDim;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (rows[p] < 0) continue;
      uint8_t* row = codes + (4 * p + sub) * kHeadDim;
      *reinterpret_cast<uint2*>(row + 8 * ca) =
          make_uint2(e4m3x2_of(x[p].x, inv) | (static_cast<uint32_t>(e4m3x2_of(x[p].y, inv)) << 16),
                     e4m3x2_of(x[p].z, inv) | (static_cast<uint32_t>(e4m3x2_of(x[p].w, inv)) << 16));
      *reinterpret_cast<uint2*>(row + 8 * cb) =
          make_uint2(e4m3x2_of(y[p].x, inv) | (static_cast<uint32_t>(e4m3x2_of(y[p].y, inv)) << 16),
                     e4m3x2_of(y[p].z, inv) | (static_cast<uint32_t>(e4m3x2_of(y[p].w, inv)) << 16));
    }
    if (!fresh && now != old) {               // the scale grew: the other slots' codes anew
      const float f = __fdiv_rn(old, now);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (rows[p] >= 0) continue;
        uint4* w = reinterpret_cast<uint4*>(codes + (4 * p + sub) * kHeadDim) + j;
        *w = e4m3x16_rescale(*w, f);
      }
    }
    if (lane == 0) *scale = now;
  }
}

// ---- the table -------------------------------------------------------------------------------
// Pair i at position p turns by p * turns[i] / 2^64 of a whole turn, modulo 1: the low 64 bits of
// the product are exact but for the error of turns[i], which the host forms as a double: within 2^-55
// of a turn (the fastest pair's; over the five scalings, against 200-bit arithmetic), so 2^-38 of a turn at
// position 131,072 and 2^-24 at 2^31.  The nearest quarter turn is taken off in the product's high word, so that what
// is rounded to fp32 is an angle of at most pi/4, relative to its own size (the low word joins in
// one FMA), and sin and cos keep their relative accuracy next to their zeros.  On that interval
// the Taylor sums of sin to x^9 and of cos to x^10 are within 2^-29; both are formed for two pairs
// at a time in packed fp32.  A thread keeps four neighbouring pairs and goes down the rows: one
// 16-byte word of cos, one of sin a row.
//
// Bound by the 8 bytes a pair it writes, with about 30 instructions a pair beside them.  131,072 x 128:
// 10.7 us, 6.3 TB/s (a first form with a 64-bit division per word and sign handling in 64 bits
// took 17.1 us).
constexpr int kTableThreads = 256;

__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const RopeTableArgs a) {
  __shared__ unsigned long long all_turns[64];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  if (threadIdx.x < 64) all_turns[threadIdx.x] = a.turns[threadIdx.x];
  __syncthreads();
  const int R = a.rotary_dim, words = R >> 3;       // 16-byte words of cos in a row, 2 .. 16
  const int rows = kTableThreads / words;           // rows of a pass of the CTA
  const int r = threadIdx.x / words, c = threadIdx.x - r * words;
  if (r >= rows) return;
  unsigned t_lo[4], t_hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t_lo[i] = static_cast<unsigned>(all_turns[4 * c + i]);
    t_hi[i] = static_cast<unsigned>(all_turns[4 * c + i] >> 32);
  }
  auto both = [](float x) { return pack_f32x2(x, x); };
  const long long step = static_cast<long long>(gridDim.x) * rows;
  for (long long p = static_cast<long long>(blockIdx.x) * rows + r; p < a.max_pos; p += step) {
    const unsigned pos = static_cast<unsigned>(p);
    float x[4];
    unsigned quarter[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned long long f = static_cast<unsigned long long>(t_lo[i]) * pos +
                                   (static_cast<unsigned long long>(t_hi[i] * pos) << 32);
      const unsigned hi = static_cast<unsigned>(f >> 32);
      quarter[i] = (hi + (1u << 29)) >> 30;          // 0 .. 3 (wraps past 7/8)
      const int rest = static_cast<int>(hi - (quarter[i] << 30));
      x[i] = fmaf(static_cast<float>(static_cast<unsigned>(f)), 0x1p-32f, static_cast<float>(rest)) *
             (6.28318530717958647692f * 0x1p-32f);
    }
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t v = pack_f32x2(x[i], x[i + 1]);
      const uint64_t y = fma_f32x2(v, v, 0ull);
      uint64_t s = fma_f32x2(y, both(1.f / 362880.f), both(-1.f / 5040.f));
      s = fma_f32x2(s, y, both(1.f / 120.f));
      s = fma_f32x2(s, y, both(-1.f / 6.f));
      s = fma_f32x2(fma_f32x2(v, y, 0ull), s, v);
      uint64_t q = fma_f32x2(y, both(-1.f / 3628800.f), both(1.f / 40320.f));
      q = fma_f32x2(q, y, both(-1.f / 720.f));
      q = fma_f32x2(q, y, both(1.f / 24.f));
      q = fma_f32x2(q, y, both(-0.5f));
      q = fma_f32x2(q, y, both(1.f));
      float s0[2], c0[2];
      unpack_f32x2(s, s0[0], s0[1]);
      unpack_f32x2(q, c0[0], c0[1]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const unsigned k = quarter[i + u];
        const float c1 = (k & 1) ? s0[u] : c0[u], s1 = (k & 1) ? c0[u] : s0[u];
        cs[i + u] = __uint_as_float(__float_as_uint(c1 * a.magnitude) ^ (((k + 1) & 2u) << 30));
        sn[i + u] = __uint_as_float(__float_as_uint(s1 * a.magnitude) ^ ((k & 2u) << 30));
      }
    }
    float* row = a.cos_sin + p * R;
    *reinterpret_cast<float4*>(row + 4 * c) = make_float4(cs[0], cs[1], cs[2], cs[3]);
    *reinterpret_cast<float4*>(row + R / 2 + 4 * c) = make_float4(sn[0], sn[1], sn[2], sn[3]);
  }
}

cudaLaunchConfig_t chained(unsigned ctas, unsigned threads, cudaLaunchAttribute* attr, cudaStream_t stream) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Warps of a token that has `vectors` head vectors, one for each group of `group`, as long as the grid
// stays within 304 CTAs (one wave): a lone wave's time is its longest chain of loads.
int warps_per_token(int vectors, int group, unsigned token_ctas) {
  const int groups = (vectors + group - 1) / group;
  const int room = 304 / static_cast<int>(token_ctas > 304 ? 304 : token_ctas);
  return groups < room ? groups : room;
}

}  // namespace

cudaError_t launch_rope_form_store(const RopeFormArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const unsigned token_ctas = static_cast<unsigned>((static_cast<long long>(a.num_tokens) + kFormWarps - 1) / kFormWarps);
  if (a.kv_scale) {
    // Rows of a window: the most that leave 304 windows (two for each SM), up to 64; a decode batch's rows
    // are runs of their own and want many windows, a prompt's windows of 16 rows and more hold whole
    // blocks.  8 K prefill rows: 33.1 us with 304, 34.0 with 608, 34.9 with 152; 2048 rows in runs of 1 to 8:
    // 5.7, 7.0, 6.6 us.
    int window = 1;
    while (window < kRunWindow && static_cast<long long>(window) * 2 * 304 <= a.num_tokens) window *= 2;
    const unsigned kv_ctas = static_cast<unsigned>((static_cast<long long>(a.num_tokens) + window - 1) / window);
    const int q_parts = warps_per_token(a.num_q_heads, 8, token_ctas);
    cudaLaunchConfig_t cfg = chained(kv_ctas + token_ctas * q_parts, kFormWarps * 32, &attr, stream);
    auto kernel = a.interleaved ? rope_block_store_kernel<true> : rope_block_store_kernel<false>;
    return cudaLaunchKernelEx(&cfg, kernel, a, window, static_cast<int>(kv_ctas), q_parts);
  }
  cudaLaunchConfig_t cfg = chained(token_ctas, kFormWarps * 32, &attr, stream);
  const bool many = a.num_tokens > 2048;
  if (!many) cfg.gridDim.y = warps_per_token(a.num_q_heads + 2 * a.num_kv_heads, 16, token_ctas);
  if (a.interleaved)
    return many ? cudaLaunchKernelEx(&cfg, rope_form_store_kernel<true, 2>, a)
                : cudaLaunchKernelEx(&cfg, rope_form_store_kernel<true, 4>, a);
  return many ? cudaLaunchKernelEx(&cfg, rope_form_store_kernel<false, 2>, a)
              : cudaLaunchKernelEx(&cfg, rope_form_store_kernel<false, 4>, a);
}

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t stream) {
  const int rows = kTableThreads / (a.rotary_dim / 8);
  long long ctas = (static_cast<long long>(a.max_pos) + rows - 1) / rows;
  if (ctas > 152 * 8) ctas = 152 * 8;   // 8 CTAs of 256 threads fit an SM
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = chained(static_cast<unsigned>(ctas), kTableThreads, &attr, stream);
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, a);
}

}  // namespace pa
