// How the lanes of a warp hold and turn head vectors of a RoPE form; shared by the fused RoPE stores.
//
// A form rotates the first R of a head's 128 dims (R a multiple of 16), pairing dims (i, i +
// R/2) or (2i, 2i + 1).  Eight lanes hold a head, two 16-byte chunks (8 dims) each, chosen so
// that every pair lies within one lane: lanes j < R/16 hold the dims of pairs 8j .. 8j + 7 --
// chunks j and j + R/16 for the half layout, 2j and 2j + 1 for the interleaved one -- and lanes
// j >= R/16 two chunks of the dims that pass through, 2j and 2j + 1 for both.  So one lane reads
// cos and sin of 8 angles, as two 16-byte words each, whatever the form.
#pragma once

#include "pa_device.cuh"

namespace pa {

struct Angles {
  float4 c0, c1, s0, s1;  // cos and sin of pairs 8j .. 8j + 7
};

__device__ __forceinline__ Angles load_angles(const float* cos_sin, int pos, int R, int j) {
  const float4* row = reinterpret_cast<const float4*>(cos_sin + static_cast<size_t>(pos) * R);
  Angles a;
  a.c0 = row[2 * j];
  a.c1 = row[2 * j + 1];
  a.s0 = row[R / 8 + 2 * j];
  a.s1 = row[R / 8 + 2 * j + 1];
  return a;
}

// Chunks of lane j (of 8).
template <bool kInterleaved>
__device__ __forceinline__ void lane_chunks(int j, int R, int& ca, int& cb) {
  const int n = R >> 4;
  if (!kInterleaved && j < n) {
    ca = j;
    cb = j + n;
  } else {
    ca = 2 * j;
    cb = 2 * j + 1;
  }
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate_chunks(uint4& x, uint4& y, const Angles& a) {
  const float2 c0 = make_float2(a.c0.x, a.c0.y), c1 = make_float2(a.c0.z, a.c0.w);
  const float2 c2 = make_float2(a.c1.x, a.c1.y), c3 = make_float2(a.c1.z, a.c1.w);
  const float2 s0 = make_float2(a.s0.x, a.s0.y), s1 = make_float2(a.s0.z, a.s0.w);
  const float2 s2 = make_float2(a.s1.x, a.s1.y), s3 = make_float2(a.s1.z, a.s1.w);
  if constexpr (kInterleaved) {
    rope_rotate_interleaved(x.x, x.y, c0, s0);
    rope_rotate_interleaved(x.z, x.w, c1, s1);
    rope_rotate_interleaved(y.x, y.y, c2, s2);
    rope_rotate_interleaved(y.z, y.w, c3, s3);
  } else {
    rope_rotate_pairs(x.x, y.x, c0, s0);
    rope_rotate_pairs(x.y, y.y, c1, s1);
    rope_rotate_pairs(x.z, y.z, c2, s2);
    rope_rotate_pairs(x.w, y.w, c3, s3);
  }
}

}  // namespace pa
