// The 4-bit cache's record, its quantisation and its reading, shared by the kernels that touch it.
//
// A record holds the 16 tokens of one (block, KV head), K and V, in one run of memory: the attention
// kernels bring it in whole.  element = s (c - z) with a code c and a zero point z in 0 .. 15.  The
// scale s has four significant bits, so that an element has at most eight and is exact in bf16, and a
// scale word holds both numbers: the bf16 pattern of s, whose last four bits are free for z.
//
//   0     K codes: word 4 i + g of a token's sixteen 32-bit words has dims 32 g + 8 i .. + 7, so that the
//         16 bytes i of a token are the share of one of four lanes in each of the four groups
//   1024  V codes: dims 32 u .. + 31 at 16-byte unit u ^ (token / 2 % 4), the order in which eight tokens'
//         units lie on distinct banks
//   2048  K scales: a word for each 32 dims of a token
//   2176  V scales: a word a token
//
// In a word, code pair j (bits 4j .. 4j + 3 of both halves) is dims 2j and 2j + 1 of its eight, so that one mask gives a
// pair of 16-bit integers: with 0x4300 in each half the bf16 pair 128 + c, shifted a pair of small f16 values.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kInt4Record = PA_INT4_RECORD_BYTES;
constexpr int kInt4VCodes = 1024, kInt4KScales = 2048, kInt4VScales = 2176;
static_assert(kInt4VScales + 2 * kBlockSize == kInt4Record && kInt4Record % 32 == 0, "record");

constexpr uint32_t kPairLo = 0x000f000fu;

// Byte offsets in a record: the word of dims 8 ch .. 8 ch + 7 of token t.
__device__ __forceinline__ int int4_k_word(int t, int ch) { return 64 * t + 16 * (ch & 3) + 4 * (ch >> 2); }
__device__ __forceinline__ int int4_v_word(int t, int ch) {
  return kInt4VCodes + 64 * t + 16 * ((ch >> 2) ^ ((t >> 1) & 3)) + 4 * (ch & 3);
}

// ---- quantisation --------------------------------------------------------------------------
// Of a set of values: the largest, and the largest of the negated ones, as bf16 magnitudes in the low and high
// half of a word (at least 0; infinities do not count; 0x7fc0 in both where there is a NaN).  Sets join by
// __vmaxu2.  `wild` is set where there was an infinity or a NaN.
__device__ __forceinline__ uint32_t int4_extremes(uint4 w, bool& wild) {
  // as signed 16-bit integers positive values order as they are and stand above all negative ones, which
  // order the other way round: unsigned maxima find the smallest value, if one is negative
  auto join = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t hi = __vmaxs2(__vmaxs2(a, b), __vmaxs2(c, d)), lo = __vmaxu2(__vmaxu2(a, b), __vmaxu2(c, d));
    // (largest, smallest) of the low halves and of the high ones, joined
    const uint32_t e = __vmaxs2(__byte_perm(hi, lo ^ 0x80008000u, 0x5410), __byte_perm(hi, lo ^ 0x80008000u, 0x7632));
    return __vmaxs2(e, 0u);
  };
  uint32_t e = join(w.x, w.y, w.z, w.w);
  if (__vcmpgeu2(e, 0x7f807f80u)) {                 // an infinity or a NaN
    auto finite = [](uint32_t x) { return x & __vcmpltu2(x & 0x7fff7fffu, 0x7f807f80u); };
    const bool nan = __vcmpgtu2(e, 0x7f807f80u) != 0;
    wild = true;
    e = nan ? 0x7fc07fc0u : join(finite(w.x), finite(w.y), finite(w.z), finite(w.w));
  }
  return e;
}

struct Int4Scale {
  float inv;       // 1 / s, 2^-20 of it larger
  float origin;    // 2^23 + 2^22 + z
  uint32_t word;
  bool wild;       // the range is more than 15 s
};

// The smallest s of four significant bits with 15 s >= hi - lo (rounded to fp32), in [2^-40, 2^40], and
// z = -lo / s rounded, for extremes as above.  Quotients round to the nearest integer, ties away from
// zero: a bf16 value over such an s is a tie or 2^-9 of itself away from one, so 1 / s made 2^-20 larger
// settles ties and moves nothing else.
__device__ __forceinline__ Int4Scale int4_scale(uint32_t extremes) {
  const float hi = __uint_as_float(extremes << 16), neg = __uint_as_float(extremes & 0xffff0000u);
  const float range = hi + neg;
  uint32_t s = (__float_as_uint(range * (1.f / 15.f)) + 0x000fffffu) & 0xfff00000u;
  if (15.f * __uint_as_float(s - 0x00100000u) >= range) s -= 0x00100000u;
  else if (15.f * __uint_as_float(s) < range) s += 0x00100000u;
  const float scale = fminf(fmaxf(__uint_as_float(s), 0x1p-40f), 0x1p40f);
  Int4Scale q;
  q.inv = rcp_ftz(scale) * (1.f + 0x1p-20f);
  q.origin = fmaf(fminf(neg * q.inv, 15.f), 1.f, 12582912.f);
  q.word = (__float_as_uint(scale) >> 16) | (__float_as_uint(q.origin) & 15u);
  q.wild = !(range <= 0x1p43f);
  if ((extremes & 0xffffu) == 0x7fc0u) q.word = 0x7fc0u;
  return q;
}

// The code of x (in the low four bits of the result, whose others are those of 2^23 + 2^22): the sum
// rounds the quotient to an integer.  Within a range that s covers it is at least 0, as round(lo / s) = -z, and may
// be 16 where both ends round up; `wild`: no such range.
template <bool kWild>
__device__ __forceinline__ uint32_t int4_code(float x, const Int4Scale& q) {
  float c = fmaf(x, q.inv, q.origin);
  if (kWild) c = fmaxf(c, 12582912.f);
  return __float_as_uint(fminf(c, 12582927.f));
}

// Codes of eight neighbouring dims (four bf16 pairs) as a word.
template <bool kWild>
__device__ __forceinline__ uint32_t int4_word_of(uint4 w, const Int4Scale& q) {
  // each shift by four moves the upper bits of 12582912 along; what they add up to is taken off
  constexpr uint32_t kBase = 0x4b400000u;
  constexpr uint32_t kSum = kBase * 0x11111111u;
  uint32_t r = int4_code<kWild>(bf16hi(w.w), q);
  r = r * 16 + int4_code<kWild>(bf16hi(w.z), q);
  r = r * 16 + int4_code<kWild>(bf16hi(w.y), q);
  r = r * 16 + int4_code<kWild>(bf16hi(w.x), q);
  r = r * 16 + int4_code<kWild>(bf16lo(w.w), q);
  r = r * 16 + int4_code<kWild>(bf16lo(w.z), q);
  r = r * 16 + int4_code<kWild>(bf16lo(w.y), q);
  r = r * 16 + int4_code<kWild>(bf16lo(w.x), q);
  return r - kSum;
}
__device__ __forceinline__ uint32_t int4_word(uint4 w, const Int4Scale& q, bool wild) {
  return wild || q.wild ? int4_word_of<true>(w, q) : int4_word_of<false>(w, q);
}

// ---- reading -------------------------------------------------------------------------------
__device__ __forceinline__ float int4_scale_of(uint32_t word) { return __uint_as_float((word & 0xfff0u) << 16); }

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A scale word (the low or the high half of `words`) as the bf16 pairs (s, s) and (128 + z, 128 + z).
__device__ __forceinline__ void int4_unpack_scale(uint32_t words, int high, uint32_t& s2, uint32_t& z2) {
  const uint32_t w = __byte_perm(words, words, high ? 0x3232 : 0x1010);
  s2 = w & 0xfff0fff0u;
  z2 = (w & kPairLo) | 0x43004300u;
}
// The eight elements of a word as bf16, exact: (128 + c) - (128 + z) is an integer of at most 15, its product with s
// has eight significant bits.
__device__ __forceinline__ uint4 int4_elements(uint32_t w, uint32_t s2, uint32_t z2) {
  uint4 r;
  r.x = mul_bf16x2(sub_bf16x2((w & kPairLo) | 0x43004300u, z2), s2);
  r.y = mul_bf16x2(sub_bf16x2(((w >> 4) & kPairLo) | 0x43004300u, z2), s2);
  r.z = mul_bf16x2(sub_bf16x2(((w >> 8) & kPairLo) | 0x43004300u, z2), s2);
  r.w = mul_bf16x2(sub_bf16x2(((w >> 12) & kPairLo) | 0x43004300u, z2), s2);
  return r;
}

// ---- rotation ------------------------------------------------------------------------------
// a b - c d rounded to fp32, as if from its exact value: the products and their difference, each with what its
// rounding left (Knuth's sum: s + t is p - q).
__device__ __forceinline__ float exact_difference(float a, float b, float c, float d) {
  const float p = __fmul_rn(a, b), q = __fmul_rn(c, d);
  const float rest = __fsub_rn(__fmaf_rn(a, b, -p), __fmaf_rn(c, d, -q));
  const float s = __fsub_rn(p, q), back = __fsub_rn(s, p);
  const float t = __fsub_rn(__fsub_rn(p, __fsub_rn(s, back)), __fadd_rn(q, back));
  return __fadd_rn(s, __fadd_rn(t, rest));
}

// A row that is quantised is rotated as if exactly, rounded to fp32 and then to bf16: a code never depends on how the
// products were formed.  rope_rotate_pairs is within two ulps of fp32, so it does wherever no value lies within four
// of a border of the bf16 rounding; `border` collects how near the values came (the halves of a word, at most 8 where
// one did), and where it says so the values are formed again by int4_rotate_exactly.
// (Again in 64 bits, value by value: 320 us for a 16,384-row store; value by value in fp32: 100 us.)
__device__ __forceinline__ uint32_t round_pair(float a, float b, uint32_t& border) {
  border = __viaddmin_u16x2(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410), 0x80048004u, border);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ bool at_border(uint32_t border) { return min(border & 0xffffu, border >> 16) <= 8u; }

__device__ __forceinline__ void int4_rotate_pairs(uint32_t& lo, uint32_t& hi, float2 c, float2 s, uint32_t& border) {
  const float x0 = bf16lo(lo), x1 = bf16hi(lo), y0 = bf16lo(hi), y1 = bf16hi(hi);
  lo = round_pair(diff_of_products(x0, c.x, y0, s.x), diff_of_products(x1, c.y, y1, s.y), border);
  hi = round_pair(diff_of_products(y0, c.x, -x0, s.x), diff_of_products(y1, c.y, -x1, s.y), border);
}
// x and y rotated again, to lo and hi, which hold the first form's values: those stay where a number is infinite
// or a product passes fp32, and this form would say NaN.
__device__ __forceinline__ void int4_rotate_exactly(uint32_t x, uint32_t y, float2 c, float2 s, uint32_t& lo, uint32_t& hi) {
  auto take = [](uint32_t exact, uint32_t& at) {
    const uint32_t finite = __vcmpltu2(exact & 0x7fff7fffu, 0x7f807f80u);
    at = (exact & finite) | (at & ~finite);
  };
  const float x0 = bf16lo(x), x1 = bf16hi(x), y0 = bf16lo(y), y1 = bf16hi(y);
  take(pack_bf16x2(exact_difference(x0, c.x, y0, s.x), exact_difference(x1, c.y, y1, s.y)), lo);
  take(pack_bf16x2(exact_difference(y0, c.x, -x0, s.x), exact_difference(y1, c.y, -x1, s.y)), hi);
}

// Two adjacent pairs, halves apart (kInterleaved: (x0, y0), (x1, y1)), by the first form and where it asks for it by
// the second.
template <bool kInterleaved>
__device__ __forceinline__ void int4_rotate(uint32_t& w0, uint32_t& w1, float2 c, float2 s) {
  uint32_t lo = kInterleaved ? __byte_perm(w0, w1, 0x5410) : w0, hi = kInterleaved ? __byte_perm(w0, w1, 0x7632) : w1;
  uint32_t border = 0xffffffffu, a = lo, b = hi;
  int4_rotate_pairs(a, b, c, s, border);
  if (at_border(border)) int4_rotate_exactly(lo, hi, c, s, a, b);
  w0 = kInterleaved ? __byte_perm(a, b, 0x5410) : a;
  w1 = kInterleaved ? __byte_perm(a, b, 0x7632) : b;
}

}  // namespace pa
