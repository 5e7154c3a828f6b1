// Rows of a 4-bit cache: head_dim codes of 0..15, two to a byte (the even
// dimension in the low half), and one bf16 pair (scale s, minimum m) in a
// 32-bit word, s in the low half. The value is m + s * code.
//
// Encoding of a row x of bf16 values: m = min x, s the smallest bf16 with
// 15 s >= max x - m (so that no code is clamped), code = (x - m) / s rounded to
// nearest, ties to even. Every decision is the exact one, in 32-bit arithmetic:
//  - max x - m is rounded up to fp32. 15 s has at most 12 significant bits, so
//    it is an fp32 value, and 15 s >= max x - m holds exactly when 15 s reaches
//    the rounded difference.
//  - t = x - m is held as a pair of floats (the rounded difference and its
//    error, exact). A border between two codes is (c + 1/2) s, 13 bits: it and
//    the rounded t lie on a grid of which the error of t is at most half a step,
//    so the rounded t decides unless it is the border.
// Magnitudes above 2^126 are taken as 2^126 (the range then has an fp32 value).
// A row with a value that is not finite gets s = NaN: it reads back as NaN.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace mqa {

constexpr uint32_t kU4NanPair = 0x00007fc0u;  // s = NaN, m = 0

__device__ __forceinline__ float u4_clamp(float x) { return fminf(fmaxf(x, -0x1p126f), 0x1p126f); }

__device__ __forceinline__ float u4_scale(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float u4_min(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// The pair of a row from its minimum and maximum, both bf16 values.
__device__ __forceinline__ uint32_t u4_pair(float lo, float hi) {
  lo = __fadd_rn(lo, 0.f);  // no -0
  const float d = __fadd_rn(__fsub_ru(hi, lo), 0.f);
  // a bf16 at most two steps below the first that reaches d, then up to that
  uint32_t s = __float_as_uint(__fmul_rd(d, 0x1.11110ep-4f)) >> 16;  // (a little less than 1 / 15)
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (__fmul_rn(__uint_as_float(s << 16), 15.0f) < d) ++s;
  return s | (__float_as_uint(lo) & 0xffff0000u);
}

// Whether a row's values and scale are of sizes that u4_codes takes as they are:
// else they are clamped, and a small scale and its values brought up by 2^64.
__device__ __forceinline__ bool u4_plain(float lo, float hi, float s) {
  return lo >= -0x1p126f && hi <= 0x1p126f && s >= 0x1p-100f;
}

// Code c of x, t = x - m rounded, where over = t - c s reaches half = s / 2: a
// border, which what rounding left of t decides, or a wrong c.
static __device__ __noinline__ float u4_border(float x, float m, float t, float over, float half, float c) {
  const float back = __fsub_rn(x, t);  // two-sum: t + err == x - m
  const float err = __fsub_rn(__fsub_rn(x, __fadd_rn(t, back)), __fsub_rn(m, back));
  const bool odd = static_cast<int>(c) & 1;
  if (over >= half && (over > half || err > 0.f || (err == 0.f && odd))) return c + 1.f;
  if (over <= -half && (over < -half || err < 0.f || (err == 0.f && odd))) return c - 1.f;
  return c;
}

// The codes of 8 values, packed: s > 0 and m the row's scale and minimum, inv
// 1 / s to a few units in the last place. The whole number c nearest to t inv is
// the code unless t - c s reaches s / 2. (That difference is exact: t is within
// a factor of two of c s, or c = 0.)
__device__ __forceinline__ uint32_t u4_codes(const float (&x)[8], float s, float m, float inv) {
  const float half = 0.5f * s;
  float packed[2] = {0x1p23f, 0x1p23f};  // whole numbers below 2^16 in its low bits
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fsub_rn(x[i], m);
    float c = __fsub_rn(fmaf(t, inv, 0x1.8p23f), 0x1.8p23f);
    const float over = fmaf(-c, s, t);
    if (fabsf(over) >= half) c = u4_border(x[i], m, t, over, half, c);
    packed[i / 4] = fmaf(c, static_cast<float>(1 << (4 * (i % 4))), packed[i / 4]);
  }
  return __byte_perm(__float_as_uint(packed[0]), __float_as_uint(packed[1]), 0x5410);
}

}  // namespace mqa
