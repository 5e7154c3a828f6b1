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
//    error, exact). A border between two codes is (c + 1/2) s, 13 bits; a fused
//    multiply-add gives the sign of t - (c + 1/2) s: the rounded t and the border
//    both lie on a grid of which the error of t is at most half a step.
// Magnitudes above 2^126 are taken as 2^126 (the range then has an fp32 value).
// A row with a value that is not finite gets s = NaN: it reads back as NaN.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace mqa {

constexpr uint32_t kU4NanPair = 0x00007fc0u;  // s = NaN, m = 0

__device__ __forceinline__ float u4_clamp(float x) { return fminf(fmaxf(x, -0x1p126f), 0x1p126f); }

// The pair of a row from its (clamped) minimum and maximum, both bf16 values.
__device__ __forceinline__ uint32_t u4_pair(float lo, float hi) {
  lo = __fadd_rn(lo, 0.f);  // no -0
  const float d = __fadd_rn(__fsub_ru(hi, lo), 0.f);
  // a bf16 at most two steps below d / 15, then up to the first that reaches d
  uint32_t s = __float_as_uint(__fdiv_rd(d, 15.0f)) >> 16;
  if (__fmul_rn(__uint_as_float(s << 16), 15.0f) < d) ++s;
  return s | (__float_as_uint(lo) & 0xffff0000u);
}

__device__ __forceinline__ float u4_scale(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float u4_min(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// inv: 1 / s to a few units in the last place, or 0 for s = 0
__device__ __forceinline__ uint32_t u4_code(float x, float s, float m, float inv) {
  const float t = __fsub_rn(x, m);
  const float back = __fsub_rn(x, t);  // two-sum: t + err == x - m
  const float err = __fsub_rn(__fsub_rn(x, __fadd_rn(t, back)), __fsub_rn(m, back));
  const float c = fminf(floorf(__fmul_rn(t, inv)), 15.0f);
  float r = c;  // the border above c, then the one below
  float over = fmaf(-(c + 0.5f), s, t);
  if (over == 0.0f) over = err;
  if (over > 0.0f || (over == 0.0f && (static_cast<int>(c) & 1))) r = c + 1.0f;
  float under = fmaf(-(c - 0.5f), s, t);
  if (under == 0.0f) under = err;
  if (under < 0.0f || (under == 0.0f && (static_cast<int>(c) & 1))) r = c - 1.0f;
  return static_cast<uint32_t>(fminf(fmaxf(r, 0.0f), 15.0f));
}

}  // namespace mqa
