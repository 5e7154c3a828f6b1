// kv_append_norm_rope kernel, and kv_append_rope over a 4-bit cache: each
// query and key head is normalised (y = x / sqrt(mean x^2 + eps) * w, when
// weights are given), its adjacent pairs are turned by their position -- one
// position, or one of up to four axes for each section of the pairs -- and the
// rows go where they belong: q as fp32 to q_rot, k and v into the cache in its
// type.
//
// A stored key is the 64-bit result rounded once to the type of k_new; a
// one-byte or 4-bit cache holds that bf16 row encoded. A rounding that falls the
// other way changes a whole code there. So the key is formed in fp32 first, with
// a bound on its error; where a value lies so near a rounding border that this
// does not settle it (a normal row of 128: 4 in 100 with a norm, 1 without) the
// row is formed again in pairs of floats (a value and what its rounding left, 2^-37 of the
// pair's length and better), not in fp64, whose rate on this part is 1/64 of
// fp32's. The sines and cosines are such pairs, from their Taylor series about
// the nearest multiple of pi / 2; only the reduction of the angle is fp64. A
// query, which fp32 holds, takes the fp32 part alone.
//
// A lane holds 8 neighbouring values of a row, so a warp two rows (d = 128) or
// four (d = 64) at a time: what a row costs once -- its scale, its addresses,
// the steps of its sums -- is paid by half or a quarter of a warp. Of the query
// several such groups are requested together. A block serves one token, or four
// (eight) of a long prompt: their d / 2 sines and cosines are formed once, by
// all threads, then its warps take the heads, the keys and values first.
//
// What bounds it: a prompt (8 x 4096 tokens, 32 query and 8 kv heads of 128, into
// a 4-bit cache) 215 us, 975 MB at 4.5 TB/s, two thirds of the copy rate: memory
// busy 60%, the issue of instructions 65%, half of them the forming and encoding
// of keys and values. A warp a row with all keys as pairs took 530 us, four
// query rows a warp with keys in fp32 300, 8 values a lane 270, and 215 with the
// rare paths out of line, for the warps had waited for their code. Two groups
// of query rows at a time, or one, 286 and 305 us (with the rows read back, 267
// so), three or five blocks on an SM 301 and 284. One token of each of 32
// sequences 4.1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "rope.cuh"
#include "u4.cuh"

namespace mqa {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;

// ------------------------------------------------ pairs of floats: hi + lo
struct Dd {
  float h, l;
};

// |a| >= |b| or a = 0
__device__ __forceinline__ Dd fast_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Dd two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Dd two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, fmaf(a, b, -p)};
}
// (not renormalised: |l| is a few units of h's last place)
__device__ __forceinline__ Dd mul(Dd a, Dd b) {
  Dd p = two_prod(a.h, b.h);
  p.l = fmaf(a.h, b.l, fmaf(a.l, b.h, p.l));
  return p;
}
__device__ __forceinline__ Dd add(Dd a, Dd b) {
  const Dd s = two_sum(a.h, b.h);
  return fast_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}

// c + z v for a constant c with |c| >= |z v|, given as hi + lo
__device__ __forceinline__ Dd horner(double c, Dd z, Dd v) {
  const float ch = static_cast<float>(c), cl = static_cast<float>(c - static_cast<double>(ch));
  const Dd p = mul(z, v), s = fast_sum(ch, p.h);
  return {s.h, __fadd_rn(s.l, __fadd_rn(p.l, cl))};
}

// cos and sin of pos * theta. The angle is formed and reduced by the nearest
// multiple k of pi / 2 in fp64 (pi / 2 in two parts, 106 bits), then
// both series in z = r^2, |r| <= pi / 4: the terms that are below 2^-14 of the
// result are summed in fp32, the others as pairs (error 2^-37).
__device__ __forceinline__ void cos_sin(int pos, double theta, Dd* c, Dd* s) {
  const double x = static_cast<double>(pos) * theta;
  // k = the nearest whole number to 2 x / pi: by adding 1.5 2^52, whose low bits then hold it
  const double big = fma(x, 4.0 * kInvTwoPi, 0x1.8p52), k = big - 0x1.8p52;
  double r = fma(-k, 0.25 * kTwoPi1, x);
  r = fma(-k, 0.25 * kTwoPi2, r);
  const int quad = __double2loint(big) & 3;
  Dd a;
  a.h = static_cast<float>(r);
  a.l = static_cast<float>(r - static_cast<double>(a.h));
  const Dd z = mul(a, a);
  constexpr float s4 = -1.0 / 5040, s5 = 1.0 / 362880, s6 = -1.0 / 39916800, s7 = 1.0 / 6227020800.0;
  Dd v = {fmaf(z.h, fmaf(z.h, fmaf(z.h, s7, s6), s5), s4), 0.f};
  v = horner(1.0 / 120, z, v);
  v = horner(-1.0 / 6, z, v);
  v = mul(mul(z, v), a);
  const Dd t = fast_sum(a.h, v.h);
  const Dd sn = fast_sum(t.h, __fadd_rn(t.l, __fadd_rn(v.l, a.l)));
  constexpr float c4 = 1.0 / 40320, c5 = -1.0 / 3628800, c6 = 1.0 / 479001600, c7 = -1.0 / 87178291200.0;
  Dd u = {fmaf(z.h, fmaf(z.h, fmaf(z.h, c7, c6), c5), c4), 0.f};
  u = horner(-1.0 / 720, z, u);
  u = horner(1.0 / 24, z, u);
  u = horner(-0.5, z, u);
  u = horner(1.0, z, u);
  const Dd cs = fast_sum(u.h, u.l);
  const Dd cc = quad & 1 ? sn : cs, ss = quad & 1 ? cs : sn;
  const float fc = (quad == 1 || quad == 2) ? -1.f : 1.f, fs = quad >= 2 ? -1.f : 1.f;
  *c = {fc * cc.h, fc * cc.l};
  *s = {fs * ss.h, fs * ss.l};
}

// sum over the L lanes that hold a row
template <int L>
__device__ __forceinline__ Dd row_sum(Dd v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1)
    v = add(v, {__shfl_xor_sync(0xffffffffu, v.h, off), __shfl_xor_sync(0xffffffffu, v.l, off)});
  return v;
}

// 1 / sqrt(mean + eps) of the row of d values that L lanes hold, by one Newton
// step on the fp32 root: with r0 = (1 + e) / sqrt(h), r0 (1 + (1 - h r0^2) / 2)
// is within 1.5 e^2. Squares at the ends of the fp32 range, or beyond, are formed
// of values scaled by 2^-70 or 2^60 (*scale): the root then is that of the scaled
// row, which goes with x *scale. (All lanes of the warp take part.)
template <int L>
__device__ __noinline__ Dd inv_rms(const float (&x)[8], float eps, float* scale) {
  constexpr float inv_d = 1.f / (8 * L);  // a power of two
  float sc = 1.f;
  Dd v = {0.f, 0.f};
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    Dd sum = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = add(sum, two_prod(x[i] * sc, x[i] * sc));
    sum = row_sum<L>(sum);
    v = add({sum.h * inv_d, sum.l * inv_d}, {eps * sc * sc, 0.f});
    if (round == 0) sc = !(v.h < 0x1p113f) ? 0x1p-70f : v.h < 0x1p-100f ? 0x1p60f : 1.f;
    if (!__any_sync(0xffffffffu, sc != 1.f)) break;
  }
  *scale = sc;
  const float r = rsqrtf(v.h);
  const Dd q = two_prod(r, r);
  float e = fmaf(-v.h, q.h, 1.f);
  e = fmaf(-v.h, q.l, e);
  e = fmaf(-v.l, q.h, e);
  return {r, 0.5f * r * e};
}

// The same in fp32, within 8.5 2^-24 for bf16 values: their squares are exact,
// four sums in a lane, four between lanes and the one with eps 2^-24 each, half
// of them in the root; rsqrtf adds two units of 2^-23. inf, 0 or NaN where the
// sum leaves the range.
template <int L>
__device__ __forceinline__ float fast_inv_rms(const float (&x)[8], float eps) {
  float a = x[0] * x[0], b = x[4] * x[4];
#pragma unroll
  for (int i = 1; i < 4; ++i) a = fmaf(x[i], x[i], a), b = fmaf(x[4 + i], x[4 + i], b);
  float s = a + b;
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return rsqrtf(fmaf(s, 1.f / (8 * L), eps));
}

// hi + lo rounded once to bf16: hi with its last bit made sticky (odd where
// something is left), which bf16's 16 fewer bits then round correctly
__device__ __forceinline__ float round_bf16_once(Dd v) {
  const Dd n = fast_sum(v.h, v.l);
  uint32_t b = __float_as_uint(n.h);
  if (n.l != 0.f && !(b & 1u) && isfinite(n.h)) b += (n.l > 0.f) == (n.h > 0.f) ? 1u : 0xffffffffu;
  return __bfloat162float(__float2bfloat16_rn(__uint_as_float(b)));
}

__device__ __forceinline__ float approx_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool NAN_STAYS>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (NAN_STAYS)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool NAN_STAYS>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (NAN_STAYS)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 8 values of a row of T
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* src, long long at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + at);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = bf16lo_to_f32(w.x), x[1] = bf16hi_to_f32(w.x), x[2] = bf16lo_to_f32(w.y), x[3] = bf16hi_to_f32(w.y);
    x[4] = bf16lo_to_f32(w.z), x[5] = bf16hi_to_f32(w.z), x[6] = bf16lo_to_f32(w.w), x[7] = bf16hi_to_f32(w.w);
  }
};
template <>
struct Piece<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* src, long long at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
    a = p[0], b = p[1];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t e5m2_pair(uint32_t w) {  // (a NaN keeps its sign)
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(bf16hi_to_f32(w)), "f"(bf16lo_to_f32(w)));
  return r | (w >> 8 & 0x80u) | (w >> 16 & 0x8000u);
}

// A row of bf16 values (fp32 for an fp32 cache) as the cache holds it: x this
// lane's 8 from place 8 at on, row its index. L lanes hold it; `live`: it is
// stored (all lanes of the warp come here).
template <int CACHE, int L, typename T>
__device__ __forceinline__ void store_row(void* cache, void* sz, long long row, int at, bool live, const Piece<T>& x) {
  constexpr int D = 8 * L;
  if constexpr (CACHE == kDtypeF32) {
    if (!live) return;
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(cache) + row * D + 8 * at);
    dst[0] = x.a, dst[1] = x.b;
  } else if constexpr (CACHE == kDtypeBf16) {
    if (live) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + row * D + 8 * at) = x.w;
  } else if constexpr (CACHE == kDtypeF8) {
    if (live)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + 8 * at) =
          make_uint2(e5m2_pair(x.w.x) | e5m2_pair(x.w.y) << 16, e5m2_pair(x.w.z) | e5m2_pair(x.w.w) << 16);
  } else {
    // (maximum, -minimum) of the row
    constexpr bool kNan = CACHE == kDtypeU4;
    const uint32_t mx = max2<kNan>(max2<kNan>(x.w.x, x.w.y), max2<kNan>(x.w.z, x.w.w));
    const uint32_t mn = min2<kNan>(min2<kNan>(x.w.x, x.w.y), min2<kNan>(x.w.z, x.w.w)) ^ 0x80008000u;
    uint32_t r = max2<kNan>(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) r = max2<kNan>(r, __shfl_xor_sync(0xffffffffu, r, off));
    if (!live) return;
    const float hi = bf16lo_to_f32(r), lo = -bf16hi_to_f32(r);
    float v[8];
    x.values(v);
    if constexpr (CACHE == kDtypeU8) {
      const float2 p = u8_params(lo, hi);
      uint32_t w[2] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i / 4] |= u8_code(v[i], p) << (8 * (i % 4));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + 8 * at) = make_uint2(w[0], w[1]);
      if (at == 0) static_cast<float2*>(sz)[row] = p;
    } else {
      const bool finite = hi < INFINITY && lo > -INFINITY;
      const uint32_t pair = finite ? u4_pair(u4_clamp(lo), u4_clamp(hi)) : kU4NanPair;
      float s = u4_scale(pair), m = u4_min(pair);
      uint32_t w = 0;
      if (u4_plain(lo, hi, s)) {
        w = u4_codes(v, s, m, approx_rcp(s));
      } else if (s > 0.f) {  // (not 0, not NaN: codes 0)
        const float up = s < 0x1p-100f ? 0x1p64f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u4_clamp(v[i]) * up;
        w = u4_codes(v, s * up, m * up, approx_rcp(s * up));
      }
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(cache) + row * (D / 2) + 4 * at) = w;
      if (at == 0) static_cast<uint32_t*>(sz)[row] = pair;
    }
  }
}

// A key row in pairs of floats: x the row, w its weights (norm), cs and low the
// lane's (cos, sin) and what their rounding left; y rounded once to T.
template <int L, typename T>
__device__ __noinline__ void exact_key(const Piece<T>& k, const float (&w)[8], bool norm, float eps, const float2* cs,
                                       const float2* low, Piece<T>& out) {
  float x[8], y[8], scale = 1.f;
  k.values(x);
  Dd r = {1.f, 0.f};
  if (norm) r = inv_rms<L>(x, eps, &scale);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const Dd c = {cs[j / 2].x, low[j / 2].x}, s = {cs[j / 2].y, low[j / 2].y};
    Dd a = {x[j], 0.f}, e = {x[j + 1], 0.f}, root = r;
    if (norm) {
      // (a row above 2^56 has small values as they are: scaled, they would leave the normal numbers)
      const bool as_is = scale < 1.f && fmaxf(fabsf(x[j]), fabsf(x[j + 1])) <= 1.f;
      const float f = as_is ? 1.f : scale;
      a = two_prod(x[j] * f, w[j]);
      e = two_prod(x[j + 1] * f, w[j + 1]);
      if (as_is) root = {r.h * scale, r.l * scale};
    }
    const Dd es = mul(e, s), ec = mul(e, c);
    Dd u = add(mul(a, c), {-es.h, -es.l}), v = add(mul(a, s), ec);
    if (norm) {
      u = mul(u, root);
      v = mul(v, root);
    }
    if constexpr (std::is_same<T, float>::value) {
      y[j] = __fadd_rn(u.h, u.l);
      y[j + 1] = __fadd_rn(v.h, v.l);
    } else {
      y[j] = round_bf16_once(u);
      y[j + 1] = round_bf16_once(v);
    }
  }
  if constexpr (std::is_same<T, float>::value) {
    out.a = make_float4(y[0], y[1], y[2], y[3]);
    out.b = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    out.w = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  }
}

// 8 floats; `wide`: their place is a multiple of 32 bytes
__device__ __forceinline__ void store8(float* dst, const float (&y)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(dst), "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]) : "memory");
  } else {
    reinterpret_cast<float4*>(dst)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
}

// TOK tokens a block; blockIdx.y: a share of the heads (TOK = 1). Q groups of
// query rows at a time.
template <int CACHE, int D, int TOK, int Q>
__global__ void __launch_bounds__(kNormThreads, 4) append_norm_kernel(const NormAppendParams p) {
  using T = typename std::conditional<CACHE == kDtypeF32, float, __nv_bfloat16>::type;
  constexpr int L = D / 8, kRows = 32 / L, kHalf = D / 2;
  __shared__ __align__(16) float2 s_cs[TOK][kHalf], s_low[TOK][kHalf];  // (cos, sin), and what their rounding left
  __shared__ long long s_row[TOK];                                     // kv head 0's row of the token, or -1
  grid_dependents_launch();  // the attention launch of the same step may start its prologue
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = p.batch * p.n_new, bt0 = blockIdx.x * TOK;  // (sequence, new token)
  for (int i = threadIdx.x; i < TOK * kHalf; i += kNormThreads) {
    const int tok = i / kHalf, t = i % kHalf, bt = bt0 + tok;
    if (bt >= tokens) break;
    const int b = bt / p.n_new, pos = p.pos[b] + (bt - b * p.n_new);
    int at = pos;
    if (p.axis_pos != nullptr) {
      int axis = 0;
      while (axis < kMaxAxes - 1 && t >= p.section_end[axis]) ++axis;
      at = p.axis_pos[static_cast<long long>(axis) * tokens + bt];
    }
    Dd c, s;
    cos_sin(at, p.theta[t], &c, &s);
    s_cs[tok][t] = make_float2(c.h, s.h);
    s_low[tok][t] = make_float2(c.l, s.l);
    if (t != 0) continue;
    long long row = -1;
    int bad = 0;
    if (p.paged) {
      const int lp = pos >= 0 ? pos / p.page_size : p.max_pages;
      if (lp >= p.max_pages) {
        bad = MQA_DEVERR_POS_RANGE;
      } else {
        const int page = p.block_table[static_cast<long long>(b) * p.max_pages + lp];
        if (page < 0 || page >= p.num_pages)
          bad = MQA_DEVERR_PAGE_RANGE;
        else
          row = static_cast<long long>(page) * p.h_kv * p.page_size + pos % p.page_size;
      }
    } else if (pos < 0 || pos >= p.capacity) {
      bad = MQA_DEVERR_POS_RANGE;
    } else {
      row = static_cast<long long>(b) * p.h_kv * p.capacity + pos;
    }
    if (bad && blockIdx.y == 0) atomicOr(p.err, bad);
    s_row[tok] = row;
  }
  if (p.zero != nullptr && blockIdx.x == 0 && blockIdx.y == 0)
    for (int k = threadIdx.x; k < p.zero_count; k += kNormThreads) p.zero[k] = 0;
  __syncthreads();

  const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
  const bool wide = (reinterpret_cast<uintptr_t>(p.q_rot) & 31u) == 0;
  const int at = lane % L, sub = lane / L;  // place in the row, row of the group
  const int here = tokens - bt0 < TOK ? tokens - bt0 : TOK;
  const int kv_items = (p.h_kv + kRows - 1) / kRows, q_items = (p.h_q + kRows * Q - 1) / (kRows * Q);
  for (int it = blockIdx.y * kNormWarps + warp; it < here * (kv_items + q_items); it += gridDim.y * kNormWarps) {
    if (it < here * kv_items) {
      const int tok = TOK == 1 ? 0 : it / kv_items;
      if (s_row[tok] < 0) continue;
      const int h = (it - tok * kv_items) * kRows + sub;
      const bool live = h < p.h_kv;
      const int head = live ? h : p.h_kv - 1;
      const long long src = (static_cast<long long>(bt0 + tok) * p.h_kv + head) * D + 8 * at;
      const long long row = s_row[tok] + head * (p.paged ? static_cast<long long>(p.page_size) : p.capacity);
      Piece<T> k, v, key;
      k.load(p.k_new, src);
      v.load(p.v_new, src);
      float w[8];
      if (norm_k) {
        Piece<T> t;
        t.load(p.k_weight, 8 * at);
        t.values(w);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
      }
      const float2* cs = &s_cs[tok][4 * at];
      bool settled = false;
      if constexpr (CACHE != kDtypeF32) {
        // u = a c - e s with a = x w exact: the product e s, its rounding and the low parts of c and s are added up apart, so
        // that what is left is 2^-24 |u| of each of two sums (and 2^-45 (|a| + |e|)). With a norm r is within 8.5 2^-24 and
        // its product 2^-24; a border's own sum adds 2^-24. A row with squares that leave the range is not settled.
        float x[8], r = 1.f, bound = 3.5f * 0x1p-24f;
        k.values(x);
        if (norm_k) {
          r = fast_inv_rms<L>(x, p.eps);
          bound = 13.f * 0x1p-24f;
        }
        settled = r > 0x1p-58f && r < 0x1p30f;
        const float2* low = &s_low[tok][4 * at];
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 t = cs[j / 2], tl = low[j / 2];
          const float a = x[j] * w[j], e = x[j + 1] * w[j + 1], size = (fabsf(a) + fabsf(e)) * r;
          const float es = e * t.y, ec = e * t.x;
          const float u = __fadd_rn(fmaf(a, t.x, -es), fmaf(a, tl.x, -fmaf(e, tl.y, fmaf(e, t.y, -es)))) * r;
          const float z = __fadd_rn(fmaf(a, t.y, ec), fmaf(a, tl.y, fmaf(e, tl.x, fmaf(e, t.x, -ec)))) * r;
          const float ou = fmaf(fabsf(u), bound, size * 0x1p-36f), oz = fmaf(fabsf(z), bound, size * 0x1p-36f);
          out[j / 2] = pack_bf16x2(__fsub_rn(u, ou), __fsub_rn(z, oz));
          settled = settled && out[j / 2] == pack_bf16x2(__fadd_rn(u, ou), __fadd_rn(z, oz)) &&
                    ((size >= 0x1p-60f && size <= 0x1p120f) || size == 0.f);
        }
        key.w = make_uint4(out[0], out[1], out[2], out[3]);
      }
      if (!__all_sync(0xffffffffu, settled)) exact_key<L>(k, w, norm_k, p.eps, cs, &s_low[tok][4 * at], key);
#pragma unroll 1
      for (int i = 0; i < 2; ++i)  // (one copy of the code: with more the warps wait for instructions)
        store_row<CACHE, L>(i ? p.v_cache : p.k_cache, i ? p.v_sz : p.k_sz, row, at, live, i ? v : key);
      continue;
    }
    const int qi = it - here * kv_items, tok = TOK == 1 ? 0 : qi / q_items;
    const int h0 = (qi - tok * q_items) * (kRows * Q) + sub;
    const long long src = (static_cast<long long>(bt0 + tok) * p.h_q + h0) * D + 8 * at;
    Piece<T> q[Q];
#pragma unroll
    for (int g = 0; g < Q; ++g)  // (a row behind the last head: the first again)
      q[g].load(p.q_new, h0 + g * kRows < p.h_q ? src + g * (kRows * D) : 8 * at);
    float w[8];
    if (norm_q) {
      Piece<T> t;
      t.load(p.q_weight, 8 * at);
      t.values(w);
    }
    float2 cs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[j] = s_cs[tok][4 * at + j];
    float r[Q];
    if (norm_q) {
      bool out_of_range = false;
#pragma unroll
      for (int g = 0; g < Q; ++g) {
        float x[8];
        q[g].values(x);
        r[g] = fast_inv_rms<L>(x, p.eps);
        out_of_range = out_of_range || !(r[g] > 0x1p-58f && r[g] < 0x1p50f);
      }
      if (__any_sync(0xffffffffu, out_of_range)) {
#pragma unroll
        for (int g = 0; g < Q; ++g) {
          float x[8], scale;
          q[g].values(x);
          const float h = inv_rms<L>(x, p.eps, &scale).h;
          r[g] = h * scale;
        }
      }
    }
#pragma unroll
    for (int g = 0; g < Q; ++g) {
      float x[8], y[8];
      q[g].values(x);
      if (norm_q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= w[i] * r[g];
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        y[j] = fmaf(x[j], cs[j / 2].x, -(x[j + 1] * cs[j / 2].y));
        y[j + 1] = fmaf(x[j], cs[j / 2].y, x[j + 1] * cs[j / 2].x);
      }
      if (h0 + g * kRows < p.h_q) store8(p.q_rot + src + g * (kRows * D), y, wide);
    }
  }
}

// A block a token with its heads spread over several blocks, while that fills
// the GPU; with two such blocks an SM and more, several tokens a block, which fill
// its threads with sines and cosines, and more query rows at a time. (One token a
// block and several, 32 and 8 heads of 128 into a 4-bit cache: 640 tokens, one
// block an SM of several, 11.4 and 12.3 us; 1216 tokens, two, 16.0 and 14.6; 2368,
// three, 28.1 and 21.6; 3648, six, 39.9 and 32.0. A bf16 cache alike.)
template <int CACHE, int D>
cudaError_t launch_norm_d(const NormAppendParams& p, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kNormThreads);
  cfg.stream = stream;
  const int tokens = p.batch * p.n_new;
  constexpr int kTok = 512 / D, kRows = 256 / D;
  if (tokens / kTok >= 2 * sms) {
    cfg.gridDim = dim3(static_cast<unsigned>((tokens - 1) / kTok + 1));
    return cudaLaunchKernelEx(&cfg, append_norm_kernel<CACHE, D, kTok, CACHE == kDtypeF32 ? 2 : 4>, p);
  }
  const int items = (p.h_kv + kRows - 1) / kRows + (p.h_q + kRows - 1) / kRows;
  const int most = (items + kNormWarps - 1) / kNormWarps;
  int y = 4 * sms / tokens;
  y = y < 1 ? 1 : y > most ? most : y;
  cfg.gridDim = dim3(static_cast<unsigned>(tokens), static_cast<unsigned>(y));
  return cudaLaunchKernelEx(&cfg, append_norm_kernel<CACHE, D, 1, 1>, p);
}

template <int CACHE>
cudaError_t launch_norm_c(const NormAppendParams& p, int sms, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_norm_d<CACHE, 128>(p, sms, stream) : launch_norm_d<CACHE, 64>(p, sms, stream);
}

}  // namespace

cudaError_t launch_append_norm(const NormAppendParams& p, int sms, cudaStream_t stream) {
  switch (p.cache_dtype) {
    case kDtypeBf16: return launch_norm_c<kDtypeBf16>(p, sms, stream);
    case kDtypeF32: return launch_norm_c<kDtypeF32>(p, sms, stream);
    case kDtypeU8: return launch_norm_c<kDtypeU8>(p, sms, stream);
    case kDtypeF8: return launch_norm_c<kDtypeF8>(p, sms, stream);
    default: return launch_norm_c<kDtypeU4>(p, sms, stream);
  }
}

}  // namespace mqa
