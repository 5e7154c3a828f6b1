// kv_append_norm_rope kernel, and kv_append_rope over a 4-bit cache: each
// query and key head is normalised (y = x / sqrt(mean x^2 + eps) * w, when
// weights are given), its adjacent pairs are turned by their position -- one
// position, or one of up to four axes for each section of the pairs -- and the
// rows go where they belong: q as fp32 to q_rot, k and v into the cache in its
// type.
//
// A stored key is the 64-bit result rounded once to the type of k_new; a
// one-byte or 4-bit cache holds that bf16 row encoded. A rounding that falls the
// other way changes a whole code there, so the key is formed in pairs of floats
// (a value and what its rounding left, 2^-37 of the pair's length and better)
// instead of fp64, whose rate on this part is 1/64 of fp32's: sine and cosine
// from their Taylor series about the nearest multiple of pi / 2 (only the
// reduction of the angle is fp64: 7 operations for each pair of a token), the
// sum of squares and its root likewise. A query, which fp32 holds, takes the
// fp32 part alone.
//
// One warp forms a row, a lane 4 (d = 128) or 2 (d = 64) neighbouring values.
// A block serves one token: its d / 2 sines and cosines are formed once, then
// its warps take the heads. What bounds it is the memory: a prompt writes 4
// bytes for each value of q it reads.
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
// multiple k of pi / 2 in fp64 (three parts of pi / 2, as reduce_two_pi), then
// both series in z = r^2, |r| <= pi / 4: the terms that are below 2^-14 of the
// result are summed in fp32, the others as pairs (error 2^-37).
__device__ __forceinline__ void cos_sin(int pos, double theta, Dd* c, Dd* s) {
  const double x = static_cast<double>(pos) * theta;
  const double k = rint(x * (4.0 * kInvTwoPi));
  double r = fma(-k, 0.25 * kTwoPi1, x);
  r = fma(-k, 0.25 * kTwoPi2, r);
  r = fma(-k, 0.25 * kTwoPi3, r);
  const int quad = static_cast<int>(static_cast<long long>(k) & 3);
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

__device__ __forceinline__ Dd warp_sum(Dd v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    v = add(v, {__shfl_xor_sync(0xffffffffu, v.h, off), __shfl_xor_sync(0xffffffffu, v.l, off)});
  return v;
}

// 1 / sqrt(mean + eps) of the row whose values the lanes hold, by one Newton
// step on the fp32 root: with r0 = (1 + e) / sqrt(h), r0 (1 + (1 - h r0^2) / 2)
// is within 1.5 e^2. Squares that leave the fp32 range are formed of values
// scaled by 2^-70.
template <int N>
__device__ __forceinline__ Dd inv_rms(const float (&x)[N], int d, float eps) {
  Dd sum = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) sum = add(sum, two_prod(x[i], x[i]));
  sum = warp_sum(sum);
  float down = 1.f;
  if (!(sum.h < 0x1p120f)) {  // the same for all lanes
    down = 0x1p-70f;
    sum = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) sum = add(sum, two_prod(x[i] * down, x[i] * down));
    sum = warp_sum(sum);
  }
  const float inv_d = 1.f / static_cast<float>(d);  // a power of two
  const Dd v = add({sum.h * inv_d, sum.l * inv_d}, {eps * (down * down), 0.f});
  const float r = rsqrtf(v.h);
  const Dd q = two_prod(r, r);
  float e = fmaf(-v.h, q.h, 1.f);
  e = fmaf(-v.h, q.l, e);
  e = fmaf(-v.l, q.h, e);
  return {r * down, 0.5f * r * e * down};
}

// hi + lo rounded once to bf16: hi with its last bit made sticky (odd where
// something is left), which bf16's 16 fewer bits then round correctly
__device__ __forceinline__ float round_bf16_once(Dd v) {
  const Dd n = fast_sum(v.h, v.l);
  uint32_t b = __float_as_uint(n.h);
  if (n.l != 0.f && !(b & 1u) && isfinite(n.h)) b += (n.l > 0.f) == (n.h > 0.f) ? 1u : 0xffffffffu;
  return __bfloat162float(__float2bfloat16_rn(__uint_as_float(b)));
}

template <typename T, int N>
__device__ __forceinline__ void load_row(const void* src, long long at, float (&x)[N]) {
  if constexpr (std::is_same<T, float>::value) {
    const float* p = static_cast<const float*>(src) + at;
    if constexpr (N == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      x[0] = v.x, x[1] = v.y;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(src) + at;
    if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      x[0] = bf16lo_to_f32(v.x), x[1] = bf16hi_to_f32(v.x), x[2] = bf16lo_to_f32(v.y), x[3] = bf16hi_to_f32(v.y);
    } else {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
      x[0] = bf16lo_to_f32(v), x[1] = bf16hi_to_f32(v);
    }
  }
}

// A row of bf16 values (fp32 for an fp32 cache) as the cache holds it, row =
// its index; lane's values N lane ..
template <int CACHE, int N>
__device__ __forceinline__ void store_row(void* cache, void* sz, long long row, int lane, const float (&x)[N]) {
  constexpr int D = 32 * N;
  if constexpr (CACHE == kDtypeF32) {
    float* dst = static_cast<float*>(cache) + row * D + N * lane;
    if constexpr (N == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
  } else if constexpr (CACHE == kDtypeBf16) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(cache) + row * D + N * lane);
    if constexpr (N == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else
      *dst = pack_bf16x2(x[0], x[1]);
  } else {
    uint32_t code[N] = {};
    if constexpr (CACHE == kDtypeF8) {
#pragma unroll
      for (int i = 0; i < N; ++i) code[i] = e5m2_code_f(x[i]);
    } else {
      float lo = x[0], hi = x[0];
      bool bad = false;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad |= !isfinite(x[i]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      }
      if constexpr (CACHE == kDtypeU8) {
        const float2 p = u8_params(lo, hi);
#pragma unroll
        for (int i = 0; i < N; ++i) code[i] = u8_code(x[i], p);
        if (lane == 0) static_cast<float2*>(sz)[row] = p;
      } else {
        lo = u4_clamp(lo), hi = u4_clamp(hi);
        const uint32_t pair = __any_sync(0xffffffffu, bad) ? kU4NanPair : u4_pair(lo, hi);
        const float s0 = u4_scale(pair);
        const float up = s0 < 0x1p-100f ? 0x1p64f : 1.f;  // (a NaN scale gives codes 0 below)
        const float s = s0 * up, m = u4_min(pair) * up, inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) w |= (s > 0.f ? u4_code(u4_clamp(x[i]) * up, s, m, inv) : 0u) << (4 * i);
        uint8_t* dst = static_cast<uint8_t*>(cache) + row * (D / 2) + N / 2 * lane;
        if constexpr (N == 4)
          *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w);
        else
          *dst = static_cast<uint8_t>(w);
        if (lane == 0) static_cast<uint32_t*>(sz)[row] = pair;
        return;
      }
    }
    uint8_t* dst = static_cast<uint8_t*>(cache) + row * D + N * lane;
    if constexpr (N == 4)
      *reinterpret_cast<uint32_t*>(dst) = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
    else
      *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(code[0] | code[1] << 8);
  }
}

template <int CACHE, int D>
__global__ void __launch_bounds__(kNormThreads) append_norm_kernel(const NormAppendParams p) {
  using T = typename std::conditional<CACHE == kDtypeF32, float, __nv_bfloat16>::type;
  constexpr int N = D / 32, kHalf = D / 2;
  __shared__ Dd s_cos[kHalf], s_sin[kHalf];
  grid_dependents_launch();  // the attention launch of the same step may start its prologue
  const int bt = blockIdx.x;  // (sequence, new token)
  const int b = bt / p.n_new, i = bt - b * p.n_new;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pos = p.pos[b] + i;
  if (threadIdx.x < kHalf) {
    int at = pos;
    if (p.axis_pos != nullptr) {
      int axis = 0;
      while (axis < kMaxAxes - 1 && static_cast<int>(threadIdx.x) >= p.section_end[axis]) ++axis;
      at = p.axis_pos[static_cast<long long>(axis) * p.batch * p.n_new + bt];
    }
    cos_sin(at, p.theta[threadIdx.x], &s_cos[threadIdx.x], &s_sin[threadIdx.x]);
  }
  if (p.zero != nullptr && blockIdx.x == 0 && blockIdx.y == 0)
    for (int k = threadIdx.x; k < p.zero_count; k += kNormThreads) p.zero[k] = 0;
  __syncthreads();

  // the place of the token's rows, of kv head 0, and from one head to the next
  long long row0 = -1, stride = 0;
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
        row0 = static_cast<long long>(page) * p.h_kv * p.page_size + pos % p.page_size;
      stride = p.page_size;
    }
  } else if (pos < 0 || pos >= p.capacity) {
    bad = MQA_DEVERR_POS_RANGE;
  } else {
    row0 = static_cast<long long>(b) * p.h_kv * p.capacity + pos;
    stride = p.capacity;
  }
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, bad);

  const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
  float wq[N], wk[N];
  if (norm_q) load_row<T>(p.q_weight, N * lane, wq);
  if (norm_k) load_row<T>(p.k_weight, N * lane, wk);
  // the kv heads first: theirs is the longer work
  const int rows = p.h_kv + p.h_q;
  for (int h = blockIdx.y * kNormWarps + warp; h < rows; h += gridDim.y * kNormWarps) {
    float x[N];
    if (h >= p.h_kv) {
      const long long at = (static_cast<long long>(bt) * p.h_q + (h - p.h_kv)) * D + N * lane;
      load_row<T>(p.q_new, at, x);
      float r = 1.f;
      if (norm_q) r = inv_rms(x, D, p.eps).h;
      float y[N];
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const int t = (N * lane + j) / 2;
        const float c = s_cos[t].h, s = s_sin[t].h;
        const float a = norm_q ? x[j] * wq[j] * r : x[j], e = norm_q ? x[j + 1] * wq[j + 1] * r : x[j + 1];
        y[j] = fmaf(a, c, -(e * s));
        y[j + 1] = fmaf(a, s, e * c);
      }
      if constexpr (N == 4)
        *reinterpret_cast<float4*>(p.q_rot + at) = make_float4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<float2*>(p.q_rot + at) = make_float2(y[0], y[1]);
      continue;
    }
    if (row0 < 0) continue;
    const long long at = (static_cast<long long>(bt) * p.h_kv + h) * D + N * lane, row = row0 + h * stride;
    float v[N];
    load_row<T>(p.k_new, at, x);
    load_row<T>(p.v_new, at, v);
    Dd r = {1.f, 0.f};
    if (norm_k) r = inv_rms(x, D, p.eps);
    float y[N];
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const int t = (N * lane + j) / 2;
      const Dd c = s_cos[t], s = s_sin[t];
      Dd a = {x[j], 0.f}, e = {x[j + 1], 0.f};
      if (norm_k) {
        a = two_prod(x[j], wk[j]);
        e = two_prod(x[j + 1], wk[j + 1]);
      }
      const Dd es = mul(e, s), ec = mul(e, c);
      Dd u = add(mul(a, c), {-es.h, -es.l}), w = add(mul(a, s), ec);
      if (norm_k) {
        u = mul(u, r);
        w = mul(w, r);
      }
      if constexpr (CACHE == kDtypeF32) {
        y[j] = __fadd_rn(u.h, u.l);
        y[j + 1] = __fadd_rn(w.h, w.l);
      } else {
        y[j] = round_bf16_once(u);
        y[j + 1] = round_bf16_once(w);
      }
    }
    store_row<CACHE>(p.k_cache, p.k_sz, row, lane, y);
    store_row<CACHE>(p.v_cache, p.v_sz, row, lane, v);
  }
}

template <int CACHE>
cudaError_t launch_norm_c(const NormAppendParams& p, dim3 grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kNormThreads);
  cfg.stream = stream;
  return p.head_dim == 128 ? cudaLaunchKernelEx(&cfg, append_norm_kernel<CACHE, 128>, p)
                           : cudaLaunchKernelEx(&cfg, append_norm_kernel<CACHE, 64>, p);
}

}  // namespace

cudaError_t launch_append_norm(const NormAppendParams& p, int sms, cudaStream_t stream) {
  // few tokens: their heads over several blocks, while that fills the GPU
  const long long tokens = static_cast<long long>(p.batch) * p.n_new;
  const int most = (p.h_q + p.h_kv + kNormWarps - 1) / kNormWarps;
  long long y = 4ll * sms / tokens;
  y = y < 1 ? 1 : y > most ? most : y;
  if (y > 65535) y = 65535;
  const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(y));
  switch (p.cache_dtype) {
    case kDtypeBf16: return launch_norm_c<kDtypeBf16>(p, grid, stream);
    case kDtypeF32: return launch_norm_c<kDtypeF32>(p, grid, stream);
    case kDtypeU8: return launch_norm_c<kDtypeU8>(p, grid, stream);
    case kDtypeF8: return launch_norm_c<kDtypeF8>(p, grid, stream);
    default: return launch_norm_c<kDtypeU4>(p, grid, stream);
  }
}

}  // namespace mqa
