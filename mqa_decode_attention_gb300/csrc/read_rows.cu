// kv_read_rows kernel: rows of a cache of any type as bf16 or fp32 values, in
// the layout of a contiguous cache [batch, h_kv, n_rows, head_dim].
//
// A thread turns 16 neighbouring values (8 bytes of a 4-bit cache, up to 64 of
// an fp32 one) into one or two stores of 32 bytes; kUnroll such pieces of rows
// further on are requested together, so that enough loads are in flight to keep
// the memory busy. uint8: (code - zero) * scale, one subtraction and one
// product in fp32; 4 bit: m + s * code in one fused multiply-add. Then one
// rounding to bf16.
//
// What bounds it is the memory, once a value costs few instructions: with 8
// values a thread, sizes that only the launch knew and conversions of codes
// (a quarter of the rate; here a code is put into a mantissa) half of the time
// was the issue of instructions. 32 x 8 x 4096 rows of 4 bits as bf16 29 us, 5.8
// TB/s, 86% of the copy rate (34 so); 24 ragged prefixes of uint8 pages as fp32
// 42 us, 5.5 TB/s (48).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "u4.cuh"

namespace mqa {
namespace {

constexpr int kReadThreads = 256;
constexpr int kUnroll = 4;

// code of 8 bits, byte b of w, as a float
template <int B>
__device__ __forceinline__ float byte_value(uint32_t w) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + B)) - 0x1p23f;
}

template <int CACHE>
struct Piece;  // 16 values as they are stored, and what their row adds
template <>
struct Piece<kDtypeU4> {
  uint2 w;
  uint32_t pair;
  __device__ __forceinline__ void load(const void* c, const void* sz, long long row, long long at) {
    w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c) + at / 2);
    pair = static_cast<const uint32_t*>(sz)[row];
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
    const float s = u4_scale(pair), m = u4_min(pair);
    const uint32_t half[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
    // (a code of bits 4 j .. 4 j + 3 is c in the mantissa of 2^(23 - 4 j))
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t one = 0x4b000000u - i % 4 * 0x02000000u;
      x[i] = fmaf(__uint_as_float((half[i / 4] & (15u << (4 * (i % 4)))) | one) - __uint_as_float(one), s, m);
    }
  }
};
template <>
struct Piece<kDtypeU8> {
  uint4 w;
  float2 sz;
  __device__ __forceinline__ void load(const void* c, const void* s, long long row, long long at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c) + at);
    sz = static_cast<const float2*>(s)[row];
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = byte_value<0>(v[i]), x[4 * i + 1] = byte_value<1>(v[i]);
      x[4 * i + 2] = byte_value<2>(v[i]), x[4 * i + 3] = byte_value<3>(v[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__fsub_rn(x[i], sz.y), sz.x);
  }
};
template <>
struct Piece<kDtypeF8> {
  uint4 w;
  __device__ __forceinline__ void load(const void* c, const void*, long long, long long at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c) + at);
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {  // an e5m2 code is the high byte of a half
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>((v[i / 4] >> (8 * (i % 4)) & 255u) << 8)));
  }
};
template <>
struct Piece<kDtypeBf16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const void* c, const void*, long long, long long at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c) + at);
    w[0] = p[0], w[1] = p[1];
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[8 * i] = bf16lo_to_f32(w[i].x), x[8 * i + 1] = bf16hi_to_f32(w[i].x);
      x[8 * i + 2] = bf16lo_to_f32(w[i].y), x[8 * i + 3] = bf16hi_to_f32(w[i].y);
      x[8 * i + 4] = bf16lo_to_f32(w[i].z), x[8 * i + 5] = bf16hi_to_f32(w[i].z);
      x[8 * i + 6] = bf16lo_to_f32(w[i].w), x[8 * i + 7] = bf16hi_to_f32(w[i].w);
    }
  }
};
template <>
struct Piece<kDtypeF32> {
  float4 v[4];
  __device__ __forceinline__ void load(const void* c, const void*, long long, long long at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(c) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * i] = v[i].x, x[4 * i + 1] = v[i].y, x[4 * i + 2] = v[i].z, x[4 * i + 3] = v[i].w;
  }
};

// 32 bytes; `wide`: their place is a multiple of 32
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// blockIdx.x: chunk of rows of one (sequence, kv head), all of them in order;
// blockIdx.y: K or V
template <int CACHE, int D, bool PAGED, bool BF16>
__global__ void __launch_bounds__(kReadThreads) read_rows_kernel(const ReadParams p, int chunks, int page_shift) {
  constexpr int kPerRow = D / 16, kPass = kReadThreads / kPerRow;
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x - unit * chunks;  // unit: sequence * h_kv + head
  const int b = unit / p.h_kv;
  const int start = p.start != nullptr ? p.start[b] : 0, rows = p.num_rows != nullptr ? p.num_rows[b] : p.n_rows;
  int bad = 0;
  if (rows < 0 || rows > p.n_rows)
    bad = MQA_DEVERR_SEQ_LEN;
  else if (rows > 0 && (start < 0 || start > p.limit - rows))
    bad = MQA_DEVERR_POS_RANGE;
  if (bad) {
    if (chunk == 0 && unit == b * p.h_kv && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.err, bad);
    return;
  }
  const int at = threadIdx.x % kPerRow * 16;
  const unsigned row0 = static_cast<unsigned>(chunk) * (kPass * kUnroll) + threadIdx.x / kPerRow;  // (past 2^31 behind the last row)
  if (row0 >= static_cast<unsigned>(rows)) return;
  const int first = static_cast<int>(row0);
  const void* cache = blockIdx.y ? p.v_cache : p.k_cache;
  const void* sz = blockIdx.y ? p.v_sz : p.k_sz;
  Piece<CACHE> piece[kUnroll];
  bool live[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    live[u] = u * kPass < rows - first;
    if (!live[u]) continue;
    const int t = start + first + u * kPass;
    long long row;
    if constexpr (PAGED) {
      const int page = p.block_table[static_cast<long long>(b) * p.max_pages + (t >> page_shift)];
      if (page < 0 || page >= p.num_pages) {
        live[u] = false;
        atomicOr(p.err, static_cast<int>(MQA_DEVERR_PAGE_RANGE));
        continue;
      }
      row = ((static_cast<long long>(page) * p.h_kv + (unit - b * p.h_kv)) << page_shift) + (t & (p.page_size - 1));
    } else {
      row = unit * p.capacity + t;
    }
    piece[u].load(cache, sz, row, row * D + at);
  }
  void* out = blockIdx.y ? p.v_out : p.k_out;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (!live[u]) continue;
    const long long dst = (static_cast<long long>(unit) * p.n_rows + first + u * kPass) * D + at;
    float x[16];
    piece[u].values(x);
    uint32_t w[8];
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      store32(static_cast<__nv_bfloat16*>(out) + dst, w, wide);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[8 * h + i]);
        store32(static_cast<float*>(out) + dst + 8 * h, w, wide);
      }
    }
  }
}

template <int CACHE, int D, bool PAGED>
cudaError_t launch_read_d(const ReadParams& p, cudaStream_t stream) {
  constexpr int kPerBlock = kReadThreads / (D / 16) * kUnroll;
  const int chunks = (p.n_rows - 1) / kPerBlock + 1;
  int shift = 0;
  while (PAGED && (1 << shift) < p.page_size) ++shift;
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(chunks) * p.batch * p.h_kv), 2);
  if (p.out_dtype == kDtypeBf16)
    read_rows_kernel<CACHE, D, PAGED, true><<<grid, kReadThreads, 0, stream>>>(p, chunks, shift);
  else
    read_rows_kernel<CACHE, D, PAGED, false><<<grid, kReadThreads, 0, stream>>>(p, chunks, shift);
  return cudaGetLastError();
}

template <int CACHE>
cudaError_t launch_read_c(const ReadParams& p, cudaStream_t stream) {
  if (p.head_dim == 128) return p.paged ? launch_read_d<CACHE, 128, true>(p, stream) : launch_read_d<CACHE, 128, false>(p, stream);
  return p.paged ? launch_read_d<CACHE, 64, true>(p, stream) : launch_read_d<CACHE, 64, false>(p, stream);
}

}  // namespace

cudaError_t launch_read_rows(const ReadParams& p, cudaStream_t stream) {
  switch (p.cache_dtype) {
    case kDtypeBf16: return launch_read_c<kDtypeBf16>(p, stream);
    case kDtypeF32: return launch_read_c<kDtypeF32>(p, stream);
    case kDtypeU8: return launch_read_c<kDtypeU8>(p, stream);
    case kDtypeF8: return launch_read_c<kDtypeF8>(p, stream);
    default: return launch_read_c<kDtypeU4>(p, stream);
  }
}

}  // namespace mqa
