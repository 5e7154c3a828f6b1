// kv_read_rows kernel: rows of a cache of any type as bf16 or fp32 values, in
// the layout of a contiguous cache [batch, h_kv, n_rows, head_dim].
//
// A thread turns 8 neighbouring values (4 bytes of a 4-bit cache, up to 32 of
// an fp32 one) into 16 or 32 bytes; kUnroll such pieces of rows further on are
// requested together, so that enough loads are in flight to keep the memory
// busy, which is all that bounds this kernel. uint8: (code - zero) * scale, one
// subtraction and one product in fp32; 4 bit: m + s * code in one fused
// multiply-add. Then one rounding to bf16.
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

template <int CACHE>
struct Piece;  // 8 values as they are stored, and what their row adds
template <>
struct Piece<kDtypeU4> {
  uint32_t w, pair;
  __device__ __forceinline__ void load(const void* c, const void* sz, long long row, int at, int d) {
    w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c) + row * (d / 2) + at / 2);
    pair = static_cast<const uint32_t*>(sz)[row];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const float s = u4_scale(pair), m = u4_min(pair);
    // (a code in the low bits of 2^23: conversions run at a quarter of the rate)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(__uint_as_float((w >> (4 * i) & 15u) | 0x4b000000u) - 0x1p23f, s, m);
  }
};
template <>
struct Piece<kDtypeU8> {
  uint2 w;
  float2 sz;
  __device__ __forceinline__ void load(const void* c, const void* s, long long row, int at, int d) {
    w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c) + row * d + at);
    sz = static_cast<const float2*>(s)[row];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(i < 4 ? w.x : w.y, 0x4b000000u, 0x7540 + (i & 3))) - 0x1p23f, sz.y), sz.x);
  }
};
template <>
struct Piece<kDtypeF8> {
  uint2 w;
  __device__ __forceinline__ void load(const void* c, const void*, long long row, int at, int d) {
    w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c) + row * d + at);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {  // an e5m2 code is the high byte of a half
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(((i < 4 ? w.x : w.y) >> (8 * (i & 3)) & 255u) << 8)));
  }
};
template <>
struct Piece<kDtypeBf16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* c, const void*, long long row, int at, int d) {
    w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c) + row * d + at);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = bf16lo_to_f32(w.x), x[1] = bf16hi_to_f32(w.x), x[2] = bf16lo_to_f32(w.y), x[3] = bf16hi_to_f32(w.y);
    x[4] = bf16lo_to_f32(w.z), x[5] = bf16hi_to_f32(w.z), x[6] = bf16lo_to_f32(w.w), x[7] = bf16hi_to_f32(w.w);
  }
};
template <>
struct Piece<kDtypeF32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* c, const void*, long long row, int at, int d) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(c) + row * d + at);
    a = p[0], b = p[1];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// blockIdx.x: chunk of rows of one (sequence, kv head), all of them in order;
// blockIdx.y: K or V
template <int CACHE, bool BF16>
__global__ void __launch_bounds__(kReadThreads) read_rows_kernel(const ReadParams p, int chunks) {
  const int per_row = p.head_dim / 8, per_pass = kReadThreads / per_row;
  const int chunk = blockIdx.x % chunks;
  const int unit = blockIdx.x / chunks;  // sequence * h_kv + head
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
  const int at = threadIdx.x % per_row * 8;
  const int first = chunk * per_pass * kUnroll + threadIdx.x / per_row;
  if (first >= rows) return;
  const void* cache = blockIdx.y ? p.v_cache : p.k_cache;
  const void* sz = blockIdx.y ? p.v_sz : p.k_sz;
  Piece<CACHE> piece[kUnroll];
  bool live[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = first + u * per_pass;
    live[u] = i < rows;
    if (!live[u]) continue;
    const int t = start + i;
    long long row;
    if (p.paged) {
      const int page = p.block_table[static_cast<long long>(b) * p.max_pages + t / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        live[u] = false;
        atomicOr(p.err, static_cast<int>(MQA_DEVERR_PAGE_RANGE));
        continue;
      }
      row = (static_cast<long long>(page) * p.h_kv + (unit - b * p.h_kv)) * p.page_size + t % p.page_size;
    } else {
      row = unit * p.capacity + t;
    }
    piece[u].load(cache, sz, row, at, p.head_dim);
  }
  void* out = blockIdx.y ? p.v_out : p.k_out;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (!live[u]) continue;
    const long long dst = (static_cast<long long>(unit) * p.n_rows + first + u * per_pass) * p.head_dim + at;
    float x[8];
    piece[u].values(x);
    if constexpr (BF16) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + dst) =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + dst);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <int CACHE>
cudaError_t launch_read_c(const ReadParams& p, cudaStream_t stream) {
  const int per_block = kReadThreads / (p.head_dim / 8) * kUnroll;
  const int chunks = (p.n_rows + per_block - 1) / per_block;
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(chunks) * p.batch * p.h_kv), 2);
  if (p.out_dtype == kDtypeBf16)
    read_rows_kernel<CACHE, true><<<grid, kReadThreads, 0, stream>>>(p, chunks);
  else
    read_rows_kernel<CACHE, false><<<grid, kReadThreads, 0, stream>>>(p, chunks);
  return cudaGetLastError();
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
