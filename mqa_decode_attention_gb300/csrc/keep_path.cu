// Keeping an accepted path in the caches: in every layer and kv head, the
// rows of the path's nodes move up behind the cached tokens,
//   row pos + path[i]  ->  row pos + i,   i = 0 .. kept - 1,
// in place. path is strictly increasing and starts anywhere at or above 0, so
// path[i] >= i: a row is only ever written at or before the place it came
// from. A block takes (sequence, layer, some kv heads) and moves 16-byte
// pieces in rounds of ascending rows: all of a round's pieces are read, then
// (after a barrier) written. A later round reads rows path[i] >= i, past
// every row an earlier round wrote. Rows already in place are not touched.
//
// Bound: the launch and two dependent memory round trips (the path, then the
// rows) at serving sizes; all layers go into one launch.
#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"

namespace mqa {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 8;  // pieces a thread holds in a round

__global__ void __launch_bounds__(kThreads) keep_path_kernel(const __grid_constant__ KeepParams p) {
  __shared__ long long s_src[kMaxTreeNodes], s_dst[kMaxTreeNodes];  // cache rows of kv head 0
  __shared__ int s_first, s_bad;
  const int tid = threadIdx.x;
  const int b = blockIdx.x, h0 = blockIdx.y * p.heads_per_block;
  const int heads = min(p.heads_per_block, p.h_kv - h0);
  const KeepLayer& L = p.layer[blockIdx.z];
  const int kept = p.num_kept[b], pos = p.pos[b];
  if (tid == 0) {
    s_first = 0x7fffffff;
    s_bad = 0;
  }
  __syncthreads();
  const int count = kept < 0 || kept > p.n ? 0 : kept;
  int bad = 0;
  if (tid == 0) {
    if (kept < 0 || kept > p.n) bad |= static_cast<int>(MQA_DEVERR_TREE);
    if (pos < 0) bad |= static_cast<int>(MQA_DEVERR_POS_RANGE);
  }
  for (int i = tid; i < count; i += kThreads) {
    const int32_t* path = p.path + static_cast<long long>(b) * p.n;
    const int at = path[i], prev = i > 0 ? path[i - 1] : -1;
    if (at <= prev || at >= p.n) {
      bad |= static_cast<int>(MQA_DEVERR_TREE);
      continue;
    }
    const long long t = static_cast<long long>(pos) + at, d = static_cast<long long>(pos) + i;
    if (at != i) atomicMin(&s_first, i);
    if (pos < 0 || t >= p.capacity) {
      bad |= static_cast<int>(MQA_DEVERR_POS_RANGE);
    } else if (!p.paged) {
      s_src[i] = static_cast<long long>(b) * p.h_kv * p.capacity + t;
      s_dst[i] = static_cast<long long>(b) * p.h_kv * p.capacity + d;
    } else if (at != i) {  // (the pages of rows that stay are not looked up)
      const int32_t* table = L.block_table + static_cast<long long>(b) * p.max_pages;
      const int ps = table[t / p.page_size], pd = table[d / p.page_size];
      if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) bad |= static_cast<int>(MQA_DEVERR_PAGE_RANGE);
      s_src[i] = static_cast<long long>(ps) * p.h_kv * p.page_size + t % p.page_size;
      s_dst[i] = static_cast<long long>(pd) * p.h_kv * p.page_size + d % p.page_size;
    }
  }
  if (bad) {
    atomicOr(&s_bad, bad);
    atomicOr(p.err, bad);
  }
  __syncthreads();
  if (s_bad) return;  // nothing of this sequence moves in this layer
  const int first = s_first, rows = count - first;
  if (first >= count) return;

  const long long head_rows = p.paged ? p.page_size : p.capacity;  // cache rows from one kv head to the next
  const int pieces = p.row_bytes / 16;
  const int items = heads * 2 * rows * pieces;  // ((head, K or V), row, piece): rows ascend within a head's cache
  for (int i0 = 0; i0 < items; i0 += kThreads * kPieces) {
    uint4 w[kPieces];
    uint4* to[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int it = i0 + u * kThreads + tid;
      to[u] = nullptr;
      if (it < items) {
        const int piece = it % pieces, x = it / pieces, r = first + x % rows, hv = x / rows;
        unsigned char* cache = static_cast<unsigned char*>(hv & 1 ? L.v : L.k);
        const long long head = static_cast<long long>(h0 + (hv >> 1)) * head_rows;
        w[u] = *(reinterpret_cast<const uint4*>(cache + (s_src[r] + head) * p.row_bytes) + piece);
        to[u] = reinterpret_cast<uint4*>(cache + (s_dst[r] + head) * p.row_bytes) + piece;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      if (to[u] != nullptr) *to[u] = w[u];
  }
  if (L.k_sz != nullptr) {  // uint8: the rows' (scale, zero point)
    const int pairs = heads * 2 * rows;
    for (int i0 = 0; i0 < pairs; i0 += kThreads) {
      const int it = i0 + tid;
      float2 w = make_float2(0.f, 0.f);
      float2* to = nullptr;
      if (it < pairs) {
        const int r = first + it % rows, hv = it / rows;
        float2* sz = hv & 1 ? L.v_sz : L.k_sz;
        const long long head = static_cast<long long>(h0 + (hv >> 1)) * head_rows;
        w = sz[s_src[r] + head];
        to = sz + s_dst[r] + head;
      }
      __syncthreads();
      if (to != nullptr) *to = w;
    }
  }
}

}  // namespace

cudaError_t launch_keep_path(KeepParams p, int layers, int sms, cudaStream_t stream) {
  // kv heads of a block: two, more when the blocks would not be resident at
  // once (eight to an SM): 32 layers x 32 sequences x 8 heads 18.0 us with two
  // heads a block, whose dependent loads then run three times over
  const long long heads = static_cast<long long>(p.batch) * layers * p.h_kv;
  const long long want = (heads + 8ll * sms - 1) / (8ll * sms);
  p.heads_per_block = static_cast<int>(want < 2 ? 2 : (want < p.h_kv ? want : p.h_kv));
  if (p.heads_per_block > p.h_kv) p.heads_per_block = p.h_kv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch), static_cast<unsigned>((p.h_kv + p.heads_per_block - 1) / p.heads_per_block),
                     static_cast<unsigned>(layers));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, keep_path_kernel, p);
}

}  // namespace mqa
