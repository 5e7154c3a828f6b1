// The append of a tree of drafted tokens over a bf16 cache: node i of sequence b
// is rotated by its position pos[b] + depth[b, i], its k and v go into cache
// row pos[b] + i, its rotated q (bf16, the attention's operand) into q_rot. The
// cache rows are those of append_rope.cu's kernels bit for bit: k is the fp64
// rotation rounded once, decided from an fp32 rotation wherever its error
// bound settles the rounding (rope_k_bf16_fast), v a copy. (One-byte caches
// take append_rope.cu's kernels.)
//
// A block takes several nodes. Per node it forms the d / 2 reduced angles (fp64)
// and their fp32 sines and cosines once, turns all heads with 16-byte loads and
// stores, and notes the key pairs that fp32 leaves open (about one in a
// thousand). Those are turned in fp64 at the end, all of the block's at once:
// a warp's fp64 sine and cosine keep this part's narrow fp64 pipe busy for some
// 3000 cycles whether one lane needs them or all, and evaluated where they
// occur, as in append_rope.cu, they are half the append's time.
//
// Bound: the HBM stream of q, k, v in and q_rot out from a thousand nodes on,
// below that the chain position - angle - rotation - store. 2048 nodes of 32 + 8
// heads, 50 MB: 11.7 us (append_rope.cu's kernel: 21.7); 512 nodes: 6.2 us (10.4).
//
// One block of 1024 threads an SM: what matters to a step is when the last block
// of each SM leaves, since the attention's blocks need the SM's whole shared
// memory. Steps called one after the other, of 32 x 64 nodes at 4096 keys 174.5 us
// with it, 174.5 with four blocks of 256, 173.8 with two of 512; of 32 x 16 nodes
// 106.3, 108.5, 108.6.
#include <cuda_bf16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace mqa {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxNodes = 16;  // nodes of a block
constexpr int kQueue = 256;    // open pairs a block notes (more are turned where they occur)

template <int D>
__global__ void __launch_bounds__(kThreads) append_tree_kernel(const AppendParams p, int per_block) {
  constexpr int kHalf = D / 2, kUnits = D / 8;  // rotation pairs, 16-byte units of a head's row
  __shared__ double s_ang[kMaxNodes][kHalf];
  __shared__ __align__(16) float s_cos[kMaxNodes][kHalf], s_sin[kMaxNodes][kHalf];
  __shared__ long long s_row[kMaxNodes];  // element offset of the node's row in kv head 0, -1: none to write
  __shared__ int s_live[kMaxNodes];
  __shared__ unsigned s_queue[kQueue];
  __shared__ int s_open;
  grid_dependents_launch();
  const int tid = threadIdx.x;
  const int first = blockIdx.x * per_block, total = p.batch * p.n_new;
  const int count = min(per_block, total - first);
  if (blockIdx.x == 0 && p.zero != nullptr)
    for (int i = tid; i < p.zero_count; i += kThreads) p.zero[i] = 0;
  const long long stride = (p.paged ? static_cast<long long>(p.page_size) : p.capacity) * D;  // from one kv head to the next
  const long long limit = p.paged ? static_cast<long long>(p.max_pages) * p.page_size : p.capacity;  // slots of a sequence
  if (tid == 0) s_open = 0;
  // ---- angles: thread (node, pair); the pair's first thread finds the row
  for (int e = tid; e < count * kHalf; e += kThreads) {
    const int k = e / kHalf, pi = e - k * kHalf, bt = first + k, b = bt / p.n_new, i = bt - b * p.n_new;
    const int pos = p.pos[b], nodes = p.num_nodes != nullptr ? p.num_nodes[b] : p.n_new;
    int depth = p.depth[bt];
    // (at a negative position none: nodes in rows 0, 1, .. would overwrite cached tokens)
    const bool live = nodes >= 0 && nodes <= p.n_new && i < nodes && pos >= 0;
    if (pi == 0) {
      int err = 0;
      if ((nodes < 0 || nodes > p.n_new) && i == 0) err |= static_cast<int>(MQA_DEVERR_SEQ_LEN);
      if (pos < 0 && nodes > 0 && nodes <= p.n_new && i == 0) err |= static_cast<int>(MQA_DEVERR_POS_RANGE);
      long long row = -1;
      if (live) {
        if (depth < 0 || depth >= p.n_new) err |= static_cast<int>(MQA_DEVERR_TREE);
        const long long slot = static_cast<long long>(pos) + i;
        if (slot >= limit) {
          err |= static_cast<int>(MQA_DEVERR_POS_RANGE);
        } else if (!p.paged) {
          row = (static_cast<long long>(b) * p.h_kv * p.capacity + slot) * D;
        } else {
          const int page = p.block_table[static_cast<long long>(b) * p.max_pages + slot / p.page_size];
          if (page < 0 || page >= p.num_pages)
            err |= static_cast<int>(MQA_DEVERR_PAGE_RANGE);
          else
            row = (static_cast<long long>(page) * p.h_kv * p.page_size + slot % p.page_size) * D;
        }
      }
      if (err) atomicOr(p.err, err);
      s_row[k] = row;
      s_live[k] = live;
    }
    depth = min(max(depth, 0), p.n_new - 1);
    const double ang = reduce_two_pi(static_cast<double>(static_cast<long long>(pos) + depth) * p.theta[pi]);
    float sf, cf;
    sincosf(static_cast<float>(ang), &sf, &cf);
    s_ang[k][pi] = ang;
    s_cos[k][pi] = cf;
    s_sin[k][pi] = sf;
  }
  __syncthreads();
  // ---- q: unit (node, head, 8 dims), four in flight
  const uint4* qn = static_cast<const uint4*>(p.q_new) + static_cast<long long>(first) * p.h_q * kUnits;
  uint4* qr = reinterpret_cast<uint4*>(p.q_rot) + static_cast<long long>(first) * p.h_q * kUnits;
  const int q_units = count * p.h_q * kUnits;
  constexpr int kU = 4;
  for (int w0 = tid; w0 < q_units; w0 += kU * kThreads) {
    uint4 raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int w = w0 + u * kThreads;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (w < q_units) raw[u] = qn[w];
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int w = w0 + u * kThreads;
      const int k = w / (p.h_q * kUnits), i0 = (w % kUnits) * 4;
      if (w >= q_units || !s_live[k]) continue;
      const float4 c = *reinterpret_cast<const float4*>(&s_cos[k][i0]), s = *reinterpret_cast<const float4*>(&s_sin[k][i0]);
      auto turn = [](uint32_t v, float c, float s) {
        const float x = bf16lo_to_f32(v), y = bf16hi_to_f32(v);
        return pack_bf16x2(x * c - y * s, x * s + y * c);
      };
      qr[w] = make_uint4(turn(raw[u].x, c.x, s.x), turn(raw[u].y, c.y, s.y), turn(raw[u].z, c.z, s.z),
                         turn(raw[u].w, c.w, s.w));
    }
  }
  // ---- k and v
  const uint4* kn = static_cast<const uint4*>(p.k_new) + static_cast<long long>(first) * p.h_kv * kUnits;
  const uint4* vn = static_cast<const uint4*>(p.v_new) + static_cast<long long>(first) * p.h_kv * kUnits;
  __nv_bfloat16* kc = static_cast<__nv_bfloat16*>(p.k_cache);
  __nv_bfloat16* vc = static_cast<__nv_bfloat16*>(p.v_cache);
  const int kv_units = count * p.h_kv * kUnits;
  for (int w0 = tid; w0 < kv_units; w0 += 2 * kThreads) {
    uint4 rk[2], rv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int w = w0 + u * kThreads;
      rk[u] = rv[u] = make_uint4(0u, 0u, 0u, 0u);
      if (w < kv_units) {
        rk[u] = kn[w];
        rv[u] = vn[w];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int w = w0 + u * kThreads;
      if (w >= kv_units) continue;
      const int k = w / (p.h_kv * kUnits), h = w / kUnits - k * p.h_kv, un = w % kUnits;
      if (s_row[k] < 0) continue;
      const long long dst = s_row[k] + h * stride + 8 * un;
      uint32_t out[4];
      const uint32_t in[4] = {rk[u].x, rk[u].y, rk[u].z, rk[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int pi = 4 * un + e;
        __nv_bfloat162 r;
        if (!rope_k_bf16_fast(bf16lo_to_f32(in[e]), bf16hi_to_f32(in[e]), s_cos[k][pi], s_sin[k][pi], &r)) {
          const int at = atomicAdd(&s_open, 1);
          if (at < kQueue)
            s_queue[at] = static_cast<unsigned>(w) * 4u + static_cast<unsigned>(e);
          else
            r = rope_k_bf16_fp64(bf16lo_to_f32(in[e]), bf16hi_to_f32(in[e]), s_ang[k][pi]);
        }
        out[e] = *reinterpret_cast<const uint32_t*>(&r);  // (a noted pair is written again below)
      }
      *reinterpret_cast<uint4*>(kc + dst) = make_uint4(out[0], out[1], out[2], out[3]);
      *reinterpret_cast<uint4*>(vc + dst) = rv[u];
    }
  }
  __syncthreads();
  // ---- the noted pairs
  const int open = min(s_open, kQueue);
  for (int i = tid; i < open; i += kThreads) {
    const int w = static_cast<int>(s_queue[i] >> 2), e = static_cast<int>(s_queue[i] & 3u);
    const int k = w / (p.h_kv * kUnits), h = w / kUnits - k * p.h_kv, un = w % kUnits;
    const uint32_t in = reinterpret_cast<const uint32_t*>(kn)[static_cast<long long>(w) * 4 + e];
    const __nv_bfloat162 r = rope_k_bf16_fp64(bf16lo_to_f32(in), bf16hi_to_f32(in), s_ang[k][4 * un + e]);
    *reinterpret_cast<__nv_bfloat162*>(kc + s_row[k] + h * stride + 8 * un + 2 * e) = r;
  }
}

}  // namespace

cudaError_t launch_append_tree(const AppendParams& p, int sms, cudaStream_t stream) {
  const int total = p.batch * p.n_new;
  int per = (total + sms - 1) / sms;  // nodes of a block
  per = per < 1 ? 1 : (per > kMaxNodes ? kMaxNodes : per);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((total + per - 1) / per));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  return p.head_dim == 128 ? cudaLaunchKernelEx(&cfg, append_tree_kernel<128>, p, per)
                           : cudaLaunchKernelEx(&cfg, append_tree_kernel<64>, p, per);
}

}  // namespace mqa
