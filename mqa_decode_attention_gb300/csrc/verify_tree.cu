// Verification of a tree of drafted tokens against the target's probabilities
// from given random numbers (speculative sampling over several candidates),
// "Arsitektur Inferensi LLM", section 7: the result follows the target's
// distribution whatever the draft proposes.
//
// Node 0 is the last committed token. From it the walk goes down: p and q are
// the target's and the draft's next-token probabilities after the current
// node, its children c (in index order) are tried one after the other. With
// R_0 = p, S_0 = 1, a child with token x is accepted iff u_c q(x) S_k < R_k(x);
// a rejection leaves the residual max(R_k - S_k q, 0), whose value after k
// rejections is, in closed form,
//   R_k(v) = max(p(v) - c_k q(v), 0),  c_0 = 0,  c_{k+1} = c_k + S_k,  S_k = sum_v R_k(v)
// (where p <= c_k q it stays 0 for every larger c). When no child is left the
// next token is drawn from R_k: the smallest v with cumsum(R_k)(v) > u S_k.
// Without draft probabilities (deterministic drafts) q is 1 at the child's
// token: R_k is p without the rejected tokens, and no sum over the
// vocabulary is needed before the last one.
//
// Only the rows the walk needs are read: those of nodes where a child is
// rejected, and of the node it ends at. What is compared decides tokens, so
// the sums carry 64-bit accuracy: a weight is formed as an unevaluated pair
// of floats (the product's and the difference's rounding errors kept), a
// thread's sum as such a pair (relative error below 2^-44), and everything
// across threads in fp64; the fp64 pipe of this part is too narrow for a
// vocabulary's worth of additions.
//
// A cluster of up to 8 blocks serves one sequence: every block walks the tree
// alike, a sum over the vocabulary is split over the blocks (consecutive
// slices), their warps (consecutive runs) and met through distributed shared
// memory; the block, then the warp whose run holds the goal looks it up.
#include <cuda_bf16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"

namespace mqa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// value = hi + lo
struct Pair {
  float hi, lo;
};

// p - c q as a pair, c = ch + cl; the caller takes it as 0 unless hi + lo > 0
__device__ __forceinline__ Pair residual(float p, float q, float ch, float cl) {
  const float m = __fmul_rn(ch, q);
  const float me = __fmaf_rn(cl, q, __fmaf_rn(ch, q, -m));  // c q = m + me
  const float s = __fsub_rn(p, m);
  const float bb = __fsub_rn(s, p);
  const float se = __fsub_rn(__fsub_rn(p, __fsub_rn(s, bb)), __fadd_rn(m, bb));  // p - m = s + se
  return {s, __fsub_rn(se, me)};
}

__device__ __forceinline__ void add(Pair& a, float hi, float lo) {
  const float s = __fadd_rn(a.hi, hi);
  const float bb = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, bb)), __fsub_rn(hi, bb));
  a.lo = __fadd_rn(a.lo, __fadd_rn(e, lo));
  a.hi = s;
}

__device__ __forceinline__ double dsmem_ld_f64(uint32_t cluster_addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  return static_cast<float>(x);
}

// 16 bytes of a row as floats
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    f[0] = bf16lo_to_f32(w.x), f[1] = bf16hi_to_f32(w.x), f[2] = bf16lo_to_f32(w.y), f[3] = bf16hi_to_f32(w.y);
    f[4] = bf16lo_to_f32(w.z), f[5] = bf16hi_to_f32(w.z), f[6] = bf16lo_to_f32(w.w), f[7] = bf16hi_to_f32(w.w);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_tree_kernel(const VerifyParams p) {
  constexpr int N = Vec<T>::kN;
  __shared__ int s_parent[kMaxTreeNodes], s_token[kMaxTreeNodes], s_path[kMaxTreeNodes];
  __shared__ float s_u[kMaxTreeNodes], s_p[kMaxTreeNodes], s_q[kMaxTreeNodes];
  __shared__ int s_out[kMaxTreeNodes];   // deterministic drafts: tokens rejected at the current node
  __shared__ double s_warp[kWarps];      // sums of the warps' runs
  __shared__ double s_sum[2];            // this block's sum, by the sweep's parity
  __shared__ float s_top[kWarps];
  __shared__ int s_at[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int b = blockIdx.x / cs;
  const int V = p.vocab;
  const T* P = static_cast<const T*>(p.target);
  const T* Q = static_cast<const T*>(p.draft);

  int nodes = p.num_nodes != nullptr ? p.num_nodes[b] : p.n;
  if (nodes < 0 || nodes > p.n) {
    if (tid == 0 && rank == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_SEQ_LEN));
    nodes = 0;
  }
  // the nodes, with both probabilities of each one's token after its parent;
  // a child that names no earlier node or no token is never tried
  for (int i = tid; i < nodes; i += kThreads) {
    const long long at = static_cast<long long>(b) * p.n + i;
    int par = i == 0 ? -1 : p.parents[at];
    const int tok = p.tokens[at];
    s_u[i] = p.u_accept[at];
    float pv = 0.f, qv = 0.f;
    if (i > 0) {
      if (par < 0 || par >= i || tok < 0 || tok >= V) {
        par = -1;
        if (rank == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_TREE));
      } else {
        const long long o = (static_cast<long long>(b) * p.n + par) * p.row_stride + tok;
        pv = to_f32(P[o]);
        if (Q != nullptr) qv = to_f32(Q[o]);
      }
    }
    s_parent[i] = par;
    s_token[i] = tok;
    s_p[i] = pv;
    s_q[i] = qv;
  }
  __syncthreads();

  // this lane's nodes lane + 32 w: their parents (-1: none, and node 0)
  int par[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) par[w] = lane + 32 * w < nodes ? s_parent[lane + 32 * w] : -1;
  auto next_child = [&](int cur, int after) {  // the first child of cur past node `after`, -1: none
    int found = -1;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t hit = __ballot_sync(0xffffffffu, par[w] == cur && lane + 32 * w > after);
      if (found < 0 && hit != 0) found = 32 * w + __ffs(static_cast<int>(hit)) - 1;
    }
    return found;
  };

  // ---- the vocabulary in 16-byte groups of a row (aligned in memory: the
  // first and the last may be cut), shared out to blocks and warps in runs
  long long row = 0;  // element offset of the current row
  int mis = 0, run0 = 0, run1 = 0, per_warp = 1, per_cta = 1;
  auto set_row = [&](int node) {
    row = (static_cast<long long>(b) * p.n + node) * p.row_stride;
    mis = static_cast<int>(row & (N - 1));
    const int groups = (V + mis + N - 1) / N;
    per_cta = (groups + cs - 1) / cs;
    per_warp = (per_cta + kWarps - 1) / kWarps;
    const int end = min(groups, (rank + 1) * per_cta);
    run0 = min(end, rank * per_cta + warp * per_warp);
    run1 = min(end, run0 + per_warp);
  };
  auto load_group = [&](const T* src, int g, float (&f)[N]) {  // elements N g - mis .. + N, zeros outside the row
    const int v0 = N * g - mis;
    if (v0 >= 0 && v0 + N <= V) {
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(src + row + v0)), f);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = v0 + e >= 0 && v0 + e < V ? to_f32(src[row + v0 + e]) : 0.f;
    }
  };

  int rejected = 0;  // entries of s_out (deterministic drafts)
  int parity = 0;
  double cta_sum[kMaxCluster];
  // S of the current row for the coefficient c; leaves s_warp and cta_sum
  auto sweep = [&](double c) {
    const float ch = static_cast<float>(c), cl = static_cast<float>(c - static_cast<double>(ch));
    Pair acc = {0.f, 0.f};
    constexpr int kU = 4;
    for (int g0 = run0 + lane; g0 < run1; g0 += 32 * kU) {
      float fp[kU][N], fq[kU][N];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int g = g0 + 32 * u;
#pragma unroll
        for (int e = 0; e < N; ++e) fp[u][e] = fq[u][e] = 0.f;
        if (g < run1) {
          load_group(P, g, fp[u]);
          if (Q != nullptr && c != 0.0) load_group(Q, g, fq[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const Pair r = residual(fp[u][e], fq[u][e], ch, cl);
          if (__fadd_rn(r.hi, r.lo) > 0.f) add(acc, r.hi, r.lo);  // (NaN: no weight)
        }
    }
    double s = static_cast<double>(acc.hi) + static_cast<double>(acc.lo);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    // deterministic drafts: rejected tokens weigh nothing
    for (int i = 0; i < rejected; ++i) {
      const int g = (s_out[i] + mis) / N;
      if (g >= run0 && g < run1) {
        const float w = to_f32(P[row + s_out[i]]);
        if (w > 0.f) s -= static_cast<double>(w);
      }
    }
    if (lane == 0) s_warp[warp] = s > 0.0 ? s : 0.0;
    __syncthreads();
    double mine = 0.0;
    for (int w = 0; w < kWarps; ++w) mine += s_warp[w];
    if (tid == 0) s_sum[parity] = mine;
    double total = 0.0;
    if (cs > 1) {
      cluster_sync_all();
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        cta_sum[r] = r < cs ? dsmem_ld_f64(dsmem_map(smem_u32(&s_sum[parity]), r)) : 0.0;
        total += cta_sum[r];
      }
    } else {
      cta_sum[0] = total = mine;
    }
    parity ^= 1;
    return total;
  };

  // ---- the walk
  int cur = 0, last = 0, kept = nodes > 0 ? 1 : 0;
  bool swept = false;  // the sums of (cur, c) are there
  double c = 0.0, S = 1.0;
  if (kept) {
    s_path[0] = 0;
    set_row(0);
    while (true) {
      const int child = next_child(cur, last);
      if (child < 0) break;
      last = child;
      const double u = s_u[child], x = s_p[child], y = s_q[child];
      bool accept;
      if (Q != nullptr) {
        const double r = x - c * y;
        accept = u * y * S < (r > 0.0 ? r : 0.0);
      } else {
        bool seen = false;
        for (int i = 0; i < rejected; ++i) seen |= s_out[i] == s_token[child];
        const double r = seen || !(x > 0.0) ? 0.0 : x;
        accept = u * S < r;
        if (!accept) {
          S -= r;
          // (an entry for each rejected token once: the sums subtract every entry)
          if (!seen) {
            __syncthreads();
            if (tid == 0) s_out[rejected] = s_token[child];
            ++rejected;
            __syncthreads();
          }
        }
      }
      if (accept) {
        cur = child;
        if (tid == 0) s_path[kept] = child;
        ++kept;
        c = 0.0, S = 1.0;
        swept = false;
        rejected = 0;
        set_row(cur);
      } else if (Q != nullptr && S > 0.0) {  // (S = 0: nothing is left at all, for any larger c)
        c += S;
        S = sweep(c);
        swept = true;
      }
    }
    if (!swept) S = sweep(c);
  }
  __syncthreads();
  // ---- outputs
  if (rank == 0) {
    for (int i = tid; i < p.n; i += kThreads) p.path[static_cast<long long>(b) * p.n + i] = i < kept ? s_path[i] : -1;
    if (tid == 0) {
      p.num_kept[b] = kept;
      if (kept == 0) p.next_token[b] = -1;
    }
  }
  if (kept) {
    if (S > 0.0) {
      const double goal = static_cast<double>(p.u_next[b]) * S;
      // the first block, warp, element whose running sum passes the goal (the
      // last one with any weight, should rounding leave the goal past it)
      int at = -1, some = 0;
      double before = 0.0, run = 0.0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < cs) {
          if (cta_sum[r] > 0.0 && at < 0) {
            some = r;
            before = run;
            if (run + cta_sum[r] > goal) at = r;
          }
          run += cta_sum[r];
        }
      if ((at < 0 ? some : at) == rank) {
        int wat = -1, wsome = 0;
        double wbefore = before;
        run = before;
        for (int w = 0; w < kWarps; ++w) {
          if (s_warp[w] > 0.0 && wat < 0) {
            wsome = w;
            wbefore = run;
            if (run + s_warp[w] > goal) wat = w;
          }
          run += s_warp[w];
        }
        if ((wat < 0 ? wsome : wat) == warp) {
          run = wbefore;
          int token = -1, fallback = -1;
          for (int g0 = run0; g0 < run1 && token < 0; g0 += 32) {
            const int g = g0 + lane;
            float fp[N], fq[N];
#pragma unroll
            for (int e = 0; e < N; ++e) fp[e] = fq[e] = 0.f;
            if (g < run1) {
              load_group(P, g, fp);
              if (Q != nullptr && c != 0.0) load_group(Q, g, fq);
            }
            double w[N], sum = 0.0;
            int mine = -1;  // this lane's last element with any weight
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const double r = static_cast<double>(fp[e]) - c * static_cast<double>(fq[e]);
              w[e] = r > 0.0 ? r : 0.0;
              for (int i = 0; i < rejected; ++i)
                if (s_out[i] == N * g - mis + e) w[e] = 0.0;
              sum += w[e];
              if (w[e] > 0.0) mine = N * g - mis + e;
            }
            double incl = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const double o = __shfl_up_sync(0xffffffffu, incl, d);
              if (lane >= d) incl += o;
            }
            const uint32_t pass = __ballot_sync(0xffffffffu, run + incl > goal && sum > 0.0);
            const uint32_t any = __ballot_sync(0xffffffffu, mine >= 0);
            if (any) fallback = __shfl_sync(0xffffffffu, mine, 31 - __clz(any));
            if (pass) {
              const int who = __ffs(static_cast<int>(pass)) - 1;
              double a = run + incl - sum;
              int hit = -1;
#pragma unroll
              for (int e = 0; e < N; ++e) {
                a += w[e];
                if (hit < 0 && w[e] > 0.0 && a > goal) hit = N * g - mis + e;
              }
              if (hit < 0) hit = mine;
              token = __shfl_sync(0xffffffffu, hit, who);
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
          }
          if (lane == 0) p.next_token[b] = token >= 0 ? token : fallback;
        }
      }
    } else {
      // nothing is left (p <= c q everywhere): the target's most probable token, the lowest of equals
      float top = -INFINITY;
      int at = 0x7fffffff;
      if (rank == 0) {
        for (int v = tid; v < V; v += kThreads) {
          const float f = to_f32(P[row + v]);
          if (f > top) top = f, at = v;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, top, d);
          const int oa = __shfl_xor_sync(0xffffffffu, at, d);
          if (o > top || (o == top && oa < at)) top = o, at = oa;
        }
        if (lane == 0) s_top[warp] = top, s_at[warp] = at;
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kWarps; ++w)
            if (s_top[w] > top || (s_top[w] == top && s_at[w] < at)) top = s_top[w], at = s_at[w];
          p.next_token[b] = at < V ? at : 0;
        }
      }
    }
  }
  if (cs > 1) cluster_sync_all();  // no block leaves while another reads its sum
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyParams& p, int sms, cudaStream_t stream) {
  // blocks per sequence: as many as fill the GPU (four 512-thread blocks an
  // SM), each with 4096 tokens of the vocabulary or more
  int cs = kMaxCluster;
  while (cs > 1 && (static_cast<long long>(p.batch) * cs > 4ll * sms || static_cast<long long>(cs) * 4096 > p.vocab))
    cs >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * cs);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.dtype == kDtypeBf16 ? cudaLaunchKernelEx(&cfg, verify_tree_kernel<__nv_bfloat16>, p)
                               : cudaLaunchKernelEx(&cfg, verify_tree_kernel<float>, p);
}

}  // namespace mqa
