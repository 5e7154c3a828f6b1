// Verification of a tree of drafted tokens against the target's probabilities
// from given random numbers (speculative sampling over several candidates),
// "Arsitektur Inferensi LLM", section 7: the result follows the target's
// distribution if a node's children are independent draws from the draft's, or
// (no draft probabilities given) whatever they are.
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
// the sums carry 64-bit accuracy. The fp64 pipe of this part takes 16 cycles
// for one warp's addition (with fp64 across the threads a sweep of 128000
// tokens took 40 us), so weights and sums are unevaluated pairs of floats, the
// rounding errors of each product, difference and sum kept, down to one value
// per block; only the walk's own comparisons and the last element's search are
// fp64, by one warp. A weight p - c q is within 2^-46 of c q; a sum of n weights on
// one lane is off by n^2 2^-49 of itself at most and by about n 2^-51 as a rule (n
// = 63 for 128000 tokens on eight blocks). Rejected tokens of deterministic
// drafts are left out of the sums, not taken off them: what remains may weigh
// less than the rounding of what was rejected, or nothing at all.
//
// A cluster of up to 8 blocks serves one sequence: warp 0 of every block walks
// the tree alike; when it needs a sum over the vocabulary every warp of the
// cluster adds its share (consecutive slices for blocks, consecutive runs for
// warps), and the blocks' sums meet through distributed shared memory. The
// next token is found by the block, then the warp's run, then the eighth of it
// that holds the goal.
//
// Bound: latency at every size -- a row of 128000 fp32 probabilities is 0.08 us
// of the HBM rate. A sweep is two barriers, a memory round trip or two and a
// cluster barrier.
#include <cuda_bf16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"

namespace mqa {
namespace {

constexpr int kThreads = 256;
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
__global__ void __launch_bounds__(kThreads, 3) verify_tree_kernel(const VerifyParams p) {
  constexpr int N = Vec<T>::kN;
  __shared__ int s_parent[kMaxTreeNodes], s_token[kMaxTreeNodes], s_path[kMaxTreeNodes];
  __shared__ float s_u[kMaxTreeNodes], s_p[kMaxTreeNodes], s_q[kMaxTreeNodes];
  __shared__ int s_out[kMaxTreeNodes];  // deterministic drafts: tokens rejected at the current node
  __shared__ Pair s_part[kWarps];       // sums of the warps' runs
  __shared__ double s_sum[2];           // this block's sum, by the sweep's parity
  __shared__ struct {
    int what;       // 0 done, 1 a sweep, 2 the eighths of run `run`
    int node, run;  // the row
    int rejected;   // entries of s_out
    float ch, cl;   // the coefficient
  } s_cmd;
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

  // ---- the vocabulary in 16-byte groups of a row (aligned in memory: the
  // first and the last may be cut), shared out to blocks and warps in runs
  struct Row {
    long long off;  // element offset
    int mis, groups, per_cta, per_warp;
  };
  auto row_of = [&](int node) {
    Row r;
    r.off = (static_cast<long long>(b) * p.n + node) * p.row_stride;
    r.mis = static_cast<int>(r.off & (N - 1));
    r.groups = (V + r.mis + N - 1) / N;
    r.per_cta = (r.groups + cs - 1) / cs;
    r.per_warp = (r.per_cta + kWarps - 1) / kWarps;
    return r;
  };
  auto run_of = [&](const Row& r, int w, int* g0, int* g1) {  // warp w's run of this block's slice
    const int end = min(r.groups, (rank + 1) * r.per_cta);
    *g0 = min(end, rank * r.per_cta + w * r.per_warp);
    *g1 = min(end, *g0 + r.per_warp);
  };
  auto eighth_of = [&](int g0, int g1, int w, int* h0, int* h1) {  // part w of a run
    const int per = (g1 - g0 + kWarps - 1) / kWarps;
    *h0 = min(g1, g0 + w * per);
    *h1 = min(g1, *h0 + per);
  };
  auto load_group = [&](const Row& r, const T* src, int g, float (&f)[N]) {  // zeros outside the row
    const int v0 = N * g - r.mis;
    if (v0 >= 0 && v0 + N <= V) {
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(src + r.off + v0)), f);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = v0 + e >= 0 && v0 + e < V ? to_f32(src[r.off + v0 + e]) : 0.f;
    }
  };
  // the weight of groups [g0, g1) for the command's coefficient, on lane 0
  auto run_sum = [&](const Row& r, int g0, int g1) {
    const float ch = s_cmd.ch, cl = s_cmd.cl;
    const bool with_q = Q != nullptr && (ch != 0.f || cl != 0.f);
    Pair acc = {0.f, 0.f};
    constexpr int kU = 16 / N;
    // deterministic drafts: rejected tokens weigh nothing. The run goes in pieces
    // from one group that holds any to the next; of such a group lane e takes
    // element e, if it was not rejected.
    const int rejected = s_cmd.rejected;
    while (true) {
      int cut = 0x7fffffff;  // the next such group
      for (int i = lane; i < rejected; i += 32) {
        const int g = (s_out[i] + r.mis) / N;
        if (g >= g0) cut = min(cut, g);
      }
      cut = __reduce_min_sync(0xffffffffu, cut);
      const int end = min(cut, g1);
#pragma unroll 1
      for (int a = g0 + lane; a < end; a += 32 * kU) {
        float fp[kU][N], fq[kU][N];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int g = a + 32 * u;
#pragma unroll
          for (int e = 0; e < N; ++e) fp[u][e] = fq[u][e] = 0.f;
          if (g < end) {
            load_group(r, P, g, fp[u]);
            if (with_q) load_group(r, Q, g, fq[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const Pair w = residual(fp[u][e], fq[u][e], ch, cl);
            if (__fadd_rn(w.hi, w.lo) > 0.f) add(acc, w.hi, w.lo);  // (NaN: no weight)
          }
      }
      if (cut >= g1) break;
      const int v = N * cut - r.mis + lane;
      bool live = lane < N && v >= 0 && v < V;
      for (int i = 0; i < rejected; ++i) live &= s_out[i] != v;
      const float w = live ? to_f32(P[r.off + v]) : 0.f;
      if (w > 0.f) add(acc, w, 0.f);
      g0 = cut + 1;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      add(acc, __shfl_xor_sync(0xffffffffu, acc.hi, d), __shfl_xor_sync(0xffffffffu, acc.lo, d));
    return acc;
  };
  // a command's share of this warp, and what follows for all warps
  auto serve = [&]() {
    const Row r = row_of(s_cmd.node);
    int g0, g1;
    if (s_cmd.what == 1) {
      run_of(r, warp, &g0, &g1);
    } else {
      int r0, r1;
      run_of(r, s_cmd.run, &r0, &r1);
      eighth_of(r0, r1, warp, &g0, &g1);
    }
    const Pair s = run_sum(r, g0, g1);
    if (lane == 0) s_part[warp] = s;
    __syncthreads();
  };

  if (warp != 0) {
    while (true) {
      __syncthreads();  // the command
      const int what = s_cmd.what;
      if (what == 0) break;
      serve();
      if (what == 1 && cs > 1) cluster_sync_all();
    }
  } else {
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
    auto command = [&](int what, int node, int run, int rejected, double c) {
      __syncwarp();
      if (lane == 0) {
        const float ch = static_cast<float>(c);
        s_cmd.what = what;
        s_cmd.node = node;
        s_cmd.run = run;
        s_cmd.rejected = rejected;
        s_cmd.ch = ch;
        s_cmd.cl = static_cast<float>(c - static_cast<double>(ch));
      }
      __syncthreads();
      if (what != 0) serve();
    };
    // lane i: the sum of part i (a run, or an eighth of one) as a double
    auto parts = [&]() {
      return lane < kWarps ? static_cast<double>(s_part[lane].hi) + static_cast<double>(s_part[lane].lo) : 0.0;
    };
    // inclusive running sum over the lanes, in lane order
    auto running = [&](double x) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
      }
      return x;
    };
    // the first lane with any weight whose running sum passes the goal (else
    // the last with any weight, should rounding leave the goal past it)
    auto pick = [&](double x, double incl, double goal) {
      const uint32_t some = __ballot_sync(0xffffffffu, x > 0.0), pass = __ballot_sync(0xffffffffu, x > 0.0 && incl > goal);
      return pass ? __ffs(static_cast<int>(pass)) - 1 : 31 - __clz(some);
    };
    int parity = 0;
    double block = 0.0;  // lane r: block r's sum
    auto sweep = [&](int node, int rejected, double c) {
      command(1, node, 0, rejected, c);
      const double mine = __shfl_sync(0xffffffffu, running(parts()), 31);
      if (cs > 1) {
        if (lane == 0) s_sum[parity] = mine;
        cluster_sync_all();
        block = lane < cs ? dsmem_ld_f64(dsmem_map(smem_u32(&s_sum[parity]), lane)) : 0.0;
        parity ^= 1;
      } else {
        block = lane == 0 ? mine : 0.0;
      }
      return __shfl_sync(0xffffffffu, running(block), 31);
    };

    // ---- the walk
    int cur = 0, last = 0, kept = nodes > 0 ? 1 : 0, rejected = 0;
    bool swept = false;  // the sums of (cur, c) are there
    double c = 0.0, S = 1.0;
    if (kept) {
      if (lane == 0) s_path[0] = 0;
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
            // (an entry for each rejected token once)
            if (!seen) {
              if (lane == 0) s_out[rejected] = s_token[child];
              ++rejected;
              __syncwarp();
            }
          }
        }
        if (accept) {
          cur = child;
          if (lane == 0) s_path[kept] = child;
          ++kept;
          c = 0.0, S = 1.0;
          swept = false;
          rejected = 0;
        } else if (Q != nullptr && S > 0.0) {  // (S = 0: nothing is left at all, for any larger c)
          c += S;
          S = sweep(cur, 0, c);
          swept = true;
        }
      }
      if (!swept) S = sweep(cur, rejected, c);
    }
    __syncwarp();
    // ---- outputs
    if (rank == 0) {
      for (int i = lane; i < p.n; i += 32) p.path[static_cast<long long>(b) * p.n + i] = i < kept ? s_path[i] : -1;
      if (lane == 0) {
        p.num_kept[b] = kept;
        if (kept == 0) p.next_token[b] = -1;
      }
    }
    if (kept && S > 0.0) {
      const double goal = static_cast<double>(p.u_next[b]) * S;
      const double upto = running(block);
      const int at = pick(block, upto, goal);
      if (at == rank) {
        double before = __shfl_sync(0xffffffffu, upto - block, at);
        const Row r = row_of(cur);
        double x = parts(), incl = running(x);
        const int run = pick(x, before + incl, goal);
        before += __shfl_sync(0xffffffffu, incl - x, run);
        command(2, cur, run, rejected, c);
        x = parts();
        incl = running(x);
        const int part = pick(x, before + incl, goal);
        before += __shfl_sync(0xffffffffu, incl - x, part);
        int r0, r1, h0, h1;
        run_of(r, run, &r0, &r1);
        eighth_of(r0, r1, part, &h0, &h1);
        int token = -1, fallback = 0;
        for (int a = h0; a < h1 && token < 0; a += 32) {
          const int g = a + lane;
          float fp[N], fq[N];
#pragma unroll
          for (int e = 0; e < N; ++e) fp[e] = fq[e] = 0.f;
          if (g < h1) {
            load_group(r, P, g, fp);
            if (Q != nullptr && c != 0.0) load_group(r, Q, g, fq);
          }
          double w[N], sum = 0.0;
          int mine = -1;  // this lane's last element with any weight
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const Pair d = residual(fp[e], fq[e], s_cmd.ch, s_cmd.cl);  // (as in the sums that led here)
            w[e] = __fadd_rn(d.hi, d.lo) > 0.f ? static_cast<double>(d.hi) + static_cast<double>(d.lo) : 0.0;
            for (int i = 0; i < rejected; ++i)
              if (s_out[i] == N * g - r.mis + e) w[e] = 0.0;
            sum += w[e];
            if (w[e] > 0.0) mine = N * g - r.mis + e;
          }
          const double in = running(sum);
          const uint32_t pass = __ballot_sync(0xffffffffu, sum > 0.0 && before + in > goal);
          const uint32_t any = __ballot_sync(0xffffffffu, mine >= 0);
          if (any) fallback = __shfl_sync(0xffffffffu, mine, 31 - __clz(any));
          if (pass) {
            double acc = before + in - sum;
            int hit = -1;
#pragma unroll
            for (int e = 0; e < N; ++e) {
              acc += w[e];
              if (hit < 0 && w[e] > 0.0 && acc > goal) hit = N * g - r.mis + e;
            }
            token = __shfl_sync(0xffffffffu, hit < 0 ? mine : hit, __ffs(static_cast<int>(pass)) - 1);
          }
          before += __shfl_sync(0xffffffffu, in, 31);
        }
        if (lane == 0) p.next_token[b] = token >= 0 ? token : fallback;
      }
    } else if (kept && rank == 0) {
      // nothing is left (p <= c q everywhere): the target's most probable token, the lowest of equals
      const Row r = row_of(cur);
      float top = -INFINITY;
      int at = 0x7fffffff;
      for (int v = lane; v < V; v += 32) {
        const float f = to_f32(P[r.off + v]);
        if (f > top) top = f, at = v;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, top, d);
        const int oa = __shfl_xor_sync(0xffffffffu, at, d);
        if (o > top || (o == top && oa < at)) top = o, at = oa;
      }
      if (lane == 0) p.next_token[b] = at < V ? at : 0;
    }
    command(0, 0, 0, 0, 0.0);
  }
  if (cs > 1) cluster_sync_all();  // no block leaves while another reads its sum
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyParams& p, int sms, cudaStream_t stream) {
  // blocks per sequence: as many as fill the GPU once (three blocks an SM),
  // each with 2048 tokens of the vocabulary or more
  int cs = kMaxCluster;
  while (cs > 1 && (static_cast<long long>(p.batch) * cs > 3ll * sms || static_cast<long long>(cs) * 2048 > p.vocab))
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
