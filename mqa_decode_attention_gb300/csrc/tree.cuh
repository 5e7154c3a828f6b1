// What the tree-attention kernels share: the division of the work among the
// blocks, the mask bits of a run of keys, and the merge of partial results.
//
// A unit is (sequence b, kv head j, row block rb): up to `rows` of kv head j's
// (node i, query head h = j G + hl) pairs, row = i G + hl, over every key
// tile of the sequence. The units' tiles in order (b, j, rb, tile) form one
// long line, which is cut into equal runs, one for each block: every block
// streams the same number of key tiles whatever the lengths, the tree sizes
// and the batch are. A block's run of one unit is a segment. A segment that
// holds a whole unit writes its output; otherwise it leaves an unnormalised
// partial result, and the block that arrives last at the unit's counter merges
// its partials in block order (the same sums whichever block that is).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"

namespace mqa {

// One sequence as the kernels see it. An invalid one (a negative position,
// more nodes than the call's, a length past the bound) has no work: nothing of
// it is read or written.
struct TreeSeq {
  int pos, nodes, len;  // cached tokens, nodes, both
  int lo;               // first key that any node can attend to
  int first;            // lo rounded down to a multiple of 64: key 0 of tile 0
  int tiles, blocks;    // key tiles; row blocks
  bool bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b, int tile, int rows) {
  TreeSeq s;
  s.pos = p.pos[b];
  s.nodes = p.num_nodes != nullptr ? p.num_nodes[b] : p.n;
  const long long limit = p.capacity < p.max_seq_len ? p.capacity : p.max_seq_len;
  s.bad = s.pos < 0 || s.nodes < 0 || s.nodes > p.n || static_cast<long long>(s.pos) + s.nodes > limit;
  if (s.bad) s.pos = s.nodes = 0;
  s.len = s.pos + s.nodes;
  // (a node's position is at least pos: the smallest depth is 0)
  s.lo = p.window > 0 ? max(0, s.pos + 1 - p.window) : 0;
  s.first = s.lo / 64 * 64;
  s.tiles = s.nodes > 0 ? (s.len - s.first + tile - 1) / tile : 0;
  s.blocks = (s.nodes * p.group + rows - 1) / rows;
  return s;
}

__device__ __forceinline__ long long tree_work(const TreeParams& p, const TreeSeq& s) {
  return static_cast<long long>(s.tiles) * s.blocks * p.h_kv;
}

// Block `cta`'s run of the line: tiles [run * cta, run * (cta + 1)), the run as
// short as the blocks allow, but p.min_tiles at least (merging more partials
// would cost more than the shorter runs save). Runs of one whole length fall on
// the units' ends more often than runs of total / blocks tiles, none longer: 2 x 8
// units of 32 tiles, 64 nodes, 54.7 -> 50.0 us.
struct TreePlan {
  long long total, begin, end, run;
  long long before;  // tiles of the sequences before b
  int b;             // the sequence holding `begin`
  TreeSeq s;         // that sequence
};

// By one whole warp; `out` in shared memory. Lane l sums the tiles of its
// share of the sequences (consecutive ones), a scan over the lanes finds the
// lane whose share holds `begin`, and that lane walks its share again.
__device__ __forceinline__ void tree_plan(const TreeParams& p, int tile, int rows, int cta, int grid, TreePlan* out) {
  const int lane = threadIdx.x & 31;
  const int per = (p.batch + 31) / 32, b0 = min(lane * per, p.batch), b1 = min(b0 + per, p.batch);
  long long sum = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const TreeSeq s = tree_seq(p, b, tile, rows);
    sum += tree_work(p, s);
    bad |= s.bad;
  }
  if (bad && cta == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_SEQ_LEN));
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  const long long total = __shfl_sync(0xffffffffu, incl, 31);
  const long long run = max((total + grid - 1) / grid, static_cast<long long>(p.min_tiles));
  const long long begin = min(total, run * cta), end = min(total, begin + run);
  const long long excl = incl - sum;
  if (lane == 0) {
    out->total = total;
    out->begin = begin;
    out->end = end;
    out->run = run;
  }
  if (begin < end && begin >= excl && begin < incl) {  // one lane: the shares are disjoint
    long long before = excl;
    int b = b0;
    while (b < b1 - 1) {
      const long long w = tree_work(p, tree_seq(p, b, tile, rows));
      if (begin < before + w) break;
      before += w;
      ++b;
    }
    out->before = before;
    out->b = b;
    out->s = tree_seq(p, b, tile, rows);
  }
  __syncwarp();
}

struct TreeSegment {
  int b, j, rb;     // the unit
  int t0, nt;       // first tile, tiles
  bool head, tail;  // holds the unit's first / last tile
  long long u0;     // the unit's first tile on the line
  TreeSeq s;
};

// A block's segments one after the other.
struct TreeWalk {
  long long at, end, before;
  int b;
  TreeSeq s;
  __device__ __forceinline__ void start(const TreePlan& pl) {
    at = pl.begin;
    end = pl.end;
    before = pl.before;
    b = pl.b;
    s = pl.s;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, int tile, int rows, TreeSegment& g) {
    if (at >= end) return false;
    while (true) {
      const long long w = tree_work(p, s);
      if (at < before + w) break;
      if (++b >= p.batch) return false;  // (never: at < end <= total)
      before += w;
      s = tree_seq(p, b, tile, rows);
    }
    const long long off = at - before;
    const int unit = static_cast<int>(off / s.tiles);
    g.b = b;
    g.t0 = static_cast<int>(off - static_cast<long long>(unit) * s.tiles);
    g.j = unit / s.blocks;
    g.rb = unit - g.j * s.blocks;
    g.nt = static_cast<int>(min(static_cast<long long>(s.tiles - g.t0), end - at));
    g.head = g.t0 == 0;
    g.tail = g.t0 + g.nt == s.tiles;
    g.u0 = at - g.t0;
    g.s = s;
    at += g.nt;
    return true;
  }
};

// The block whose run holds tile x of the line.
__device__ __forceinline__ int tree_cta_of(const TreePlan& pl, long long x) { return static_cast<int>(x / pl.run); }

// Four uint8 codes minus the zero point as two bf16 pairs, times 2^-6, exactly.
// A code in the low byte is the bf16 code * 2^-133 (subnormal below 128, normal
// from there on: the patterns go on evenly), so one fused multiply-add makes
// code * 2^-6 - zero point * 2^-6: an integer of 8 bits at most, times 2^-6. The
// 2^6 goes into the row's scale. z = u8_zero(zero point); two instructions for
// two codes (through fp32 and a conversion: four).
constexpr float kU8Unit = 64.f;
__device__ __forceinline__ uint32_t u8_zero(float zero_point) {
  return pack_bf16x2(zero_point * -(1.f / kU8Unit), zero_point * -(1.f / kU8Unit));
}
__device__ __forceinline__ uint2 widen_u8(uint32_t w, uint32_t z) {
  uint2 r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r.x) : "r"(__byte_perm(w, 0u, 0x4140)), "r"(0x7f007f00u), "r"(z));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r.y) : "r"(__byte_perm(w, 0u, 0x4342)), "r"(0x7f007f00u), "r"(z));
  return r;
}

// Two probabilities as two bf16 terms: the upper half of each value's bits, and
// what that leaves (below 2^-7 of the value), rounded: together within 2^-15.
__device__ __forceinline__ void split_p(float2 v, uint32_t& hi, uint32_t& lo) {
  const uint32_t x = __float_as_uint(v.x), y = __float_as_uint(v.y);
  hi = __byte_perm(x, y, 0x7632);
  lo = pack_bf16x2(v.x - __uint_as_float(x & 0xffff0000u), v.y - __uint_as_float(y & 0xffff0000u));
}

// 32 bits, bit c = the row may attend to key k0 + c. m: the row's mask words
// with the bits of dead nodes cleared (all zero for a dead row), ka its first
// key, pos the number of cached tokens.
struct TreeRow {
  uint32_t m[4];
  int ka, pos;
};

__device__ __forceinline__ uint32_t tree_bits(const TreeRow& r, int k0) {
  // cached tokens: keys [ka, pos)
  const int a = min(max(r.ka - k0, 0), 32), e = min(max(r.pos - k0, 0), 32);
  uint32_t v = 0;
  if (e > a) v = (e == 32 ? 0xffffffffu : (1u << e) - 1u) & (0xffffffffu << a);
  // nodes: bit t of the mask is key pos + t
  const int s = k0 - r.pos;  // node of bit 0
  if (s > -32 && s < 128) {
    const int w = s >> 5, o = s & 31;  // (arithmetic shift: w = -1 for s < 0)
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i == w) lo = r.m[i];
      if (i == w + 1) hi = r.m[i];
    }
    v |= __funnelshift_r(lo, hi, o);
  }
  return v;
}

// The first key that node i (-1: none) of sequence b may attend to.
__device__ __forceinline__ int tree_first_key(const TreeParams& p, int b, const TreeSeq& s, int i) {
  if (p.window <= 0 || i < 0) return 0;
  const long long ka = static_cast<long long>(s.pos) + max(p.depth[static_cast<long long>(b) * p.n + i], 0) + 1 - p.window;
  return ka > 0 ? static_cast<int>(min(ka, static_cast<long long>(s.pos))) : 0;
}

// Row r (node i, -1: none) of a unit of sequence b.
__device__ __forceinline__ TreeRow tree_row(const TreeParams& p, int b, const TreeSeq& s, int i) {
  TreeRow r;
  r.pos = s.pos;
  r.ka = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) r.m[w] = 0;
  if (i < 0) {
    r.pos = r.ka = 0;
    return r;
  }
  const uint32_t* m = p.mask + (static_cast<long long>(b) * p.n + i) * p.words;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    if (w < p.words) {
      r.m[w] = m[w];
      const int left = s.nodes - 32 * w;  // nodes past the sequence's own
      if (left < 32) r.m[w] &= left > 0 ? (1u << left) - 1u : 0u;
    }
  if (p.window > 0) {
    const int32_t* depth = p.depth + static_cast<long long>(b) * p.n;
    const long long ka = static_cast<long long>(s.pos) + max(depth[i], 0) + 1 - p.window;
    r.ka = tree_first_key(p, b, s, i);
    for (int t = 0; t < s.nodes; ++t) {
      const bool far = static_cast<long long>(s.pos) + max(depth[t], 0) < ka;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (far && (t >> 5) == w) r.m[w] &= ~(1u << (t & 31));
    }
  }
  return r;
}

// Four consecutive output values of one row.
__device__ __forceinline__ void tree_store4(const TreeParams& p, long long o, float a, float b, float c, float d) {
  if (p.out_dtype == kDtypeBf16) {
    uint2 w;
    w.x = pack_bf16x2(a, b);
    w.y = pack_bf16x2(c, d);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(a, b, c, d);
  }
}

__device__ __forceinline__ long long tree_out_row(const TreeParams& p, const TreeSegment& g, int row) {
  const int i = row / p.group;
  return (static_cast<long long>(g.b) * p.n + i) * p.h_q + g.j * p.group + (row - i * p.group);
}

// A unit's merge: its first block, its blocks, this block among them. Partial
// k of a unit lies in the places of its k-th block.
struct TreeMerge {
  int ca, m;
};
__device__ __forceinline__ TreeMerge tree_merge(const TreePlan& pl, const TreeSegment& g) {
  const int ca = tree_cta_of(pl, g.u0), cb = tree_cta_of(pl, g.u0 + g.s.tiles - 1);
  return {ca, cb - ca + 1};
}
// where block `cta` leaves its partial of segment g
__device__ __forceinline__ float* tree_place(const TreeParams& p, const TreeSegment& g, int cta, int rows, int d) {
  return p.part + tree_part_floats(rows, d) * (2 * static_cast<size_t>(cta) + (g.head ? 1 : 0));
}

// Merges a unit all of whose partials are in the workspace, seen by the
// calling threads (all `threads` of them, tid their index):
//   M = max_k m_k,  O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k
// with a running M, in block order whichever block merges. A warp takes 8 rows
// at a time, lane (row, quarter): a load instruction reads 4 runs of 128
// bytes, a store writes whole sectors of 8 rows, and a partial's 8 loads (d =
// 128) are in flight together.
template <int D>
__device__ __forceinline__ void tree_merge_rows(const TreeParams& p, const TreeMerge& mg, const TreeSegment& g,
                                                int rows_per_block, int tid, int threads) {
  constexpr int kU = D / 16;  // 16-byte pieces of a row per lane
  const int rows = min(rows_per_block, g.s.nodes * p.group - g.rb * rows_per_block);
  const int lane = tid & 31;
  for (int r0 = (tid >> 5) * 8; r0 < rows; r0 += threads / 32 * 8) {
    const int r = min(r0 + (lane & 7), rows - 1);
    float4 acc[kU];
    float mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int u = 0; u < kU; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k = 0; k < mg.m; ++k) {
      const float* q = p.part + tree_part_floats(rows_per_block, D) * (k == 0 ? 2 * mg.ca + 1 : 2 * (mg.ca + k));
      const float mk = __ldcg(q + static_cast<size_t>(rows_per_block) * D + r);
      const float lk = __ldcg(q + static_cast<size_t>(rows_per_block) * (D + 1) + r);
      float4 o[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        o[u] = __ldcg(reinterpret_cast<const float4*>(q) + static_cast<size_t>(4 * u + (lane >> 3)) * rows_per_block + r);
      if (lk != 0.f) {  // (else no key of this part. A NaN score: the sum is NaN, whatever the maximum)
        const float top = fmaxf(mx, mk), a = exp2f(mx - top), w = exp2f(mk - top);
        mx = top;
        l = fmaf(w, lk, a * l);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          acc[u].x = fmaf(w, o[u].x, a * acc[u].x);
          acc[u].y = fmaf(w, o[u].y, a * acc[u].y);
          acc[u].z = fmaf(w, o[u].z, a * acc[u].z);
          acc[u].w = fmaf(w, o[u].w, a * acc[u].w);
        }
      }
    }
    if (r0 + (lane & 7) < rows) {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const long long o = tree_out_row(p, g, g.rb * rows_per_block + r);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        tree_store4(p, o * D + 4 * (4 * u + (lane >> 3)), acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv);
      if (lane < 8 && p.lse_out != nullptr)
        p.lse_out[o] = l != 0.f ? (mx + log2f(l)) * 0.69314718055994530942f : -INFINITY;
    }
  }
}

// After a block has written its partial of segment g (all `threads` threads,
// `sync` a barrier over them): counts it in, true when it was the unit's last.
template <class Sync>
__device__ __forceinline__ bool tree_arrive(const TreeParams& p, const TreeMerge& mg, int tid, volatile int* flag,
                                            const Sync& sync) {
  sync();
  if (tid == 0) {
    __threadfence();  // the block's partial (seen through the barrier), before the count
    *flag = atomicAdd(p.arrived + mg.ca, 1) == mg.m - 1;
    __threadfence();  // the other blocks' partials, after it
  }
  sync();
  return *flag != 0;
}

}  // namespace mqa
