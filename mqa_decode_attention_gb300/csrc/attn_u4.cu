// Attention over a 4-bit cache (rows of codes c and one bf16 pair (s, m), the
// value m + s c: u4.cuh), one to 32 new tokens per sequence.
//
// With K = m + s c and V alike, the scaling stays outside the products:
//   q . K_t = s_t (q . c_t) + m_t sum(q)
//   O       = sum_t (p_t s_t) c_t + sum_t p_t m_t,
// so the tensor cores multiply codes as they are. A code in bits 0-3 of a half
// is the fp16 number c 2^-24, in bits 4-7 16 c 2^-24 (subnormal and small
// normal numbers, exact): one AND for two codes makes an operand, a shift for
// every second one. The 16 is taken out of q (K) and of the output (V), the
// 2^-24 out of the scores' factor and of the output.
//
// q enters as fp16 (11 bits), each row scaled by a power of two to a largest
// value in [2^13, 2^14); sum(q) is that of the rounded values, since s c and m
// cancel in part. p s enters as fp16 too: with E the power of two above the
// largest s a warp has met (a running exponent, as the softmax's running maximum)
// p s 2^(11 - E) has its 11 bits down to 2^-25 of the largest. Scores, maxima, sums and O are
// fp32. A maximum is only followed when a score passes it by more than 4 (in
// log2), so p <= 16.
//
// A warp takes 8 NT query rows of one kv head and tiles of 32 tokens: S^T = K Q^T
// (m16n8k16, tokens on the rows), softmax over the lanes that hold a column,
// P^T transposed in registers (movmatrix), O^T += V^T P^T (dims on the rows, so
// O's columns are S's). Codes stream through a ring of stages of its own, filled
// with bulk copies by the warp itself: four warps of a block share a run of
// tiles and meet at the end of a unit only (unit: sequence, kv head, block of
// query rows).
//
// The tiles of all units in order are cut into equal runs, one for each block
// (as many as are resident at once), so lengths of any spread load all SMs
// alike. A unit that several blocks share is merged by the last of them to
// arrive, in the order of the blocks, so that equal calls give equal bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "u4.cuh"

namespace mqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBoost = 11;      // p s 2^(kBoost - E), p <= 2^kSlack
constexpr float kSlack = 4.f;
constexpr uint32_t kFull = 0xffffffffu;

template <int D, int NT, int STAGES>
struct Cfg {
  static constexpr int kMt = NT == 1 ? 4 : 2;      // tiles of 16 tokens whose scores are held at a time
  static constexpr int kCode = D / 2;              // bytes of a row's codes
  static constexpr int kTileCodes = kU4Tile * kCode;
  static constexpr int kStage = 2 * kTileCodes;    // V codes (swizzled), K codes
  static constexpr int kPairs = 2 * 4 * kU4Tile;   // K pairs, V pairs
  static constexpr int kRows = 8 * NT;
  static constexpr int kM = D / 16;   // 16-row tiles of O^T; also the k16 steps of q . c
  static constexpr int kPairRing = kWarps * STAGES * kStage;
  static constexpr bool kQreg = NT <= 2;  // q as operands: in registers, else [k16 step][pair of n tiles][lane][2] in shared memory
  static constexpr int kQ = kPairRing + kWarps * STAGES * kPairs;
  static constexpr int kQsum = kQ + (kQreg ? 0 : kM * NT * 32 * 8);     // [rows] (sum of q, factor)
  // parts of a unit that warps leave: O in a stage of their own ring (NT <= 2), else in one place; maxima and sums
  static constexpr int kPart = kM * NT * 32 * 16, kPartMl = 2 * NT * 32 * 8;
  static constexpr int kMerge = kQsum + (kQreg ? 0 : kRows * 8);
  static constexpr int kMl = kMerge + (kQreg ? 0 : kPart);
  static constexpr int kBar = kMl + (kQreg ? kWarps : 1) * kPartMl;     // [warps][stages], then left [warps] and taken [warps]
  static constexpr int kFlag = kBar + kWarps * (STAGES + 2) * 8;
  static_assert(!kQreg || kPart <= kStage, "a part fits a stage");
  static constexpr int kSmem = kFlag + 56 + (2 + kWarps) * 4 * kWarps;
};

// d += A B, d the pairs of columns of rows r and r + 8
__device__ __forceinline__ void mma_f16(float2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// an 8 x 8 matrix of 16-bit values across the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four codes in each half of x: codes 0 and 2 alone, and with the code after them
// times 16 (a byte of a half is the fp16 number byte 2^-24, as a code is).
__device__ __forceinline__ void split_codes(uint32_t x, uint32_t& c0, uint32_t& b0, uint32_t& c2, uint32_t& b2) {
  b0 = x & 0x00ff00ffu;
  c0 = x & 0x000f000fu;
  b2 = __byte_perm(x, 0, 0x4341);
  c2 = b2 & 0x000f000fu;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // normal e

// the tiles that a sequence's units have: those with a token some row sees
struct Span {
  int len, lo, first, tiles;  // length, first token a row sees, first tile, tiles (0: the length is out of range)
};
__device__ __forceinline__ Span span_of(const U4Params& p, int len) {
  Span s;
  s.len = len;
  const bool ok = len >= p.n_new && len <= p.max_seq_len;
  s.lo = p.window > 0 ? max(0, len - p.n_new + 1 - p.window) : 0;
  s.first = s.lo / kU4Tile;
  s.tiles = ok ? (len + kU4Tile - 1) / kU4Tile - s.first : 0;
  return s;
}

// A place in the order of all tiles, relative to a block's run: tile k of the
// run is tile k - base of unit u of sequence b, for k in [base, base + tiles).
struct Place {
  int b, u, base;
  Span s;
  __device__ __forceinline__ int end() const { return base + s.tiles; }
  __device__ __forceinline__ void next(const U4Params& p, int units) {  // (there is a next unit)
    base += s.tiles;
    if (++u < units) return;
    u = 0;
    do {
      ++b;
      s = span_of(p, p.seq_lens[b]);
    } while (s.tiles == 0 && b + 1 < p.batch);
  }
};

// A count in shared memory that one warp raises (after what it says) and another waits for; false once `limit_ns` has passed.
__device__ __forceinline__ void publish(uint32_t at, uint32_t count) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(at), "r"(count) : "memory");
}
__device__ __forceinline__ bool reached(uint32_t at, uint32_t count) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return static_cast<int>(v - count) >= 0;
}
__device__ __forceinline__ bool wait_count(uint32_t at, uint32_t count, unsigned long long limit_ns) {
  if (reached(at, count)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!reached(at, count))
    if (global_timer_ns() - t0 > limit_ns) return false;
  return true;
}

// Two parts of a softmax: top becomes the larger maximum, wa and wb what their sums are worth then.
__device__ __forceinline__ void weights(float2& top, float2 m2, float2& wa, float2& wb) {
  const float2 now = make_float2(fmaxf(top.x, m2.x), fmaxf(top.y, m2.y));
  wa = make_float2(top.x == -INFINITY ? 0.f : fast_exp2(top.x - now.x), top.y == -INFINITY ? 0.f : fast_exp2(top.y - now.y));
  wb = make_float2(m2.x == -INFINITY ? 0.f : fast_exp2(m2.x - now.x), m2.y == -INFINITY ? 0.f : fast_exp2(m2.y - now.y));
  top = now;
}

// A warp's columns of 16-row tiles i0 .. i0 + N of O^T, divided by their sums, as the rows they are of the output. A lane
// has dims 4 r + (0 .. 3) of each 32, two tiles' worth.
template <int NT, int N>
__device__ __forceinline__ void write_rows(const U4Params& p, int b, int j, int row0, const float2 (&top)[NT], const float2 (&sum)[NT],
                                           const float2 (&o)[NT][N][2], int i0) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, D = p.head_dim;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ridx = row0 + 8 * n + 2 * c + e;
      if (ridx >= p.rows) continue;
      const int tok = ridx / p.group;
      const long long orow = (static_cast<long long>(b) * p.n_new + tok) * p.h_q + j * p.group + ridx - tok * p.group;
      const float total = e ? sum[n].y : sum[n].x, inv = 1.f / total;
#pragma unroll
      for (int i = 0; i < N; ++i) {  // dims 32 (i / 2) + 4 r + 2 (i % 2)
        const float y0 = (e ? o[n][i][0].y : o[n][i][0].x) * inv, y1 = (e ? o[n][i][1].y : o[n][i][1].x) * inv;
        const long long dst = orow * D + 32 * ((i0 + i) / 2) + 4 * r + 2 * ((i0 + i) & 1);
        if (p.out_dtype == kDtypeBf16)
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + dst) = pack_bf16x2(y0, y1);
        else
          *reinterpret_cast<float2*>(static_cast<float*>(p.out) + dst) = make_float2(y0, y1);
      }
      if (p.lse_out != nullptr && r == 0 && i0 == 0) p.lse_out[orow] = ((e ? top[n].y : top[n].x) + log2f(total)) * 0.6931471805599453f;
    }
}

template <int D, int NT, bool PAGED, int STAGES, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) attn_u4_kernel(const __grid_constant__ CUtensorMap tmap_v, const U4Params p) {
  using C = Cfg<D, NT, STAGES>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int units = p.h_kv * p.row_blocks;
  const uint32_t ring = smem_u32(smem) + warp * STAGES * C::kStage;
  const uint32_t pair_ring = smem_u32(smem) + C::kPairRing + warp * STAGES * C::kPairs;
  const uint32_t bars = smem_u32(smem) + C::kBar + warp * STAGES * 8;
  const uint32_t left = smem_u32(smem) + C::kBar + kWarps * STAGES * 8;  // [w]: warp w has left its part of a unit
  const uint32_t taken = left + 8 * kWarps;                              // [w]: it has been taken
  volatile int* where = reinterpret_cast<volatile int*>(smem + C::kFlag) + 10;  // [w]: the stage that holds it
  // NT <= 2: counts of the parts left and taken instead of barriers: a warp may be any number of units ahead of another's
  // part, which the parity of a barrier's phase could not tell apart.
  const uint32_t left_count = smem_u32(smem) + C::kFlag + 56, taken_count = left_count + 4 * kWarps;
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::kFlag);  // units to merge at the end, [2]: flag, sequence, unit, base, end

  if (lane == 0) {
    if (warp == 0) prefetch_tensormap(&tmap_v);
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1);
    mbar_init(left + 8 * warp, 1);
    mbar_init(taken + 8 * warp, 1);
    publish(left_count + 4 * warp, 0);
    publish(taken_count + 4 * warp, 0);
    for (int w = 0; w < kWarps; ++w) publish(taken_count + 4 * kWarps * (1 + warp) + 4 * w, 0);
    fence_mbar_init();
    if (warp < 2) flag[5 * warp] = 0;
  }
  __syncthreads();

  // ------------------------------------------------------ this block's run
  Place at;
  int run;             // tiles of the run
  long long start = 0, run_len = 1;  // place of the run among all tiles, length of the runs
  if (p.whole) {
    at.b = blockIdx.x / units;
    at.u = blockIdx.x - at.b * units;
    at.base = 0;
    at.s = span_of(p, p.seq_lens[at.b]);
    run = at.s.tiles;
    if (run == 0 && at.u == 0 && threadIdx.x == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_SEQ_LEN));
  } else {
    // (every warp finds it for itself; 32 sequences at a time, the first 32 kept)
    auto tiles_of = [&](int b) { return b < p.batch ? span_of(p, p.seq_lens[b]).tiles : 0; };
    const int mine = tiles_of(lane);
    bool bad = lane < p.batch && mine == 0;
    unsigned long long total = __reduce_add_sync(kFull, static_cast<unsigned>(mine));
    for (int b0 = 32; b0 < p.batch; b0 += 32) {
      const int t = tiles_of(b0 + lane);
      bad |= b0 + lane < p.batch && t == 0;
      total += __reduce_add_sync(kFull, static_cast<unsigned>(t));
    }
    if (blockIdx.x == 0 && warp == 0 && __any_sync(kFull, bad) && lane == 0)
      atomicOr(p.err, static_cast<int>(MQA_DEVERR_SEQ_LEN));
    total *= units;
    run_len = total < 1ull << 31 ? static_cast<unsigned>(total + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
    run_len = max(run_len, static_cast<long long>(p.min_tiles));
    start = run_len * blockIdx.x;
    run = static_cast<int>(max(0ll, min(run_len, static_cast<long long>(total) - start)));
    long long seen = 0;  // tiles of the sequences before (of one unit each)
    at.b = at.u = at.base = 0;
    at.s = {0, 0, 0, 1};
    for (int b0 = 0; run > 0 && b0 < p.batch; b0 += 32) {
      const int t = b0 == 0 ? mine : tiles_of(b0 + lane);
      unsigned upto = t;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned v = __shfl_up_sync(kFull, upto, off);
        if (lane >= off) upto += v;
      }
      const uint32_t past = __ballot_sync(kFull, (seen + upto) * units > start);
      if (past) {
        const int l = __ffs(past) - 1;
        at.b = b0 + l;
        at.s = span_of(p, p.seq_lens[at.b]);
        const long long off = start - (seen + __shfl_sync(kFull, upto, l) - at.s.tiles) * units;
        at.u = off < 1ll << 31 ? static_cast<unsigned>(off) / at.s.tiles : static_cast<int>(off / at.s.tiles);
        at.base = -static_cast<int>(off - static_cast<long long>(at.u) * at.s.tiles);
        break;
      }
      seen += __shfl_sync(kFull, upto, 31);
    }
  }
  if (run <= 0) return;  // the whole block

  // --------------------------------------------------- filling the ring
  // Lanes 0-3 copy the V codes (a tensor map, so that they land swizzled), the K
  // codes, the K pairs and the V pairs of a tile; with pages shorter than a tile
  // lanes 4-7, .. those of its further pages.
  Place fill = at;
  int fill_k = warp, fill_stage = 0, issued = 0;
  const int kind = lane & 3;
  const int size = kind < 2 ? C::kCode : 4;  // bytes of a row
  const int piece = PAGED ? min(p.page_size, kU4Tile) : kU4Tile;  // tokens of a copy
  const int at_row = (lane >> 2) * piece;                         // the copy's first token in the tile
  const bool copies = at_row < kU4Tile;
  const unsigned char* from = kind == 1   ? p.k_cache
                              : kind == 2 ? reinterpret_cast<const unsigned char*>(p.k_sm)
                                          : reinterpret_cast<const unsigned char*>(p.v_sm);
  const uint32_t to = kind < 2 ? ring + (kind == 1 ? C::kTileCodes : 0) + at_row * C::kCode
                               : pair_ring + (kind - 2) * 4 * kU4Tile + at_row * 4;
  const int ring_step = kind < 2 ? C::kStage : C::kPairs;
  int head = 0, fill_t = 0, page = 0;  // first token of the next tile; page of this lane's copy
  const unsigned char* unit_rows = from;  // contiguous: token 0's row of the unit
  uint32_t fill_bar = bars, fill_to = to;
  auto unit_changed = [&]() {
    head = fill.u / p.row_blocks;
    if (!PAGED) {
      head += fill.b * p.h_kv;
      unit_rows = from + static_cast<long long>(head) * p.capacity * size;
    }
  };
  auto look = [&]() {  // tile fill_k's place, and its page (looked up one fill ahead)
    if (fill_k >= run) return;
    if (fill_k >= fill.end()) {
      do fill.next(p, units);
      while (fill_k >= fill.end());
      unit_changed();
    }
    fill_t = (fill.s.first + fill_k - fill.base) * kU4Tile;
    if (PAGED) {
      const int t = fill_t + at_row;
      page = -1;
      if (copies && t < fill.s.len && t + piece > fill.s.lo)
        page = p.block_table[static_cast<long long>(fill.b) * p.max_pages + t / p.page_size];
    }
  };
  unit_changed();
  look();
  // row r of n tile n of a unit's query rows, quarter c of its dims
  auto load_q = [&](const Place& u, int n, float (&q)[D / 4]) {
    const int j = u.u / p.row_blocks, ridx = (u.u - j * p.row_blocks) * C::kRows + 8 * n + r, tok = ridx / p.group;
    if (ridx < p.rows) {
      const float4* src = reinterpret_cast<const float4*>(
          p.q_rot + ((static_cast<long long>(u.b) * p.n_new + tok) * p.h_q + j * p.group + ridx - tok * p.group) * D + c * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float4 v = src[i];
        q[4 * i] = v.x, q[4 * i + 1] = v.y, q[4 * i + 2] = v.z, q[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) q[i] = 0.f;
    }
  };
  // The rows of the unit after, into the L2 cache: a load from memory would wait behind the tiles under way.
  auto prefetch_q = [&](Place u) {
    if (warp != kWarps - 1 || u.end() >= run) return;
    u.next(p, units);
    const int j = u.u / p.row_blocks;
#pragma unroll
    for (int i = lane; i < C::kRows * (D / 32); i += 32) {
      const int ridx = (u.u - j * p.row_blocks) * C::kRows + i / (D / 32), tok = ridx / p.group;
      if (ridx < p.rows)
        prefetch_l2(p.q_rot + ((static_cast<long long>(u.b) * p.n_new + tok) * p.h_q + j * p.group + ridx - tok * p.group) * D + i % (D / 32) * 32);
    }
  };
  // The first unit's q is asked for before the first tiles: behind them it would wait until they have all come (31 MB
  // from all blocks, 5 us). When the append launch still forms it, one tile goes ahead.
  float q[C::kQreg ? NT : 1][D / 4];
  if (!p.early) {
#pragma unroll
    for (int n = 0; n < (C::kQreg ? NT : 1); ++n) load_q(at, C::kQreg ? n : warp, q[n]);
    prefetch_q(at);
  }
  auto fill_next = [&]() {  // fill_k < run
    if (PAGED) {
      const int t = fill_t + at_row;
      const bool want = copies && t < fill.s.len && t + piece > fill.s.lo;
      const bool copy = want && page >= 0 && page < p.num_pages;
      if (want && !copy && kind == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_PAGE_RANGE));
      const int parts = __popc(__ballot_sync(kFull, copy)) / 4;
      if (lane == 0) mbar_arrive_expect_tx(fill_bar, parts * piece * (2 * C::kCode + 8));
      __syncwarp();
      if (copy) {
        const int in_page = t & (p.page_size - 1);
        if (kind == 0)
          tma_load_4d(fill_to, &tmap_v, 0, in_page, head, page, fill_bar);
        else
          bulk_g2s(fill_to, from + ((static_cast<long long>(page) * p.h_kv + head) * p.page_size + in_page) * size, piece * size, fill_bar);
      }
    } else {
      // (the capacity is a multiple of 4 rows: copies of 16 bytes; the tensor map's are whole tiles)
      const int n = min(kU4Tile, (fill.s.len - fill_t + 3) & ~3);
      if (lane == 0) {
        mbar_arrive_expect_tx(fill_bar, kU4Tile * C::kCode + n * (C::kCode + 8));
        tma_load_3d(fill_to, &tmap_v, 0, fill_t, head, fill_bar);
      }
      __syncwarp();
      if (lane - 1u < 3u) bulk_g2s(fill_to, unit_rows + static_cast<long long>(fill_t) * size, n * size, fill_bar);
    }
    ++issued;
    fill_to += ring_step;
    fill_bar += 8;
    if (++fill_stage == STAGES) fill_stage = 0, fill_bar = bars, fill_to = to;
    fill_k += kWarps;
    look();
  };
  // before the append has ended only a tile without new rows
  if (fill_k < run && (!p.early || fill_t + kU4Tile <= fill.s.len - p.n_new)) fill_next();
  grid_dependency_wait();
  if (p.early) {
#pragma unroll
    for (int n = 0; n < (C::kQreg ? NT : 1); ++n) load_q(at, C::kQreg ? n : warp, q[n]);
    prefetch_q(at);
  }
  while (issued < STAGES && fill_k < run) fill_next();

  // ------------------------------------------------------------ the run
  // Columns 2 c, 2 c + 1 of each n tile as pairs. o: rows r (the even dims) and
  // r + 8 (even + 16 odd, until the unit ends). base_sum: sum p (m + 8 s).
  float2 o[NT][C::kM][2];
  // ref: minus the reference of a column's exponents, 0 at first; over: what a score may pass it by before it is followed
  // (-inf before the first score).
  float2 ref[NT], over[NT], sum[NT], base_sum[NT];
  // Sum of the operands p s, by the tensor cores: 8 times it is taken from o every few tiles, which makes the codes -8 to 7.
  // (Else o grows with the number of tokens while its sum with base_sum does not, and the rounding of the accumulators shows.)
  float2 csum[NT][2];
  int consumed = 0, stage = 0, k = warp;
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out
  // [w]: parts that warp w has left, as far as this warp has come
  volatile uint32_t* parts = reinterpret_cast<volatile uint32_t*>(smem + C::kFlag + 56 + 2 * 4 * kWarps) + kWarps * warp;
  bool owed = false;        // a stage holds this warp's part, or will, and could not be filled
  uint32_t own_parts = 0;   // parts that this warp has left
  bool part_out = false;    // this warp has left a part and not heard that it was taken
  auto fill_owed = [&]() {  // (the part was written and read by threads, the tile comes by the async proxy)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    owed = part_out = false;
    fill_next();
  };
  // ldmatrix rows of V: matrices (tokens 0-7, 8-15) x two 16-byte chunks of the rows
  uint32_t v_row[D / 64];
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    const int tok = (lane & 7) + (lane & 8), chunk = 2 * q + (lane >> 4);
    v_row[q] = ring + tok * C::kCode + ((chunk ^ (D == 128 ? (lane & 7) >> 1 : (lane & 7) >> 2)) << 4);
  }
  const float2 zero2 = make_float2(0.f, 0.f);
  auto centre = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 even = mul2(csum[n][0], make_float2(-8.f * 0x1p-24f, -8.f * 0x1p-24f));
      const float2 both = mul2(csum[n][0], make_float2(-136.f * 0x1p-24f, -136.f * 0x1p-24f));
#pragma unroll
      for (int i = 0; i < C::kM; ++i) {
        o[n][i][0] = add2(o[n][i][0], even);
        o[n][i][1] = add2(o[n][i][1], both);
      }
      csum[n][0] = csum[n][1] = zero2;
    }
  };

  for (uint32_t seg = 0;; ++seg) {
    const int k1 = min(run, at.end());
    const int j = at.u / p.row_blocks, row0 = (at.u - j * p.row_blocks) * C::kRows;
    const int len = at.s.len;
    // ---- q as operands: lane (r, c) forms those of row r, quarter c of the dims, of an n tile. Even dims meet single
    // codes, odd dims code pairs (even + 16 odd): x = q_odd / 16 and q_even - x, each rounded.
    uint32_t qf[C::kQreg ? NT : 1][C::kM][2];
    float2 qs[NT];  // sum(q), and
    float f[NT];    // the factor of the scores, times which qs is
    auto operands = [&](const float (&q)[D / 4], uint32_t (&h)[C::kM][2], float& total, float& factor) {
      uint32_t most = 0;  // bits of the largest finite magnitude
#pragma unroll
      for (int i = 0; i < D / 4; ++i) {
        const uint32_t m = __float_as_uint(q[i]) & 0x7fffffffu;
        most = max(most, m < 0x7f800000u ? m : 0u);
      }
      most = __reduce_max_sync(kFull, most);  // (one factor for the 8 rows)
      const int e = min(max(static_cast<int>(most >> 23) - 127, -80), 127);  // 2^e <= largest < 2^(e + 1)
      // (two factors: their product may leave the range)
      const float up0 = pow2((13 - e) / 2), up1 = pow2((13 - e) - (13 - e) / 2);
      const float sign = p.scale > 0.f ? 1.f : p.scale < 0.f ? -1.f : 0.f;
      total = 0.f;
#pragma unroll
      for (int ks = 0; ks < C::kM; ++ks) {
        const int d = ks / 2 * 8 + (ks & 1) * 2;  // dims d, d + 1 and d + 4, d + 5
        __half2 x, y;
        x.x = __float2half_rn(q[d + 1] * sign * up0 * up1 * 0.0625f);
        x.y = __float2half_rn(q[d + 5] * sign * up0 * up1 * 0.0625f);
        const float2 xf = __half22float2(x);
        y.x = __float2half_rn(q[d] * sign * up0 * up1 - xf.x);
        y.y = __float2half_rn(q[d + 4] * sign * up0 * up1 - xf.y);
        const float2 yf = __half22float2(y);
        total += yf.x + yf.y + 17.f * (xf.x + xf.y);
        h[ks][0] = *reinterpret_cast<const uint32_t*>(&y);
        h[ks][1] = *reinterpret_cast<const uint32_t*>(&x);
      }
      total += __shfl_xor_sync(kFull, total, 1);
      total += __shfl_xor_sync(kFull, total, 2);
      factor = fabsf(p.scale) * 1.4426950408889634f * 0x1p24f / up0 / up1;
      total *= 0x1p-24f * factor;
    };
    if constexpr (C::kQreg) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float total, factor;
        operands(q[n], qf[n], total, factor);
        qs[n] = make_float2(__shfl_sync(kFull, total, 8 * c), __shfl_sync(kFull, total, 8 * c + 4));
        f[n] = factor;
      }
    } else {
      static_assert(C::kQreg || NT == kWarps, "each warp forms the operands of one n tile");
      float total, factor;
      operands(q[0], qf[0], total, factor);
      __syncthreads();  // the unit before has been read
      float2* rows = reinterpret_cast<float2*>(smem + C::kQsum);
#pragma unroll
      for (int ks = 0; ks < C::kM; ++ks)
        *reinterpret_cast<uint2*>(smem + C::kQ + ((ks * (NT / 2) + warp / 2) * 32 + lane) * 16 + (warp & 1) * 8) = make_uint2(qf[0][ks][0], qf[0][ks][1]);
      if (c == 0) rows[8 * warp + r] = make_float2(total, factor);
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 a = rows[8 * n + 2 * c], b = rows[8 * n + 2 * c + 1];
        qs[n] = make_float2(a.x, b.x);
        f[n] = a.y;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      ref[n] = zero2;
      over[n] = make_float2(-INFINITY, -INFINITY);
      sum[n] = base_sum[n] = csum[n][0] = csum[n][1] = zero2;
#pragma unroll
      for (int i = 0; i < C::kM; ++i) o[n][i][0] = o[n][i][1] = zero2;
    }
    int vexp = -100;  // every V scale so far is below 2^vexp = vlim; vf = 2^(kBoost - vexp)
    float vlim = pow2(-100), vf = pow2(kBoost + 100);
    // rows of this block: tokens first_tok .. last_tok of the new ones
    const int first_tok = row0 / p.group, last_tok = (min(row0 + C::kRows, p.rows) - 1) / p.group;
    const int full_to = len - p.n_new + first_tok + 1;  // every row sees the tokens before, from full_from
    const int full_from = p.window > 0 ? max(0, len - p.n_new + last_tok + 1 - p.window) : 0;

    if constexpr (C::kQreg) {
      if (owed && !dead && __all_sync(kFull, reached(taken_count + 4 * warp, own_parts))) fill_owed();
    }
    // NT <= 2: the warp with the unit's last tile of this run takes the others' parts
    const int k0 = max(at.base, 0);
    const int merger = C::kQreg ? (k1 - 1) % kWarps : 0;
    for (; k < k1; k += kWarps) {
      if (!dead && !__all_sync(kFull, mbar_test(bars + 8 * stage, phase)))
        dead = !__all_sync(kFull, mbar_wait(bars + 8 * stage, phase, p.wait_ns));
      if (dead) continue;
      const unsigned char* keys = smem + (warp * STAGES + stage) * C::kStage + C::kTileCodes;
      const unsigned char* pairs = smem + C::kPairRing + (warp * STAGES + stage) * C::kPairs;
      const int t0 = (at.s.first + k - at.base) * kU4Tile;
      const bool edge = t0 < full_from || t0 + kU4Tile > full_to;
#pragma unroll 1
      for (int sub = 0; sub < 4 / C::kMt; ++sub) {
        const int tok0 = 16 * C::kMt * sub + r;  // a lane's tokens: tok0 + 16 mt + 8 h
        // ---- S^T: [tile of 16 tokens][n tile], rows r, r + 8
        float2 s[C::kMt][NT][2];
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt) {
          uint32_t kw[2][D / 32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned char* src = keys + (tok0 + 16 * mt + 8 * h) * C::kCode + c * (D / 8);
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              kw[h][0] = v.x, kw[h][1] = v.y, kw[h][2] = v.z, kw[h][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              kw[h][0] = v.x, kw[h][1] = v.y;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) s[mt][n][0] = s[mt][n][1] = zero2;
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            uint32_t a[2][2], b[2][2];  // [k16 step][row]
            split_codes(kw[0][w], a[0][0], b[0][0], a[1][0], b[1][0]);
            split_codes(kw[1][w], a[0][1], b[0][1], a[1][1], b[1][1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int ks = 2 * w + i;
              if constexpr (C::kQreg) {
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(s[mt][n], a[i][0], a[i][1], b[i][0], b[i][1], qf[n][ks][0], qf[n][ks][1]);
              } else {
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                  const uint4 v = *reinterpret_cast<const uint4*>(smem + C::kQ + ((ks * (NT / 2) + n / 2) * 32 + lane) * 16);
                  mma_f16(s[mt][n], a[i][0], a[i][1], b[i][0], b[i][1], v.x, v.y);
                  mma_f16(s[mt][n + 1], a[i][0], a[i][1], b[i][0], b[i][1], v.z, v.w);
                }
              }
            }
          }
        }
        // ---- arguments of 2^x, the V pairs, and whether a maximum moves
        uint32_t vp[C::kMt][2];
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int tt = tok0 + 16 * mt + 8 * h;
            const uint32_t kp = *reinterpret_cast<const uint32_t*>(pairs + 4 * tt);
            vp[mt][h] = *reinterpret_cast<const uint32_t*>(pairs + 4 * (kU4Tile + tt));
            const float ks = u4_scale(kp), km = u4_min(kp);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float k_f = ks * f[n];
              float2& x = s[mt][n][h];
              x.x = fmaf(x.x, k_f, fmaf(km, qs[n].x, ref[n].x));
              x.y = fmaf(x.y, k_f, fmaf(km, qs[n].y, ref[n].y));
            }
          }
        if (edge) {
#pragma unroll
          for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int t = t0 + tok0 + 16 * mt + 8 * h;
              if (t >= len || t < at.s.lo) vp[mt][h] = 0;  // no row sees it, and anything may be there
            }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int tok = min(row0 + 8 * n + 2 * c + e, p.rows - 1) / p.group;
              const int last = len - p.n_new + tok, first = p.window > 0 ? max(0, last + 1 - p.window) : 0;
#pragma unroll
              for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int t = t0 + tok0 + 16 * mt + 8 * h;
                  if (t > last || t < first) (e ? s[mt][n][h].y : s[mt][n][h].x) = -INFINITY;
                }
            }
        }
        float vs[C::kMt][2], vmost = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt) {
          vs[mt][0] = u4_scale(vp[mt][0]), vs[mt][1] = u4_scale(vp[mt][1]);
          vmost = max3(vmost, fabsf(vs[mt][0]), fabsf(vs[mt][1]));
        }
        float2 most[NT];
        bool moves = vmost >= vlim;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          most[n] = make_float2(fmaxf(s[0][n][0].x, s[0][n][1].x), fmaxf(s[0][n][0].y, s[0][n][1].y));
#pragma unroll
          for (int mt = 1; mt < C::kMt; ++mt) {
            most[n].x = max3(most[n].x, s[mt][n][0].x, s[mt][n][1].x);
            most[n].y = max3(most[n].y, s[mt][n][0].y, s[mt][n][1].y);
          }
          moves |= most[n].x > over[n].x || most[n].y > over[n].y;
        }
        if (__any_sync(kFull, moves)) {
          const uint32_t big = __reduce_max_sync(kFull, vmost < INFINITY ? __float_as_uint(vmost) : 0u);
          const int e2 = max(vexp, static_cast<int>(big >> 23) - 126);
          const float down = pow2(max(vexp - e2, -126));
          vexp = e2;
          vlim = __uint_as_float(static_cast<uint32_t>(min(e2 + 127, 255)) << 23);
          vf = pow2(kBoost - vexp);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float2 m = most[n];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              m.x = fmaxf(m.x, __shfl_xor_sync(kFull, m.x, off));
              m.y = fmaxf(m.y, __shfl_xor_sync(kFull, m.y, off));
            }
            // the reference goes up by m where that is above 0, or there was none (and m is a score)
            const float2 up = make_float2(over[n].x == -INFINITY ? (m.x == -INFINITY ? 0.f : m.x) : fmaxf(m.x, 0.f),
                                          over[n].y == -INFINITY ? (m.y == -INFINITY ? 0.f : m.y) : fmaxf(m.y, 0.f));
            const float2 by = make_float2(over[n].x == -INFINITY ? 0.f : fast_exp2(-up.x), over[n].y == -INFINITY ? 0.f : fast_exp2(-up.y));
            const float2 scale = make_float2(by.x * down, by.y * down);
            if (m.x != -INFINITY) over[n].x = kSlack;
            if (m.y != -INFINITY) over[n].y = kSlack;
            ref[n] = make_float2(ref[n].x - up.x, ref[n].y - up.y);
            sum[n] = mul2(sum[n], by);
            base_sum[n] = mul2(base_sum[n], by);
            csum[n][0] = mul2(csum[n][0], scale);
#pragma unroll
            for (int i = 0; i < C::kM; ++i) {
              o[n][i][0] = mul2(o[n][i][0], scale);
              o[n][i][1] = mul2(o[n][i][1], scale);
            }
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) s[mt][n][h] = make_float2(s[mt][n][h].x - up.x, s[mt][n][h].y - up.y);
          }
        }
        // ---- p, and p s as the operand of O
        uint32_t pb[C::kMt][NT][2];
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float vm = fmaf(8.f, vs[mt][h], u4_min(vp[mt][h]));  // the codes are taken as -8 .. 7
            const float v = vs[mt][h] * vf;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float2 pr = make_float2(fast_exp2(s[mt][n][h].x), fast_exp2(s[mt][n][h].y));
              sum[n] = add2(sum[n], pr);
              base_sum[n].x = fmaf(pr.x, vm, base_sum[n].x);
              base_sum[n].y = fmaf(pr.y, vm, base_sum[n].y);
              pb[mt][n][h] = transpose8(pack_half2(pr.x * v, pr.y * v));
            }
          }
        // ---- O^T += V^T P^T: a transposed 8 x 8 matrix of 16-bit pieces holds four codes of a token in each half, tokens
        // 2 c, 2 c + 1, piece r of a 16-byte chunk
        const uint32_t ones = 0x3c003c00u;
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt) {
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(csum[n], ones, ones, ones, ones, pb[mt][n][0], pb[mt][n][1]);
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            uint32_t v[4];  // chunk 2 q: tokens 0-7, 8-15; chunk 2 q + 1
            ldsm_x4_trans(v_row[q] + stage * C::kStage + (C::kMt * sub + mt) * 16 * C::kCode, v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a[2][2], b[2][2];  // [pair of dims][tokens 0-7, 8-15]
              split_codes(v[2 * i], a[0][0], b[0][0], a[1][0], b[1][0]);
              split_codes(v[2 * i + 1], a[0][1], b[0][1], a[1][1], b[1][1]);
#pragma unroll
              for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_f16(o[n][4 * q + 2 * i + d], a[d][0], b[d][0], a[d][1], b[d][1], pb[mt][n][0], pb[mt][n][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage has been read
      if (C::kQreg && owed && !dead) {
        dead = !__all_sync(kFull, wait_count(taken_count + 4 * warp, own_parts, p.wait_ns));
        if (!dead) fill_owed();
      }
      if (fill_k < run && !dead) {
        if (C::kQreg && k + kWarps >= k1 && warp != merger)
          owed = true;  // the part goes into this stage first
        else
          fill_next();
      }
      if ((++consumed & 1) == 0) centre();
      if (++stage == STAGES) stage = 0, phase ^= 1;
    }

    // ---------------------------------------------- the end of the unit
    // o in units of V, base_sum in it
    centre();
    float2 top[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      top[n] = make_float2(over[n].x == -INFINITY ? -INFINITY : -ref[n].x, over[n].y == -INFINITY ? -INFINITY : -ref[n].y);
    const float out0 = pow2(min(max(vexp - kBoost, -126), 127)), out1 = 0x1p24f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        sum[n].x += __shfl_xor_sync(kFull, sum[n].x, off);
        sum[n].y += __shfl_xor_sync(kFull, sum[n].y, off);
        base_sum[n].x += __shfl_xor_sync(kFull, base_sum[n].x, off);
        base_sum[n].y += __shfl_xor_sync(kFull, base_sum[n].y, off);
      }
#pragma unroll
      for (int i = 0; i < C::kM; ++i) {
        const float2 even = o[n][i][0], both = o[n][i][1];
        o[n][i][0] = make_float2(fmaf(even.x * out0, out1, base_sum[n].x), fmaf(even.y * out0, out1, base_sum[n].y));
        o[n][i][1] = make_float2(fmaf((both.x - even.x) * out0, out1 * 0.0625f, base_sum[n].x),
                                 fmaf((both.y - even.y) * out0, out1 * 0.0625f, base_sum[n].y));
      }
    }
    auto merge = [&](const float2 (&m2)[NT], const float2 (&s2)[NT], auto&& load) {  // another part into this one
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 wa, wb;
        weights(top[n], m2[n], wa, wb);
        sum[n] = fma2(sum[n], wa, mul2(s2[n], wb));
#pragma unroll
        for (int i = 0; i < C::kM; ++i) {
          const float4 v = load(n * C::kM + i);
          o[n][i][0] = fma2(o[n][i][0], wa, mul2(make_float2(v.x, v.y), wb));
          o[n][i][1] = fma2(o[n][i][1], wa, mul2(make_float2(v.z, v.w), wb));
        }
      }
    };
    auto take = [&](const unsigned char* o2, const unsigned char* ml) {
      float2 m2[NT], s2[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m2[n] = reinterpret_cast<const float2*>(ml)[n * 32 + lane];
        s2[n] = reinterpret_cast<const float2*>(ml)[(NT + n) * 32 + lane];
      }
      merge(m2, s2, [&](int i) { return reinterpret_cast<const float4*>(o2)[i * 32 + lane]; });
    };
    auto leave = [&](unsigned char* o2, unsigned char* ml) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        reinterpret_cast<float2*>(ml)[n * 32 + lane] = top[n];
        reinterpret_cast<float2*>(ml)[(NT + n) * 32 + lane] = sum[n];
#pragma unroll
        for (int i = 0; i < C::kM; ++i)
          reinterpret_cast<float4*>(o2)[(n * C::kM + i) * 32 + lane] = make_float4(o[n][i][0].x, o[n][i][0].y, o[n][i][1].x, o[n][i][1].y);
      }
    };
    if constexpr (C::kQreg) {
      // A warp leaves its part in the stage that it has read last and goes on with the next unit; the stage is filled when
      // the part has been taken. Warps without a tile of the unit have no part.
      const int later = (merger + 1) % kWarps;  // the others in the order of their tiles
      uint32_t leaving = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (w != merger && k1 - 1 - (merger - w + kWarps) % kWarps >= k0) leaving |= 1u << w;
      if (lane < kWarps) parts[lane] += leaving >> lane & 1;
      __syncwarp();
      if (warp == merger) {
        for (int i = 0; i < kWarps - 1; ++i) {
          const int w = (later + i) % kWarps;
          if (!(leaving >> w & 1)) continue;
          const uint32_t n = parts[w];
          if (!dead) dead = !__all_sync(kFull, wait_count(left_count + 4 * w, n, p.wait_ns));
          if (!dead) take(smem + (w * STAGES + where[w]) * C::kStage, smem + C::kMl + w * C::kPartMl);
          __syncwarp();
          if (lane == 0) publish(taken_count + 4 * w, n);
        }
      } else if (leaving >> warp & 1) {
        const int last_stage = stage == 0 ? STAGES - 1 : stage - 1;
        if (part_out && !dead) dead = !__all_sync(kFull, wait_count(taken_count + 4 * warp, own_parts, p.wait_ns));
        part_out = true;
        ++own_parts;
        if (!dead) leave(smem + (warp * STAGES + last_stage) * C::kStage, smem + C::kMl + warp * C::kPartMl);
        if (lane == 0) where[warp] = last_stage;
        __syncwarp();
        if (lane == 0) publish(left_count + 4 * warp, own_parts);
      }
    } else {
      // The four warps' parts meet in a chain, warp 3's into warp 2's registers and so on, through one place. A warp that
      // has left its part goes on with the next unit.
      if (warp == kWarps - 1) {
        if (seg > 0 && !dead) dead = !__all_sync(kFull, mbar_wait(taken, (seg - 1) & 1, p.wait_ns));
      } else {
        if (!dead) dead = !__all_sync(kFull, mbar_wait(left + 8 * (warp + 1), seg & 1, p.wait_ns));
        take(smem + C::kMerge, smem + C::kMl);
      }
      if (warp != 0) leave(smem + C::kMerge, smem + C::kMl);
      __syncwarp();
      if (lane == 0) mbar_arrive(warp == 0 ? taken : left + 8 * warp);
    }
    if (warp == merger) {
      if (!p.whole && (at.base < 0 || at.end() > run)) {  // other blocks have parts of this unit
        const long long first = (start + at.base) / run_len, last = (start + at.end() - 1) / run_len;
        float* mine = p.part + (2 * blockIdx.x + (at.base < 0 ? 0 : 1)) * static_cast<long long>(C::kRows * (D + 2));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < C::kM; ++i)
            reinterpret_cast<float4*>(mine)[(n * C::kM + i) * 32 + lane] =
                make_float4(o[n][i][0].x, o[n][i][0].y, o[n][i][1].x, o[n][i][1].y);
          if (r == 0) {
            *reinterpret_cast<float2*>(mine + C::kRows * D + 8 * n + 2 * c) = top[n];
            *reinterpret_cast<float2*>(mine + C::kRows * (D + 1) + 8 * n + 2 * c) = sum[n];
          }
        }
        // told to the other blocks at the end of the run: a fence waits for memory that is busy with tiles (7 us here)
        if (lane == 0) {
          volatile int* todo = flag + (at.base < 0 ? 0 : 5);
          todo[0] = 1 + warp, todo[1] = at.b, todo[2] = at.u, todo[3] = static_cast<int>(first), todo[4] = static_cast<int>(last);
        }
      } else {
        write_rows(p, at.b, j, row0, top, sum, o, 0);
      }
    }
    if (k1 >= run) break;
    at.next(p, units);
#pragma unroll
    for (int n = 0; n < (C::kQreg ? NT : 1); ++n) load_q(at, C::kQreg ? n : warp, q[n]);
    prefetch_q(at);
  }

  // The last block to have left its part of a unit merges the unit's parts, in the order of the blocks; every warp takes
  // a quarter of the dims.
  if (!p.whole) {
    for (int which = 0; which < 2; ++which) {
      volatile int* todo = flag + 5 * which;
      if (todo[0] != 1 + warp) continue;  // (this warp has written the part)
      __threadfence();
      __syncwarp();
      if (lane != 0) continue;
      const bool all = atomicAdd(p.arrived + todo[3], 1) == todo[4] - todo[3];
      __threadfence();
      todo[0] = all ? -1 : 0;
    }
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
      volatile int* todo = flag + 5 * which;
      if (todo[0] == 0) continue;
      const int b_of = todo[1], u = todo[2], first = todo[3], last = todo[4], j = u / p.row_blocks, row0 = (u - j * p.row_blocks) * C::kRows;
      constexpr int kPart = C::kM / kWarps;
      float2 acc[NT][kPart][2], top[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n] = make_float2(-INFINITY, -INFINITY);
        sum[n] = zero2;
#pragma unroll
        for (int i = 0; i < kPart; ++i) acc[n][i][0] = acc[n][i][1] = zero2;
      }
      constexpr int kAhead = NT == 1 ? 4 : 2;  // parts whose loads are issued together
      for (int b0 = first; b0 <= last; b0 += kAhead) {
        float2 m2[kAhead][NT], s2[kAhead][NT];
        float4 v[kAhead][NT][kPart];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int b = min(b0 + a, last);
          const float* src = p.part + (2 * b + (b == first ? 1 : 0)) * static_cast<long long>(C::kRows * (D + 2));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            m2[a][n] = __ldcg(reinterpret_cast<const float2*>(src + C::kRows * D + 8 * n + 2 * c));
            s2[a][n] = __ldcg(reinterpret_cast<const float2*>(src + C::kRows * (D + 1) + 8 * n + 2 * c));
#pragma unroll
            for (int i = 0; i < kPart; ++i) v[a][n][i] = __ldcg(reinterpret_cast<const float4*>(src) + (n * C::kM + warp * kPart + i) * 32 + lane);
          }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (b0 + a > last) break;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float2 wa, wb;
            weights(top[n], m2[a][n], wa, wb);
            sum[n] = fma2(sum[n], wa, mul2(s2[a][n], wb));
#pragma unroll
            for (int i = 0; i < kPart; ++i) {
              acc[n][i][0] = fma2(acc[n][i][0], wa, mul2(make_float2(v[a][n][i].x, v[a][n][i].y), wb));
              acc[n][i][1] = fma2(acc[n][i][1], wa, mul2(make_float2(v[a][n][i].z, v[a][n][i].w), wb));
            }
          }
        }
      }
      write_rows(p, b_of, j, row0, top, sum, acc, warp * kPart);
    }
  }
  if (dead) {
    if (lane == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_TIMEOUT));
    for (; consumed < issued; ++consumed) {
      mbar_wait(bars + 8 * stage, phase, kWaitLimitNs);
      if (++stage == STAGES) stage = 0, phase ^= 1;
    }
  }
}

__global__ void u4_clear_kernel(int32_t* arrived, int count) {
  grid_dependents_launch();
  for (int i = threadIdx.x; i < count; i += blockDim.x) arrived[i] = 0;
}

template <int D, int NT, bool PAGED, int STAGES, int CTAS>
cudaError_t launch_u4_t(const U4Params& p, const CUtensorMap& tmap_v, int ctas, bool clear, cudaStream_t stream) {
  using C = Cfg<D, NT, STAGES>;
  const auto kernel = attn_u4_kernel<D, NT, PAGED, STAGES, CTAS>;
  // (an attribute of the function on the current device: set on each call, as it costs nothing beside the launch)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if (clear) {
    u4_clear_kernel<<<1, 256, 0, stream>>>(p.arrived, ctas);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.whole ? static_cast<long long>(p.batch) * p.h_kv * p.row_blocks : ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.early || clear ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, tmap_v, p);
}

constexpr int kStages = 2;
constexpr int kCtas1 = 3, kCtas2 = 2, kCtas4 = 2;

template <int D, bool PAGED>
cudaError_t launch_u4_d(const U4Params& p, const CUtensorMap& tv, int ctas, bool clear, cudaStream_t stream) {
  if (p.rows <= 8) return launch_u4_t<D, 1, PAGED, kStages, kCtas1>(p, tv, ctas, clear, stream);
  if (p.rows <= 16) return launch_u4_t<D, 2, PAGED, kStages, kCtas2>(p, tv, ctas, clear, stream);
  return launch_u4_t<D, 4, PAGED, kStages, kCtas4>(p, tv, ctas, clear, stream);
}

}  // namespace

U4Shape u4_shape(int head_dim, int rows) {
  (void)head_dim;
  if (rows <= 8) return {8, kCtas1};
  if (rows <= 16) return {16, kCtas2};
  return {32, kCtas4};
}

cudaError_t launch_attn_u4(const U4Params& p, const CUtensorMap& tv, int ctas, bool clear, cudaStream_t stream) {
  if (p.paged)
    return p.head_dim == 128 ? launch_u4_d<128, true>(p, tv, ctas, clear, stream) : launch_u4_d<64, true>(p, tv, ctas, clear, stream);
  return p.head_dim == 128 ? launch_u4_d<128, false>(p, tv, ctas, clear, stream) : launch_u4_d<64, false>(p, tv, ctas, clear, stream);
}

}  // namespace mqa
