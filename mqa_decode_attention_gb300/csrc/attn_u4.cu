// Attention over a 4-bit cache (rows of codes c and one bf16 pair (s, m), the
// value m + s c: u4.cuh), one to 32 new tokens per sequence.
//
// With K = m + s c and V alike, the scaling stays outside the products:
//   q . K_t = s_t (q . c_t) + m_t sum(q)
//   O       = sum_t (p_t s_t) c_t + sum_t p_t m_t,
// so the tensor cores multiply codes as they are. A code in the low bits of a
// half is the fp16 number c 2^-24, and the byte of two codes (c_even + 16 c_odd)
// 2^-24, both exact: an AND each makes an operand, without a shift or a
// conversion. So K's even places meet q_even - q_odd / 16, its odd ones q_odd / 16,
// and V's odd dims are (both - even) / 16 of what comes out. The 2^-24 goes into
// the scores' factor and the output.
//
// q enters as fp16 (11 bits), each row scaled by a power of two to a largest
// value in [2^13, 2^14); sum(q) is that of the rounded values, since s c and m
// cancel in part. p s enters as fp16 too. What has to keep its bits there is a
// column's largest p s, whatever other rows hold: so the reference that a
// column's p are relative to follows the maximum of score + log2 of the row's
// size, not of the score alone. A row's size 2^l is the power of two above s and
// |m| / 16, over 2^E and taken as 2^-60 at the least (E = 0, but where the rows of
// the unit's first tile are far from 1); p s 2^(11 - E) has its 11 bits down to
// 2^-25 of the column's largest, and p, which may be 2^64, and its sums are fp32.
// (With p relative to the largest score, and 2^E above the largest s met, one row
// of 2^36 times the others' scale and no weight took all their codes.) Scores,
// maxima, sums and O are fp32. The reference is only followed when it is passed
// by more than 4 (in log2). Every two tiles 8 sum(p s) is taken from O, which
// makes the codes -8 to 7: else O and sum p m grow with the number of tokens
// while what they leave does not (131072 tokens: error 1.7e-3, without 2.5e-3).
//
// A warp takes 8 NT query rows of one kv head and tiles of 64 tokens: S^T = K Q^T
// (m16n8k16, tokens on the rows), softmax over the lanes that hold a column,
// P^T transposed in registers (movmatrix), O^T += V^T P^T (dims on the rows, so
// O's columns are S's): nothing but K, V and q passes through shared memory.
// Codes stream through a ring of two stages of its own, filled with bulk copies
// by the warp itself: the warps of a block, four, or six where units are whole and
// few, meet at the end of a unit only (unit: sequence, kv head, block of query
// rows).
//
// Who does what: a block takes a whole unit; or all resident blocks share the
// tiles, a unit in equal parts, or all units in order cut into equal runs, so
// that lengths of any spread load all SMs alike. A unit that several blocks share
// is merged by the last of them to arrive, in the order of the blocks, so that
// equal calls give equal bits. (Both sides of these choices are measured where
// they are made.)
//
// What bounds it. Up to 8 rows with 3 blocks on every SM: HBM (1024 units of 8192
// tokens 191 us, 6.0 TB/s; pages of 64 tokens 211; of 16, whose tile is 8 bulk
// copies, 225, and some 13 more with the pairs by bulk copies too). With fewer units the
// chain products - softmax - products of a warp, 1.3 us a tile (256 units of 4096
// tokens 32 us, 4.5 TB/s), at the least 5.5 us for the launch, the first tile and
// the last merge. 9 to 32 rows: the tensor pipes, 256 multiply-adds a cycle and
// scheduler with mma.sync, half busy, since the registers leave two warps to a
// scheduler (64 MQA units of 8192 tokens 50 us, floor by
// products 15). For runs four warps and three blocks on an SM were the best of
// 6 x 2, 8 x 1 and 12 x 1; a fifth warp that fills the rings cost its registers
// more than it gave.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "u4.cuh"

namespace mqa {
namespace {

constexpr int kBoost = 11;      // p s 2^(kBoost - E), p s <= 2^(E + kSlack)
constexpr float kSlack = 4.f;
// log2 of a row's size over 2^E: a smaller row counts as 2^kLeast (bounds p), one above 2^kMost moves E. (Parts of a unit
// are merged by weights of down to 2^(kLeast - kMost), which fp32 holds.)
constexpr float kLeast = -60.f, kMost = 66.f;
constexpr uint32_t kFull = 0xffffffffu;
// The least tiles of a run (one of 1, 2, 4, 8: a batch of 8 x 32 units, one sequence of 2048 tokens and 31 of 100 in pages,
// 15.0, 14.8, 13.8, 20.4 us; 4 x 64 units, one of 4096 tokens and 63 of 64, 20.0, 20.1, 19.0, 31.9) and of a part of a unit
// (8 units of 2048 tokens 20.0, 14.8, 12.8, 12.5 us, of 1200 tokens 15.4, 12.1, 11.6, 12.1; MQA, 8 x 2048, 29.6, 24.1, 19.3,
// 20.3).
constexpr int kMinRun = 4, kMinPart = 4;

template <int D, int NT, int STAGES, int WARPS>
struct Cfg {
  static constexpr int kWarps = WARPS;
  static constexpr int kMt = NT == 1 ? 4 : NT == 2 ? 2 : 1;      // tiles of 16 tokens whose scores are held at a time
  static constexpr int kCode = D / 2;              // bytes of a row's codes
  static constexpr int kTileCodes = kU4Tile * kCode;
  static constexpr int kStage = 2 * kTileCodes;    // V codes (swizzled), K codes
  static constexpr int kPairs = 2 * 4 * kU4Tile;   // K pairs, V pairs
  static constexpr int kRows = 8 * NT;
  static constexpr int kM = D / 16;   // 16-row tiles of O^T; also the k16 steps of q . c
  static constexpr int kPairRing = kWarps * STAGES * kStage;
  // q as operands: NT <= 2 in registers, formed by each warp from the rows in shared memory (a lane's quarter row a slot
  // of 16 bytes more, so that 8 lanes read different banks); else [k16 step][pair of n tiles][lane][2], by all warps
  static constexpr bool kQreg = NT <= 2;
  static constexpr int kSlot = D + 16;
  static constexpr int kQ = kPairRing + kWarps * STAGES * kPairs;
  static constexpr int kQsum = kQ + (kQreg ? NT * 32 * kSlot : kM * NT * 32 * 8);     // [rows] (sum of q, factor)
  // parts of a unit that warps leave: O in a stage of their own ring (NT <= 2), else in one place; maxima and sums behind
  // it (NT = 1) or in places of their own
  static constexpr int kPart = kM * NT * 32 * 16, kPartMl = 2 * NT * 32 * 8;
  static constexpr int kMerge = kQsum + (kQreg ? 0 : kRows * 8);
  static constexpr int kMl = kMerge + (kQreg ? 0 : kPart);
  // .. of the run's last unit: in the pairs' ring
  static constexpr int kEnd = NT == 4 ? kMl + kPartMl : kPairRing, kEndStep = NT == 4 ? kPartMl : STAGES * kPairs;
  static constexpr int kBar = NT == 1 ? kMl : NT == 2 ? kMl + kWarps * STAGES * kPartMl : kMl + (1 + kWarps) * kPartMl;
  static_assert(NT == 4 || kPartMl <= kEndStep, "maxima and sums fit the pairs' ring");
  // barriers: a stage is full, a stage is empty [warps][stages]; q has come, q has been read; the chain [warps] and its place
  static constexpr int kFlag = kBar + (2 * kWarps * STAGES + 2 + kWarps + 1) * 8;
  static_assert(NT != 1 || kPart + kPartMl <= kStage, "a part fits a stage");
  static_assert(!kQreg || kPart <= kStage, "a part fits a stage");
  static constexpr int kWords = 10 + kWarps * (2 + 1 + kWarps + 1);  // (see flag)
  static constexpr int kSmem = kFlag + 4 * kWords;
};

// d += A B, d the pairs of columns of rows r and r + 8
__device__ __forceinline__ void mma_f16(float2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = A B
__device__ __forceinline__ void mma_f16_first(float2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0].x), "=f"(d[0].y), "=f"(d[1].x), "=f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// an 8 x 8 matrix of 16-bit values across the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
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

// 16 bytes to shared memory, and an arrival when this thread's such copies have landed
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
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

template <int D, int NT, bool PAGED, int STAGES, int CTAS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) attn_u4_kernel(const __grid_constant__ CUtensorMap tmap_v, const U4Params p) {
  using C = Cfg<D, NT, STAGES, WARPS>;
  constexpr int kWarps = WARPS, kThreads = 32 * WARPS;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int units = p.h_kv * p.row_blocks;
  // a warp's stages and their barriers
  auto stage_at = [&](int w, int st) { return (w * STAGES + st) * C::kStage; };
  auto pairs_at = [&](int w, int st) { return C::kPairRing + (w * STAGES + st) * C::kPairs; };
  const uint32_t base = smem_u32(smem);
  auto full = [&](int w, int st) { return base + C::kBar + (w * STAGES + st) * 8; };
  auto empty = [&](int w, int st) { return base + C::kBar + (kWarps * STAGES + w * STAGES + st) * 8; };
  const uint32_t q_come = base + C::kBar + 2 * kWarps * STAGES * 8, q_read = q_come + 8;
  const uint32_t chain = q_read + 8, chain_free = chain + 8 * kWarps;  // NT = 4
  // words: units to merge at the end [2]: flag, sequence, unit, first and last block; [w][2] the stage of a part that warp w
  // has left (of its n-th in n % 2); [w] how many it has left; [w][w] .. as far as another warp has come; [w] the stage of its
  // part of the run's last unit
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::kFlag);
  volatile int* where = flag + 10;
  // (counts, not a barrier: a warp may be any number of units ahead of another's part, which the parity of a phase could
  // not tell apart)
  const uint32_t left_count = base + C::kFlag + 4 * (10 + 2 * kWarps);
  volatile uint32_t* parts = reinterpret_cast<volatile uint32_t*>(flag + 10 + 3 * kWarps) + kWarps * warp;

  const int first_len = !p.whole && lane < p.batch ? p.seq_lens[lane] : 0;
  for (int i = threadIdx.x; i < C::kWords; i += kThreads) flag[i] = 0;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmap_v);
    for (int i = 0; i < 2 * kWarps * STAGES; ++i) mbar_init(base + C::kBar + 8 * i, i < kWarps * STAGES ? 1 + 32 : 1);  // (see fill_next)
    mbar_init(q_come, 1);
    mbar_init(q_read, kWarps);
    for (int w = 0; w <= kWarps; ++w) mbar_init(chain + 8 * w, 1);
    fence_mbar_init();
  }
  __syncthreads();

  // ------------------------------------------------------ this block's run
  Place at;
  int run;             // tiles of the run
  long long start = 0, run_len = 1;  // place of the run among all tiles, length of the runs
  int me = blockIdx.x;  // place of this block's work in the order of the tiles
  // one of the equal parts of a unit, of which the first `more` units have one more than the others; the first parts of all
  // units go to the first blocks, which are spread over the SMs
  auto part_of_unit = [&](int parts, int more, int least) {
    const int all = p.batch * units, part = blockIdx.x / all, unit = blockIdx.x - part * all;
    const int of = parts + (unit < more ? 1 : 0);
    me = unit * parts + min(unit, more) + part;
    at.b = unit / units;
    at.u = unit - at.b * units;
    at.s = part < of ? span_of(p, p.seq_lens[at.b]) : Span{0, 0, 0, 0};
    const int per = max(least, (at.s.tiles + of - 1) / of);
    at.base = -part * per;
    run = max(0, min(per, at.s.tiles - part * per));
    run_len = per;
    start = run_len * me;
  };
  if (p.whole) {
    part_of_unit(1, 0, 1);
    if (run == 0 && at.u == 0 && threadIdx.x == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_SEQ_LEN));
  } else {
    // (every warp finds it for itself; 32 sequences at a time, the first 32 kept)
    auto tiles_of = [&](int b) { return b < p.batch ? span_of(p, p.seq_lens[b]).tiles : 0; };
    const int mine = lane < p.batch ? span_of(p, first_len).tiles : 0;
    bool bad = lane < p.batch && mine == 0;
    unsigned long long total = __reduce_add_sync(kFull, static_cast<unsigned>(mine));
    int most = __reduce_max_sync(kFull, mine);
    for (int b0 = 32; b0 < p.batch; b0 += 32) {
      const int t = tiles_of(b0 + lane);
      bad |= b0 + lane < p.batch && t == 0;
      total += __reduce_add_sync(kFull, static_cast<unsigned>(t));
      most = max(most, __reduce_max_sync(kFull, t));
    }
    if (blockIdx.x == 0 && warp == 0 && __any_sync(kFull, bad) && lane == 0)
      atomicOr(p.err, static_cast<int>(MQA_DEVERR_SEQ_LEN));
    total *= units;
    bool placed = false;
    run_len = total < 1ull << 31 ? static_cast<unsigned>(total + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
    run_len = max(run_len, static_cast<long long>(kMinRun));
    // Parts of units where the longest is not much longer than a run, in which a change of unit costs as much as some 16
    // tiles (8 x 8 units of 32 tiles 14 us, in runs 19; 160 units of 64 tiles 28 and 31; 256 units of 128 tiles 67 and 62; 64
    // units of 128 tiles for 32 query rows 51 and 59).
    if (p.parts > 0 && (most + p.parts - 1) / p.parts <= run_len + run_len / 2 + 16) {
      part_of_unit(p.parts, gridDim.x - p.parts * p.batch * units, kMinPart);
      placed = true;
    } else {
      at.b = at.u = at.base = 0;
      at.s = {0, 0, 0, 1};
      start = run_len * blockIdx.x;
      run = static_cast<int>(max(0ll, min(run_len, static_cast<long long>(total) - start)));
    }
    long long seen = 0;  // tiles of the sequences before (of one unit each)
    for (int b0 = 0; !placed && run > 0 && b0 < p.batch; b0 += 32) {
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
        at.s = span_of(p, b0 == 0 ? __shfl_sync(kFull, first_len, l) : p.seq_lens[at.b]);
        const long long off = start - (seen + __shfl_sync(kFull, upto, l) - at.s.tiles) * units;
        at.u = off < 1ll << 31 ? static_cast<unsigned>(off) / at.s.tiles : static_cast<int>(off / at.s.tiles);
        at.base = -static_cast<int>(off - static_cast<long long>(at.u) * at.s.tiles);
        break;
      }
      seen += __shfl_sync(kFull, upto, 31);
    }
  }
  if (run <= 0) {  // the whole block; after the append, so that a launch without any work does not end before it
    grid_dependency_wait();
    return;
  }

  // -------------------------------------------------- filling the rings
  // Tile k of the run goes to warp k % kWarps, into stage k / kWarps % STAGES of its ring. Two lanes, each a bulk copy: V
  // codes (through a tensor map, so that they land swizzled) and K codes; of a paged pool two lanes for each page. The pairs
  // of K and V, 16 bytes a lane: copies that lanes issue one after the other are what the warp waits for.
  Place fill = at;
  int fill_k = warp, issued = 0;
  int fill_t = 0, head = 0, page = 0;  // the next tile's first token, its kv head, this lane's page of it
  const int kind = lane & 1;
  const int piece_shift = PAGED ? min(__ffs(p.page_size), __ffs(kU4Tile)) - 1 : 0, piece = PAGED ? 1 << piece_shift : kU4Tile;  // tokens of a copy
  const int at_row = (lane >> 1) * piece;  // a lane's first token in the tile
  const unsigned char* pairs_from = reinterpret_cast<const unsigned char*>(lane < 16 ? p.k_sm : p.v_sm);
  const int pair_row = 4 * (lane & 15);
  auto wanted = [&]() {  // this lane's page has a token that is seen
    const int t = fill_t + at_row;
    return at_row < kU4Tile && t < fill.s.len && t + piece > fill.s.lo;
  };
  const int page_shift = PAGED ? __ffs(p.page_size) - 1 : 0;
  auto enter = [&]() {  // tile fill_k is the first of its unit, or of the run, that is filled here
    while (fill_k >= fill.end()) fill.next(p, units);
    head = fill.u / p.row_blocks;
    if (!PAGED) head += fill.b * p.h_kv;
    fill_t = (fill.s.first + fill_k - fill.base) * kU4Tile;
  };
  auto look = [&]() {  // this lane's page of tile fill_k (looked up one fill ahead)
    if (PAGED && fill_k < run && wanted()) page = p.block_table[static_cast<long long>(fill.b) * p.max_pages + ((fill_t + at_row) >> page_shift)];
  };
  auto fill_next = [&](int w, int st) {  // tile fill_k < run; the stage is empty
    const uint32_t bar = full(w, st);
    const uint32_t dst = base + at_row * C::kCode + stage_at(w, st) + (kind == 1 ? C::kTileCodes : 0);
    const uint32_t pair_dst = base + pairs_at(w, st) + 16 * lane;
    // (a part of a unit may have been written and read there by threads, the tile comes by the async proxy)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (PAGED) {
      const bool seen = wanted(), copy = seen && page >= 0 && page < p.num_pages;
      if (seen && !copy && kind == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_PAGE_RANGE));
      const int copies = __popc(__ballot_sync(kFull, copy)) / 2;
      if (lane == 0) mbar_arrive_expect_tx(bar, copies * piece * (2 * C::kCode));
      __syncwarp();
      const int pair_page = __shfl_sync(kFull, copy ? page : -1, 2 * (pair_row >> piece_shift));
      if (pair_page >= 0)
        copy16(pair_dst, pairs_from + 4 * (((static_cast<long long>(pair_page) * p.h_kv + head) << page_shift) +
                                           ((fill_t + pair_row) & (p.page_size - 1))));
      if (copy) {
        const int in_page = (fill_t + at_row) & (p.page_size - 1);
        if (kind == 0)
          tma_load_4d(dst, &tmap_v, 0, in_page, head, page, bar);
        else
          bulk_g2s(dst, p.k_cache + (((static_cast<long long>(page) * p.h_kv + head) << page_shift) + in_page) * C::kCode, piece * C::kCode, bar);
      }
    } else {
      // (the capacity is a multiple of 4 rows: copies of 16 bytes; the tensor map's are whole tiles)
      const int n = min(kU4Tile, (fill.s.len - fill_t + 3) & ~3);
      const long long row = head * p.capacity + fill_t;
      if (pair_row < n) copy16(pair_dst, pairs_from + 4 * (row + pair_row));
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, (kU4Tile + n) * C::kCode);
        tma_load_3d(dst, &tmap_v, 0, fill_t, head, bar);
        bulk_g2s(dst + C::kTileCodes, p.k_cache + row * C::kCode, n * C::kCode, bar);
      }
      __syncwarp();
    }
    arrive_copies(bar);
    ++issued;
    fill_k += kWarps;
    fill_t += kWarps * kU4Tile;
    if (fill_k >= fill.end() && fill_k < run) enter();
    look();
  };
  // A unit's query rows: lane (r, c) has row r of an n tile, quarter c of its dims.
  auto q_row = [&](const Place& u, int n) -> const float* {  // null past the last row
    const int j = u.u / p.row_blocks, ridx = (u.u - j * p.row_blocks) * C::kRows + 8 * n + r, tok = ridx / p.group;
    return ridx < p.rows ? p.q_rot + ((static_cast<long long>(u.b) * p.n_new + tok) * p.h_q + j * p.group + ridx - tok * p.group) * D + c * (D / 4)
                         : nullptr;
  };
  // NT <= 2: copied by one warp, a unit ahead: a load would wait behind the tiles under way
  auto send_q = [&](const Place& u) {
    const float* src[NT];
    uint32_t bytes = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      src[n] = q_row(u, n);
      bytes += src[n] != nullptr ? D : 0;
    }
    bytes = __reduce_add_sync(kFull, bytes);
    if (lane == 0) mbar_arrive_expect_tx(q_come, bytes);
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (src[n] != nullptr) bulk_g2s(base + C::kQ + (n * 32 + lane) * C::kSlot, src[n], D, q_come);
  };
  bool dead = false;  // a wait ran out
  // before the append has ended only a tile without new rows
  if (fill_k < run) enter();
  look();
  if (p.early && fill_k < run && fill_t + kU4Tile <= fill.s.len - p.n_new) fill_next(warp, 0);
  grid_dependency_wait();
  // The first unit's q by loads ahead of the other tiles: behind them it would wait until they have all come (31 MB from
  // all blocks, 5 us). NT <= 2: warp 0 puts it where the others look for it; else a warp has the rows of its n tile.
  float4 q0[C::kQreg ? NT : 1][D / 16];
  if (warp == 0 || !C::kQreg) {
#pragma unroll
    for (int n = 0; n < (C::kQreg ? NT : 1); ++n) {
      const float4* src = reinterpret_cast<const float4*>(q_row(at, C::kQreg ? n : warp));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) q0[n][i] = src != nullptr ? src[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  while (issued < STAGES && fill_k < run) fill_next(warp, issued);

  // q as operands: lane (r, c) forms those of row r, quarter c of the dims, of an n tile. Even dims meet single codes, odd
  // dims code pairs (even + 16 odd): x = q_odd / 16 and q_even - x, each rounded.
  auto operands = [&](const float4 (&q4)[D / 16], uint32_t (&h)[C::kM][2], float& total, float& factor) {
    float q[D / 4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[4 * i] = q4[i].x, q[4 * i + 1] = q4[i].y, q[4 * i + 2] = q4[i].z, q[4 * i + 3] = q4[i].w;
    uint32_t most = 0;  // bits of the largest finite magnitude
#pragma unroll
    for (int i = 0; i < D / 4; ++i) {
      const uint32_t m = __float_as_uint(q[i]) & 0x7fffffffu;
      most = max(most, m < 0x7f800000u ? m : 0u);
    }
    most = max(most, __shfl_xor_sync(kFull, most, 1));  // (a factor for each row)
    most = max(most, __shfl_xor_sync(kFull, most, 2));
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
  // NT = 4: each warp forms the operands of an n tile for all
  auto share_q = [&](const float4 (&q4)[D / 16]) {
    uint32_t h[C::kM][2];
    float total, factor;
    operands(q4, h, total, factor);
    __syncthreads();  // the unit before has been read
    float2* rows = reinterpret_cast<float2*>(smem + C::kQsum);
#pragma unroll
    for (int ks = 0; ks < C::kM; ++ks)
      *reinterpret_cast<uint2*>(smem + C::kQ + ((ks * (NT / 2) + warp / 2) * 32 + lane) * 16 + (warp & 1) * 8) = make_uint2(h[ks][0], h[ks][1]);
    if (c == 0) rows[8 * warp + r] = make_float2(total, factor);
    __syncthreads();
  };
  if constexpr (C::kQreg) {
    if (warp == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) reinterpret_cast<float4*>(smem + C::kQ + (n * 32 + lane) * C::kSlot)[i] = q0[n][i];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_come);
    }
  } else {
    static_assert(C::kQreg || NT == kWarps, "each warp forms the operands of one n tile");
    share_q(q0[0]);
  }

  // ------------------------------------------------------------ the run
  // Columns 2 c, 2 c + 1 of each n tile as pairs. o: rows r (the even dims) and
  // r + 8 (even + 16 odd, until the unit ends). base_sum: sum p (m + 8 s).
  float2 o[NT][C::kM][2];
  // ref: minus the reference of a column's exponents, -0 before its first score (and never -0 after); over: what a score and
  // its row's size may pass it by before it is followed (-inf while a column of the lane has had none).
  float2 ref[NT], sum[NT], base_sum[NT];
  float over;
  constexpr float kNone = -0.f, kNothing = -200.f;  // kNothing: log2 of the size of a row of zeros
  auto none = [](float x) { return __float_as_uint(x) == 0x80000000u; };
  // Sum of the operands p s, by the tensor cores: 8 times it is taken from o every few tiles, which makes the codes -8 to 7.
  // (Else o grows with the number of tokens while its sum with base_sum does not, and the rounding of the accumulators shows.)
  // NT = 4: of the lane's own tokens, before they are rounded, by additions (the registers of [1], which nothing needs, are
  // short there; the difference is of the size of the rounding).
  constexpr bool kSumTc = NT <= 2;
  float2 csum[NT][kSumTc ? 2 : 1];
  int consumed = 0, stage = 0, k = warp;
  uint32_t phase = 0;
  uint32_t own_parts = 0;  // parts that this warp has left
  // a warp that fills its own ring: stages read and not filled again; the next unit's q has been sent for, units whose q has been
  int free_stages = 0;
  bool q_sent = false;
  uint32_t q_count = 1;
  // ldmatrix rows of V: matrices (tokens 0-7, 8-15) x two 16-byte chunks of the rows
  uint32_t v_row[D / 64];
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    const int tok = (lane & 7) + (lane & 8), chunk = 2 * q + (lane >> 4);
    v_row[q] = base + stage_at(warp, 0) + tok * C::kCode + ((chunk ^ (D == 128 ? (lane & 7) >> 1 : (lane & 7) >> 2)) << 4);
  }
  // Tells the other blocks of the first unit's part that this warp has written, and finds whether it was the unit's last
  // (flag[0]: 0 nothing written, 1 + warp written, 5 told, -1 all parts are there) -- some tiles after it has been written:
  // a fence right behind it waits for memory that is busy with tiles (7 us here).
  int tell_at = -1;  // when so many tiles have been read
  auto tell = [&]() {
    if (flag[0] != 1 + warp) return;
    __threadfence();
    __syncwarp();
    if (lane == 0) {
      const bool all = atomicAdd(p.arrived + flag[3], 1) == flag[4] - flag[3];
      __threadfence();
      flag[0] = all ? -1 : 5;
    }
    __syncwarp();
  };
  const float2 zero2 = make_float2(0.f, 0.f);
  auto centre = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 total = csum[n][0];
      if constexpr (!kSumTc) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          total.x += __shfl_xor_sync(kFull, total.x, off);
          total.y += __shfl_xor_sync(kFull, total.y, off);
        }
      }
      const float2 even = mul2(total, make_float2(-8.f * 0x1p-24f, -8.f * 0x1p-24f));
      const float2 both = mul2(total, make_float2(-136.f * 0x1p-24f, -136.f * 0x1p-24f));
#pragma unroll
      for (int i = 0; i < C::kM; ++i) {
        o[n][i][0] = add2(o[n][i][0], even);
        o[n][i][1] = add2(o[n][i][1], both);
      }
      csum[n][0] = zero2;
      if constexpr (kSumTc) csum[n][1] = zero2;
    }
  };

  float2 top[NT];
  int j, row0;  // kv head and first row of the unit
  for (uint32_t seg = 0;; ++seg) {
    const int k1 = min(run, at.end());
    j = at.u / p.row_blocks, row0 = (at.u - j * p.row_blocks) * C::kRows;
    const int len = at.s.len;
    uint32_t qf[C::kQreg ? NT : 1][C::kM][2];
    float2 qs[C::kQreg ? NT : 1];  // sum(q), and
    float2 f[C::kQreg ? NT : 1];   // the factor of the scores, times which qs is (NT = 4: read where they are used)
    if constexpr (C::kQreg) {
      if (!dead) dead = !__all_sync(kFull, mbar_wait(q_come, seg & 1, p.wait_ns));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float4 q4[D / 16];
        const bool live = q_row(at, n) != nullptr;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          q4[i] = live ? reinterpret_cast<const float4*>(smem + C::kQ + (n * 32 + lane) * C::kSlot)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        float total, factor;
        operands(q4, qf[n], total, factor);
        qs[n] = make_float2(__shfl_sync(kFull, total, 8 * c), __shfl_sync(kFull, total, 8 * c + 4));
        f[n] = make_float2(__shfl_sync(kFull, factor, 8 * c), __shfl_sync(kFull, factor, 8 * c + 4));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_read);
      q_sent = k1 >= run;  // (nothing to send)
    }
    auto send_next_q = [&]() {  // warp 0, when every warp has read this unit's
      Place u = at;
      u.next(p, units);
      if (seg == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the first unit's was written by threads)
      send_q(u);
      q_sent = true;
      ++q_count;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      ref[n] = make_float2(kNone, kNone);
      sum[n] = base_sum[n] = csum[n][0] = zero2;
      if constexpr (kSumTc) csum[n][1] = zero2;
#pragma unroll
      for (int i = 0; i < C::kM; ++i) o[n][i][0] = o[n][i][1] = zero2;
    }
    over = -INFINITY;
    // sizes of V rows are relative to 2^E: vf = 2^(kBoost - E), size_from = kSizeFrom + E; both 0 before a row that is not 0 has
    // been met (0 operands of O then)
    constexpr float kSizeFrom = 0x1p23f + 126.f;  // (a float's exponent bits e in the low bits of 2^23: 2^(e - 126) is above it)
    float size_from = 0.f, vf = 0.f;
    if (!C::kQreg && k1 < run) {  // the next unit's rows of q into the L2 cache
      Place u = at;
      u.next(p, units);
      const float* row = q_row(u, warp);
      if (row != nullptr) prefetch_l2(row);
    }
    // rows of this block: tokens first_tok .. last_tok of the new ones
    const int first_tok = row0 / p.group, last_tok = (min(row0 + C::kRows, p.rows) - 1) / p.group;
    const int full_to = len - p.n_new + first_tok + 1;  // every row sees the tokens before, from full_from
    const int full_from = p.window > 0 ? max(0, len - p.n_new + last_tok + 1 - p.window) : 0;

    // NT <= 2: the warp with the unit's last tile of this run takes the others' parts
    const int k0 = max(at.base, 0);
    const int merger = C::kQreg ? (k1 - 1) % kWarps : 0;
    for (; k < k1; k += kWarps) {
      {
        if (C::kQreg && warp == 0 && !q_sent && __all_sync(kFull, mbar_test(q_read, seg & 1))) send_next_q();
        // a stage that holds this warp's part is empty when the part has been taken; with no tile left to go on with, that
        // is waited for
        while (free_stages > 0 && fill_k < run && !dead) {
          const int st = issued % STAGES;
          const uint32_t parity = (issued / STAGES - 1) & 1;
          if (!__all_sync(kFull, mbar_test(empty(warp, st), parity))) {
            if (consumed < issued) break;
            dead = !__all_sync(kFull, mbar_wait(empty(warp, st), parity, p.wait_ns));
            if (dead) break;
          }
          fill_next(warp, st);
          --free_stages;
        }
      }
      if (!dead && !__all_sync(kFull, mbar_test(full(warp, stage), phase)))
        dead = !__all_sync(kFull, mbar_wait(full(warp, stage), phase, p.wait_ns));
      if (dead) continue;
      const unsigned char* keys = smem + stage_at(warp, stage) + C::kTileCodes;
      const unsigned char* pairs = smem + pairs_at(warp, stage);
      const int t0 = (at.s.first + k - at.base) * kU4Tile;
      const bool edge = t0 < full_from || t0 + kU4Tile > full_to;
#pragma unroll(NT == 4 ? 1 : 4)
      for (int sub = 0; sub < 4 / C::kMt; ++sub) {
        const int tok0 = 16 * C::kMt * sub + r;  // a lane's tokens: tok0 + 16 mt + 8 h
        // ---- S^T: [tile of 16 tokens][n tile], rows r, r + 8
        float2 s[C::kMt][NT][2];
        // (a step of every tile after the other: the products of a tile wait for each other)
        uint32_t kw[C::kMt][2][D / 32];
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned char* src = keys + (tok0 + 16 * mt + 8 * h) * C::kCode + c * (D / 8);
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              kw[mt][h][0] = v.x, kw[mt][h][1] = v.y, kw[mt][h][2] = v.z, kw[mt][h][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              kw[mt][h][0] = v.x, kw[mt][h][1] = v.y;
            }
          }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t a[C::kMt][2][2], b[C::kMt][2][2];  // [k16 step][row]
#pragma unroll
          for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) split_codes(kw[mt][h][w], a[mt][0][h], b[mt][0][h], a[mt][1][h], b[mt][1][h]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ks = 2 * w + i;
            uint32_t qv[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if constexpr (C::kQreg) {
                qv[n][0] = qf[n][ks][0], qv[n][1] = qf[n][ks][1];
              } else if (n % 2 == 0) {
                const uint4 v = *reinterpret_cast<const uint4*>(smem + C::kQ + ((ks * (NT / 2) + n / 2) * 32 + lane) * 16);
                qv[n][0] = v.x, qv[n][1] = v.y, qv[n + 1][0] = v.z, qv[n + 1][1] = v.w;
              }
            }
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (ks == 0)
                  mma_f16_first(s[mt][n], a[mt][i][0], a[mt][i][1], b[mt][i][0], b[mt][i][1], qv[n][0], qv[n][1]);
                else
                  mma_f16(s[mt][n], a[mt][i][0], a[mt][i][1], b[mt][i][0], b[mt][i][1], qv[n][0], qv[n][1]);
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
              float2 qn, fn;
              if constexpr (C::kQreg) {
                qn = qs[n], fn = f[n];
              } else {
                const float4 v = reinterpret_cast<const float4*>(smem + C::kQsum)[4 * n + c];
                qn = make_float2(v.x, v.z), fn = make_float2(v.y, v.w);
              }
              float2& x = s[mt][n][h];
              x.x = fmaf(x.x, ks * fn.x, fmaf(km, qn.x, ref[n].x));
              x.y = fmaf(x.y, ks * fn.y, fmaf(km, qn.y, ref[n].y));
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
        float vs[C::kMt][2], smost = 0.f, mmost = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt) {
          vs[mt][0] = u4_scale(vp[mt][0]), vs[mt][1] = u4_scale(vp[mt][1]);
          smost = max3(smost, fabsf(vs[mt][0]), fabsf(vs[mt][1]));
          mmost = max3(mmost, fabsf(u4_min(vp[mt][0])), fabsf(u4_min(vp[mt][1])));
        }
        // log2 of the size of the lane's largest row: with its largest score a bound on what the reference follows
        const float size = __uint_as_float(0x4b000000u | __float_as_uint(fmaxf(smost, 0.0625f * mmost)) >> 23) - size_from;
        const float limit = over - fmaxf(size, kLeast);
        float2 most[NT];
        bool moves = size > kMost;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          most[n] = make_float2(fmaxf(s[0][n][0].x, s[0][n][1].x), fmaxf(s[0][n][0].y, s[0][n][1].y));
#pragma unroll
          for (int mt = 1; mt < C::kMt; ++mt) {
            most[n].x = max3(most[n].x, s[mt][n][0].x, s[mt][n][1].x);
            most[n].y = max3(most[n].y, s[mt][n][0].y, s[mt][n][1].y);
          }
          moves |= fmaxf(most[n].x, most[n].y) > limit;
        }
        if (__any_sync(kFull, moves)) {
          float rel[C::kMt][2], big = kNothing;  // log2 of the rows' sizes
#pragma unroll
          for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t e = __float_as_uint(fmaxf(fabsf(vs[mt][h]), 0.0625f * fabsf(u4_min(vp[mt][h])))) >> 23;
              rel[mt][h] = e == 0 || e == 255 ? kNothing : static_cast<float>(static_cast<int>(e) - 126);
              big = fmaxf(big, rel[mt][h]);
            }
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, off));
          float e1 = 0.f, down = 1.f;
          if (size_from != 0.f || big != kNothing) {
            if (size_from == 0.f) {  // the first rows that are not 0
              e1 = big < kLeast + 10.f || big > kMost - 6.f ? fmaxf(big, -110.f) : 0.f;
            } else {
              const float e0 = size_from - kSizeFrom;
              e1 = fmaxf(e0, big - kMost);
              down = pow2(max(static_cast<int>(e0 - e1), -126));
            }
            size_from = kSizeFrom + e1;
            vf = pow2(kBoost - static_cast<int>(e1));
          }
#pragma unroll
          for (int mt = 0; mt < C::kMt; ++mt) rel[mt][0] = fmaxf(rel[mt][0] - e1, kLeast), rel[mt][1] = fmaxf(rel[mt][1] - e1, kLeast);
          bool all = true;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float2 m = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                m.x = fmaxf(m.x, s[mt][n][h].x + rel[mt][h]);
                m.y = fmaxf(m.y, s[mt][n][h].y + rel[mt][h]);
              }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              m.x = fmaxf(m.x, __shfl_xor_sync(kFull, m.x, off));
              m.y = fmaxf(m.y, __shfl_xor_sync(kFull, m.y, off));
            }
            // the reference goes up by m where that is above 0, or there was none (and m is a score)
            const bool none_x = none(ref[n].x), none_y = none(ref[n].y);
            const float2 up = make_float2(none_x ? (m.x == -INFINITY ? 0.f : m.x) : fmaxf(m.x, 0.f),
                                          none_y ? (m.y == -INFINITY ? 0.f : m.y) : fmaxf(m.y, 0.f));
            const float2 by = make_float2(none_x ? 0.f : fast_exp2(-up.x), none_y ? 0.f : fast_exp2(-up.y));
            const float2 scale = make_float2(by.x * down, by.y * down);
            // (0 - up: +0 for up = 0)
            if (!none_x || m.x != -INFINITY) ref[n].x = (none_x ? 0.f : ref[n].x) - up.x;
            if (!none_y || m.y != -INFINITY) ref[n].y = (none_y ? 0.f : ref[n].y) - up.y;
            all = all && !none(ref[n].x) && !none(ref[n].y);
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
          over = all ? kSlack : -INFINITY;
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
              const float2 w = make_float2(pr.x * v, pr.y * v);
              if constexpr (!kSumTc) csum[n][0] = add2(csum[n][0], w);
              pb[mt][n][h] = transpose8(pack_half2(w.x, w.y));
            }
          }
        // ---- O^T += V^T P^T: a transposed 8 x 8 matrix of 16-bit pieces holds four codes of a token in each half, tokens
        // 2 c, 2 c + 1, piece r of a 16-byte chunk
        const uint32_t ones = 0x3c003c00u;
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if constexpr (kSumTc) mma_f16(csum[n], ones, ones, ones, ones, pb[mt][n][0], pb[mt][n][1]);
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
      __syncwarp();  // the stage has been read; the last of a unit takes this warp's part first
      if (lane == 0 && !(C::kQreg && warp != merger && k + kWarps >= k1 && k1 < run)) mbar_arrive(empty(warp, stage));
      ++free_stages;
      if ((++consumed & 1) == 0) centre();
      if (consumed == tell_at) tell();
      if (++stage == STAGES) stage = 0, phase ^= 1;
    }
    if (C::kQreg && warp == 0 && !q_sent) {
      if (!dead) dead = !__all_sync(kFull, mbar_wait(q_read, seg & 1, p.wait_ns));
      if (!dead) send_next_q();
    }

    // ---------------------------------------------- the end of the unit
    // o in units of V, base_sum in it
    centre();
#pragma unroll
    for (int n = 0; n < NT; ++n)
      top[n] = make_float2(none(ref[n].x) ? -INFINITY : -ref[n].x, none(ref[n].y) ? -INFINITY : -ref[n].y);
    const float out0 = size_from == 0.f ? 0.f : pow2(static_cast<int>(size_from - kSizeFrom) - kBoost), out1 = 0x1p24f;
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
    if (k1 >= run) break;

    // ------------------------------------ a unit that ends inside the run
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
      // A warp leaves its part in the stage that it has read last and goes on with the next unit; the stage is empty when
      // the part has been taken. Warps without a tile of the unit have no part.
      const int later = (merger + 1) % kWarps;  // the others in the order of their tiles
      uint32_t leaving = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (w != merger && k1 - 1 - (merger - w + kWarps) % kWarps >= k0) leaving |= 1u << w;
      if (lane < kWarps) parts[lane] += leaving >> lane & 1;
      __syncwarp();
      auto ml_of = [&](int w, int st) {
        return smem + (NT == 1 ? stage_at(w, st) + C::kPart : C::kMl + (w * STAGES + st) * C::kPartMl);
      };
      if (warp == merger) {
        for (int i = 0; i < kWarps - 1; ++i) {
          const int w = (later + i) % kWarps;
          if (!(leaving >> w & 1)) continue;
          const uint32_t n = parts[w];
          if (!dead) dead = !__all_sync(kFull, wait_count(left_count + 4 * w, n, p.wait_ns));
          if (dead) continue;
          const int st = where[2 * w + (n & 1)];
          take(smem + stage_at(w, st), ml_of(w, st));
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(w, st));
        }
      } else if ((leaving >> warp & 1) && !dead) {
        const int st = stage == 0 ? STAGES - 1 : stage - 1;  // the one read last
        ++own_parts;
        leave(smem + stage_at(warp, st), ml_of(warp, st));
        if (lane == 0) where[2 * warp + (own_parts & 1)] = st;
        __syncwarp();
        if (lane == 0) publish(left_count + 4 * warp, own_parts);
      }
    } else {
      // The four warps' parts meet in a chain, warp 3's into warp 2's registers and so on, through one place. A warp that
      // has left its part goes on with the next unit.
      if (warp == kWarps - 1) {
        if (seg > 0 && !dead) dead = !__all_sync(kFull, mbar_wait(chain_free, (seg - 1) & 1, p.wait_ns));
      } else {
        if (!dead) dead = !__all_sync(kFull, mbar_wait(chain + 8 * (warp + 1), seg & 1, p.wait_ns));
        take(smem + C::kMerge, smem + C::kMl);
      }
      if (warp != 0) leave(smem + C::kMerge, smem + C::kMl);
      __syncwarp();
      if (lane == 0) mbar_arrive(warp == 0 ? chain_free : chain + 8 * warp);
    }
    if (warp == merger) {
      if (at.base < 0) {  // other blocks have parts of it
        const long long first = (start + at.base) / run_len, last = me;
        float* mine = p.part + 2 * me * static_cast<long long>(C::kRows * (D + 2));
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
        if (lane == 0) flag[0] = 1 + warp, flag[1] = at.b, flag[2] = at.u, flag[3] = static_cast<int>(first), flag[4] = static_cast<int>(last);
        __syncwarp();
        tell_at = consumed + 2;
      } else {
        write_rows(p, at.b, j, row0, top, sum, o, 0);
      }
    }
    at.next(p, units);
    if constexpr (!C::kQreg) {
      float4 q4[D / 16];
      const float4* src = reinterpret_cast<const float4*>(q_row(at, warp));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) q4[i] = src != nullptr ? src[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      share_q(q4);
    }
  }

  // ------------------------------------------------ the end of the run
  // Every warp leaves its part of the last unit in its ring; then each of four has a quarter of the dims, of all parts.
  constexpr int kQuarter = C::kM / 4;
  const bool joins = warp < 4;
  float2 acc[NT][kQuarter][2];
  auto clear = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n] = make_float2(-INFINITY, -INFINITY);
      sum[n] = zero2;
#pragma unroll
      for (int i = 0; i < kQuarter; ++i) acc[n][i][0] = acc[n][i][1] = zero2;
    }
  };
  auto add_part = [&](int n, float2 m2, float2 s2, const float4 (&v)[kQuarter]) {
    float2 wa, wb;
    weights(top[n], m2, wa, wb);
    sum[n] = fma2(sum[n], wa, mul2(s2, wb));
#pragma unroll
    for (int i = 0; i < kQuarter; ++i) {
      acc[n][i][0] = fma2(acc[n][i][0], wa, mul2(make_float2(v[i].x, v[i].y), wb));
      acc[n][i][1] = fma2(acc[n][i][1], wa, mul2(make_float2(v[i].z, v[i].w), wb));
    }
  };
  const int own_stage = C::kQreg ? (stage == 0 ? STAGES - 1 : stage - 1) : 0;  // (NT = 4: the whole ring)
  const int reads = (consumed + STAGES - 1 - own_stage) / STAGES;                // of that stage
  if (C::kQreg && reads > 0 && !dead)  // (it may hold the part of a unit before)
    dead = !__all_sync(kFull, mbar_wait(empty(warp, own_stage), (reads - 1) & 1, p.wait_ns));
  float4* own = reinterpret_cast<float4*>(smem + stage_at(warp, own_stage));
  float2* own_ml = reinterpret_cast<float2*>(smem + C::kEnd + warp * C::kEndStep);
  volatile int* end_stage = flag + 10 + kWarps * (3 + kWarps);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    own_ml[n * 32 + lane] = top[n];
    own_ml[(NT + n) * 32 + lane] = sum[n];
#pragma unroll
    for (int i = 0; i < C::kM; ++i) own[(n * C::kM + i) * 32 + lane] = make_float4(o[n][i][0].x, o[n][i][0].y, o[n][i][1].x, o[n][i][1].y);
  }
  if (lane == 0) end_stage[warp] = own_stage;
  __syncthreads();
  clear();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (!joins) break;
    const float4* src = reinterpret_cast<const float4*>(smem + stage_at(w, end_stage[w]));
    const float2* ml = reinterpret_cast<const float2*>(smem + C::kEnd + w * C::kEndStep);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float4 v[kQuarter];
#pragma unroll
      for (int i = 0; i < kQuarter; ++i) v[i] = src[(n * C::kM + warp * kQuarter + i) * 32 + lane];
      add_part(n, ml[n * 32 + lane], ml[(NT + n) * 32 + lane], v);
    }
  }
  if (p.whole || (at.base >= 0 && at.end() == run)) {
    if (joins) write_rows(p, at.b, j, row0, top, sum, acc, warp * kQuarter);
  } else {
    // Other blocks have parts of the unit: this one's is written, and the last block to say so merges them, in the order
    // of the blocks. The place of a unit that the block did not begin is the first of its two.
    const int first = static_cast<int>((start + at.base) / run_len), last = static_cast<int>((start + at.end() - 1) / run_len);
    float* mine = p.part + (2 * me + (at.base < 0 ? 0 : 1)) * static_cast<long long>(C::kRows * (D + 2));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (!joins) break;
#pragma unroll
      for (int i = 0; i < kQuarter; ++i)
        reinterpret_cast<float4*>(mine)[(n * C::kM + warp * kQuarter + i) * 32 + lane] =
            make_float4(acc[n][i][0].x, acc[n][i][0].y, acc[n][i][1].x, acc[n][i][1].y);
      if (warp == 0 && r == 0) {
        *reinterpret_cast<float2*>(mine + C::kRows * D + 8 * n + 2 * c) = top[n];
        *reinterpret_cast<float2*>(mine + C::kRows * (D + 1) + 8 * n + 2 * c) = sum[n];
      }
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      flag[5] = atomicAdd(p.arrived + first, 1) == last - first ? -1 : 0;
      flag[6] = at.b, flag[7] = at.u, flag[8] = first, flag[9] = last;
      __threadfence();
    }
  }
  if (!p.whole) {
    tell();
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
      volatile int* todo = flag + 5 * which;
      if (todo[0] >= 0 || !joins) continue;
      const int u = todo[2], from_block = todo[3], to_block = todo[4], ju = u / p.row_blocks;
      constexpr int kAhead = NT == 1 ? 4 : 2;  // parts whose loads are issued together
      clear();
      for (int b0 = from_block; b0 <= to_block; b0 += kAhead) {
        float2 m2[kAhead][NT], s2[kAhead][NT];
        float4 v[kAhead][NT][kQuarter];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int b = min(b0 + a, to_block);
          const float* src = p.part + (2 * b + (b == from_block ? 1 : 0)) * static_cast<long long>(C::kRows * (D + 2));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            m2[a][n] = __ldcg(reinterpret_cast<const float2*>(src + C::kRows * D + 8 * n + 2 * c));
            s2[a][n] = __ldcg(reinterpret_cast<const float2*>(src + C::kRows * (D + 1) + 8 * n + 2 * c));
#pragma unroll
            for (int i = 0; i < kQuarter; ++i)
              v[a][n][i] = __ldcg(reinterpret_cast<const float4*>(src) + (n * C::kM + warp * kQuarter + i) * 32 + lane);
          }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (b0 + a > to_block) break;
#pragma unroll
          for (int n = 0; n < NT; ++n) add_part(n, m2[a][n], s2[a][n], v[a][n]);
        }
      }
      write_rows(p, todo[1], ju, (u - ju * p.row_blocks) * C::kRows, top, sum, acc, warp * kQuarter);
    }
  }
  if (dead) {  // the copies under way land before the block ends
    if (lane == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_TIMEOUT));
    if (C::kQreg && warp == 0) mbar_wait(q_come, (q_count - 1) & 1, kWaitLimitNs);
    for (; consumed < issued; ++consumed) {
      mbar_wait(full(warp, stage), phase, kWaitLimitNs);
      if (++stage == STAGES) stage = 0, phase ^= 1;
    }
  }
}

__global__ void u4_clear_kernel(int32_t* arrived, int count) {
  grid_dependents_launch();
  for (int i = threadIdx.x; i < count; i += blockDim.x) arrived[i] = 0;
}

template <int D, int NT, bool PAGED, int STAGES, int CTAS, int WARPS>
cudaError_t launch_u4_t(const U4Params& p, const CUtensorMap& tmap_v, int ctas, bool clear, cudaStream_t stream) {
  using C = Cfg<D, NT, STAGES, WARPS>;
  const auto kernel = attn_u4_kernel<D, NT, PAGED, STAGES, CTAS, WARPS>;
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
  cfg.blockDim = dim3(32 * WARPS);
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
  if (p.rows <= 8) {
    // A unit a block, two blocks an SM at most: six warps a block (256 units of 64 tiles 34.5 us with four, 32.4 with six, of
    // 256 tiles 119 and 106; 456 units, which four warps take three blocks an SM of, 45 and 55).
    if (p.whole && static_cast<long long>(p.batch) * p.h_kv <= ctas / kCtas1 * 2)
      return launch_u4_t<D, 1, PAGED, kStages, 2, 6>(p, tv, ctas, clear, stream);
    return launch_u4_t<D, 1, PAGED, kStages, kCtas1, 4>(p, tv, ctas, clear, stream);
  }
  if (p.rows <= 16) return launch_u4_t<D, 2, PAGED, kStages, kCtas2, 4>(p, tv, ctas, clear, stream);
  return launch_u4_t<D, 4, PAGED, kStages, kCtas4, 4>(p, tv, ctas, clear, stream);
}

}  // namespace

U4Shape u4_shape(int rows) {
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
