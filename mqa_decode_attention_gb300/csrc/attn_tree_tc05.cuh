// Attention of a tree of drafted tokens over the cache on the 5th-generation
// tensor cores: head_dim 128, groups of up to 128 heads, every cache the
// tensor cores read (bf16, uint8, fp8 e5m2; contiguous or paged).
//
// One persistent block per SM streams an equal run of the key tiles (tree.cuh)
// and never lets its ring of K / V tiles run dry between two units: the
// loader warp goes straight on to the next unit's tiles while the softmax
// warps finish the last one's rows. For each 128-key tile
//   S = Q K^T      tcgen05.mma M=128 N=128 K=128, both operands bf16 in shared
//                  memory, S (f32) into tensor memory
//   softmax        one row per thread: running maximum and sum
//                  (FlashAttention, "Arsitektur Inferensi LLM", section 5), O
//                  rescaled only when a row's maximum grows by more than 2^8;
//                  P (two bf16 terms) written over its S columns
//   O += P V       tcgen05.mma with A = P from tensor memory
// Rows are (node i, query head) pairs of one kv head, whole nodes to a block.
// There are two accumulators (S and O of each in tensor memory, 512 columns)
// with a softmax warpgroup each:
//   NT = 2  (more than 128 rows per kv head) two query tiles of up to 128 rows
//           share every K / V tile; the tensor cores alternate between them.
//           One tile of K and V asks for 1.45 us of HBM and 2.0 us of products
//           (1.35 with P in one term) at an SM's share of 6.8 TB/s and of 1.89
//           PFLOP/s, and takes 2.8: what bounds it is each accumulator's chain
//           product - softmax - product (32 x 64 nodes on 4096 keys, 32 + 8 heads,
//           573 MB: a step 167 us, 178 on inputs that change, 0.8 PFLOP/s without
//           the second terms). A tree that ends in a block of up to 128 rows has
//           that block done as below.
//   NT = 1  (up to 128 rows) both accumulators hold the same rows and take the
//           tiles in turn, so that one's softmax runs beside the other's
//           products; their results meet in shared memory at a unit's end.
//           Bound by the HBM stream: a tile of K and V (64 KB) takes 1.45 us
//           of an SM's share of 6.8 TB/s, its products 1.0 us (128 rows, P in two
//           terms) (a step of 32 x 16 nodes on 4096 keys, 549 MB: 102 us, 5.4 TB/s;
//           of 4 x 32 nodes on 131040 keys, 2.15 GB: 328 us, 6.6 TB/s, 356 on inputs
//           that change).
//
// Q is loaded by TMA as the append left it (bf16, not scaled): the scale
// times log2 e goes into the exponent's fused multiply-add. A second bf16 term of
// Q has no room in shared memory beside two row tiles. P over bf16 and uint8
// caches enters as two bf16 terms (split_p, within 2^-15; the two take the columns
// that S had): with one term (2^-8) the output's error against 64 bits is 1.7 times
// that of its own rounding to bf16 for a step, with two 1.4 times, which Q's
// rounding leaves; on given bf16 queries over uint8 1.4 and 1.0 times. The price:
// bf16, 32 x 64 nodes 146 -> 169 us, 32 x 16 nodes 101 -> 103 us; uint8 227 -> 252
// and 117 -> 128 us. Over e5m2 P has an f16's 2^-11. Sums, maxima and partial
// results are fp32.
//
// One-byte caches: the loader's tiles are codes (16 KB), eight converter warps
// widen each to a 16-bit tile, exactly. An e5m2 code is the high byte of an
// IEEE half: K and V become f16, and Q and P enter as f16 too: Q's rows are made
// f16 in shared memory, each scaled by a power of two of its own. A uint8 code
// minus its zero point is an integer up to 255 and becomes a bf16 (widen_u8);
// the rows' scales are put beside the tile: a K scale multiplies its column of
// S, a V scale its column of P, in fp32, before P is rounded.
// An f16 P is within 2^-11 of its value, or within 2^-25 when it is below 2^-14.
// It is taken times 2^kHalfShift, as are the sums l (and the maxima handed on
// less that): the row's largest P is then in [2^7, 2^15], below f16's 65504, and
// a key moves the result by 2^-32 of the largest |v| at most beside its 2^-11,
// 2^17 of them by 2^-15. (Without the factor keys below 2^-25 of the largest were
// lost to O but not to l: one key before 10^5 that weigh 2.5e-8 each took up to 0.26%
// of the result, a third of a bf16 step.)
// (A step of 64 x 8 nodes of 32 heads on 8192 e5m2 keys of one kv head: 92 us, 0.75
// PFLOP/s; bound by the widening and the chains.)
//
// Keys that no node may read (past the sequence, before the window) have zero
// V rows whatever the cache holds, so that 0 * NaN never enters a sum.
//
// Warps: 0-3 and 4-7 softmax, 8 K / V loader (TMA), 9 MMA issue (converged, one
// elected lane) and tensor-memory allocation, 10 Q loader (TMA), 11 gives warps
// 0-7 and 9 their segments and counts in the first unit's partial result; 12-19
// converters. The loaders and converters walk the segments by themselves.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "tc05.cuh"
#include "tree.cuh"

namespace mqa {
namespace {

constexpr int kD = 128;
constexpr int kBM = 128;  // rows of an accumulator
constexpr int kBN = 128;  // keys per tile
constexpr int kTileBytes = kBN * kD * 2;  // a bf16 tile, 128-byte swizzled
// A bf16 tile is [2 halves of 64 dims][128 rows][128 B]; gathered from pages it
// is [16 groups of 8 rows][2 halves][8 rows][128 B], so that one copy brings a
// page's rows with both halves (a copy per page and half kept the TMA unit
// busy: 16-row pages 4.7 TB/s). Strides of the halves and of the 8-row groups:
template <bool GROUPED>
struct Tile {
  static constexpr int kHalf = GROUPED ? 1024 : 16384;
  static constexpr int kGroup = GROUPED ? 2048 : 1024;
};
template <bool GROUPED>
__device__ __forceinline__ int tile_row(int r) {  // byte offset of row r's first half
  return (r >> 3) * Tile<GROUPED>::kGroup + (r & 7) * 128;
}
constexpr int kRawBytes = kBN * kD;       // a code tile: [128 rows][128 B], swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // S / P of accumulator q at 128 q, its O at 256 + 128 q
constexpr float kRescaleLog2 = 8.0f;
constexpr float kHalfShift = 7.0f;  // P as f16: kRescaleLog2 + this < 16

// What the warps of a block share beside the tiles and barriers.
struct TreeMisc {
  TreePlan plan;
  // the segments, out of the softmax and MMA warps' registers (two places: one
  // may still be read while the next is written), and the first one
  TreeSegment seg[2], first;
  int abort, flag, pending, more[2], last[2];
  // what the two accumulators' threads of a row hand over: maxima [0] and sums
  // [1]; at a segment's start (e5m2) [0] the row's score factor
  float row[2][128];
};

// Registers: setmaxnreg moves them from the loader, MMA and converter warps
// to the softmax warps; the shares add up to no more than the block is launched
// with.
template <int NT, int DT>
struct Cfg {
  static constexpr bool kByte = DT != kDtypeBf16;
  static constexpr int kThreads = kByte ? 640 : 384;
  static constexpr int kRegsLaunch = kByte ? 96 : 168;
  static constexpr int kRegsSoftmax = kByte ? 152 : 200;
  static constexpr int kRegsAux = kByte ? (DT == kDtypeU8 ? 64 : 80) : 104;
  static constexpr int kRegsConvert = DT == kDtypeU8 ? 56 : 48;
  static_assert(256 * kRegsSoftmax + 128 * kRegsAux + (kThreads - 384) * kRegsConvert <= kThreads * kRegsLaunch,
                "register split");
  // 16-bit tiles, and code tiles
  static constexpr int kSlots = kByte ? 4 : (NT == 1 ? 6 : 5);
  static constexpr int kRaw = kByte ? (NT == 2 ? 2 : (DT == kDtypeU8 ? 3 : 4)) : 0;
  static_assert(NT == 1 || DT != kDtypeU8, "no room for two row tiles beside the scales");
  static constexpr bool kHalf = DT == kDtypeF8;  // f16 operands (else bf16)
  static constexpr bool kSplitP = !kHalf;  // P as two bf16 terms: [16 columns][16 columns] of each 32 keys
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = NT * kTileBytes;
  static constexpr int kRawOff = kRingOff + kSlots * kTileBytes;
  // uint8: the scales of each bf16 tile's rows, twice as many places as tiles:
  // a K tile is given back when its S is there, but its scales are read by
  // the softmax after that. Load u + 2 kSlots (four tiles on) only lands after
  // S of two tiles on, which is issued after the softmax of u's tile.
  static constexpr int kScaleOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kScales = 2 * kSlots;
  static constexpr int kBarOff = kScaleOff + (DT == kDtypeU8 ? kScales * kBN * 4 : 0);
  static constexpr int kMiscOff = kBarOff + 304;           // TreeMisc
  static constexpr int kSmemBytes = kMiscOff + static_cast<int>(sizeof(TreeMisc));
  // mbarriers
  static constexpr int kQFull = 0;
  static constexpr int kQFree = 1;                  // a segment of two row tiles is done with Q
  static constexpr int kXFree = 2;                  // one of one row tile: its accumulators have met
  static constexpr int kQReady = 3;                 // [2] e5m2: Q's row tile is f16
  static constexpr int kFull = 5;                   // [kSlots]
  static constexpr int kEmpty = kFull + kSlots;     // [kSlots]
  static constexpr int kRFull = kEmpty + kSlots;    // [kRaw]
  static constexpr int kREmpty = kRFull + kRaw;     // [kRaw]
  static constexpr int kSFull = kREmpty + kRaw;     // [2]
  static constexpr int kP = kSFull + 2;             // [2] keys 0-63 of P written
  static constexpr int kPHi = kP + 2;               // [2] keys 64-127
  static constexpr int kODone = kPHi + 2;
  static constexpr int kOFree = kODone + 1;
  static constexpr int kPart = kOFree + 1;  // a partial result is written
  // [2] a segment is in place 0 / 1; the softmax warps are done with it. (A
  // barrier for each place: none can be two phases ahead of a warp that waits.)
  static constexpr int kSeg = kPart + 1;
  static constexpr int kSegFree = kSeg + 2;
  static constexpr int kDrain = kSegFree + 2;
  static constexpr int kNBars = kDrain + 1;
  static_assert(kNBars * 8 + 4 <= 304, "barrier area");
  static_assert(kMiscOff % 16 == 0 && kSmemBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  float2 r;
  asm("{\n\t.reg .b64 ra, rb, rc, rr;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %4};\n\t"
      "mov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rr, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rr;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 ra, rb, rr;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rr, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rr;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 ra, rb, rr;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rr, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rr;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Four e5m2 codes as two f16 pairs: a code is the high byte of an IEEE half.
__device__ __forceinline__ uint2 half_e5m2(uint32_t w) {
  return make_uint2(__byte_perm(w, 0u, 0x1404), __byte_perm(w, 0u, 0x3424));
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack_p(float2 v) {
  if constexpr (HALF) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(v.x, v.y);
  }
}

// Row r of a bf16 Q tile in place as f16, times the power of two that brings its
// largest magnitude to [2^9, 2^10), which is returned (1 for a row of zeros or
// with an infinity or NaN).
__device__ __forceinline__ float half_row(unsigned char* tile, int r) {
  uint32_t top = 0;  // the largest magnitudes' bit patterns, which order as the values do
  auto chunk = [&](int x) { return reinterpret_cast<uint4*>(tile + (x >> 3) * 16384 + r * 128 + (((x & 7) ^ (r & 7)) << 4)); };
#pragma unroll 4
  for (int x = 0; x < 16; ++x) {
    const uint4 w = *chunk(x);
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
  }
  const uint32_t m = max(top & 0xffffu, top >> 16);  // bf16 bits
  const int e = static_cast<int>(m >> 7);            // biased exponent
  // 2^(9 - (e - 127)); the smallest rows stop at 2^126
  const float f = m == 0 || e == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(min(127 + 9 + 127 - e, 253)) << 23);
#pragma unroll 4
  for (int x = 0; x < 16; ++x) {
    uint4 w = *chunk(x);
    uint32_t* v = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(bf16lo_to_f32(v[i]) * f, bf16hi_to_f32(v[i]) * f);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *chunk(x) = w;
  }
  return f;
}

// Groups of products issued by one elected lane of a converged warp (always the
// same one, as the commits). The warp's control flow is uniform, so that the
// descriptors can stay in uniform registers: issued by a lane inside a
// divergent branch, with the operands moved there one by one, a group of eight
// took as long to issue as to run.
// D = A B^T over 128 values of K: A and B K-major in shared memory, B's second
// 64 values BH descriptor units after the first.
template <int BH>
__device__ __forceinline__ void mma_128(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, z, o;\n\t.reg .b64 x, y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 z, 0, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, z;\n\t"
      "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, 1024;\n\tadd.s64 y, %2, %4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, 1026;\n\tadd.s64 y, %2, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, 1028;\n\tadd.s64 y, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, 1030;\n\tadd.s64 y, %2, %7;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(BH), "n"(BH + 2), "n"(BH + 4), "n"(BH + 6)
      : "memory");
}
// D (+)= A B over 64 values of K (keys): A in tensor memory, 8 columns for 16
// keys (the second 32 keys AK columns after the first), B MN-major in shared
// memory, 16 keys BK descriptor units apart.
template <int BK, int AK>
__device__ __forceinline__ void mma_64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred e, z, o;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 z, %4, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, z;\n\t"
      "add.s32 x, %1, 8;\n\tadd.s64 y, %2, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %8;\n\tadd.s64 y, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %9;\n\tadd.s64 y, %2, %7;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "n"(BK), "n"(2 * BK), "n"(3 * BK), "n"(AK),
      "n"(AK + 8)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint32_t mbar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(mbar)
      : "memory");
}

// Four lanes (an aligned group) hold four pieces of four words each: lane i's
// piece j goes to lane j's place i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[16], int lane) {
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & s) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t &a = w[4 * i + e], &b = w[4 * (i | s) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, s);
        if (up)
          a = got;
        else
          b = got;
      }
    }
  }
}

template <int NT, bool PG, int DT>
__global__ void __launch_bounds__(Cfg<NT, DT>::kThreads, 1)
    attn_tree_tc05_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ CUtensorMap tmap_q, const TreeParams p) {
  using C = Cfg<NT, DT>;
  constexpr bool kByte = C::kByte;
  constexpr bool kGrouped = PG && !kByte;
  using L = Tile<kGrouped>;
  constexpr int kSlots = C::kSlots;
  extern __shared__ __align__(1024) unsigned char smem[];  // (no static part: every byte is needed)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + C::kNBars * 8);
  TreeMisc& sh = *reinterpret_cast<TreeMisc*>(smem + C::kMiscOff);
  TreePlan& plan = sh.plan;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, acc_rows = p.tokens_per_tile * G, rows_per_block = NT * acc_rows;

  if (!p.early) grid_dependency_wait();
  if (smem_u32(smem) & 1023u) {  // tiles and descriptors need the alignment that the declaration asks for
    if (tid == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_TIMEOUT));
    return;
  }
  if (tid == 0) {
    // (whatever the error word holds: an earlier call's bits are no reason to leave
    // this call's work undone, and this call's blocks are all resident at once)
    sh.abort = 0;
    mbar_init(bar(C::kQFull), 1);
    mbar_init(bar(C::kQFree), 1);
    mbar_init(bar(C::kXFree), 8);
    mbar_init(bar(C::kQReady + 0), 4);
    mbar_init(bar(C::kQReady + 1), 4);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(C::kFull + s), kByte ? 8 : 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    if constexpr (kByte) {
      for (int s = 0; s < C::kRaw; ++s) {
        mbar_init(bar(C::kRFull + s), 1);
        mbar_init(bar(C::kREmpty + s), 8);
      }
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(bar(C::kSFull + q), 1);
      mbar_init(bar(C::kP + q), 4);
      mbar_init(bar(C::kPHi + q), 4);
    }
    mbar_init(bar(C::kODone), 1);
    mbar_init(bar(C::kOFree), 8);
    mbar_init(bar(C::kPart), 8);
    mbar_init(bar(C::kSeg + 0), 1);
    mbar_init(bar(C::kSeg + 1), 1);
    mbar_init(bar(C::kSegFree + 0), 8);
    mbar_init(bar(C::kSegFree + 1), 8);
    mbar_init(bar(C::kDrain), 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tc05::tmem_alloc(smem_u32(tslot), kTmemCols);
    tc05::tmem_relinquish();
  }
  if (warp == 8) tree_plan(p, kBN, rows_per_block, blockIdx.x, gridDim.x, &plan);
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tslot);
  const uint32_t sbase = smem_u32(smem);

  auto fail = [&](bool one) {
    if (one) {
      sh.abort = 1;
      atomicOr(p.err, static_cast<int>(MQA_DEVERR_TIMEOUT));
    }
  };
  // whether a segment's rows need both accumulators (else both hold them all)
  auto is_two = [&](const TreeSegment& g) { return NT == 2 && g.s.nodes * G - g.rb * rows_per_block > acc_rows; };
  auto stop = [&]() { return *reinterpret_cast<volatile int*>(&sh.abort) != 0; };
  auto regs_aux = [&]() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsAux)); };
  auto begin = [&]() {
    TreeWalk w;
    w.start(plan);
    return w;
  };

  if (warp == 8) {
    regs_aux();
    // -------------------------------------------------------- K / V loader
    // load u (2 t + 0 / 1: K / V of the run's tile t) into slot u % slots: the
    // bf16 tile itself, or the code tile a converter widens
    constexpr int kN = kByte ? C::kRaw : kSlots;
    constexpr int kBytes = kByte ? kRawBytes : kTileBytes;
    constexpr int kRing = kByte ? C::kRawOff : C::kRingOff;
    constexpr int kF = kByte ? C::kRFull : C::kFull, kE = kByte ? C::kREmpty : C::kEmpty;
    const int ps = PG ? p.page_size : 64, rp = ps < 64 ? ps : 64, copies = kBN / rp;
    TreeWalk walk = begin();
    TreeSegment g;
    bool waited = !p.early, ok = true, bad = false;
    int u = 0;
    while (ok && walk.next(p, kBN, rows_per_block, g)) {
      const int row = g.b * p.h_kv + g.j;
      const int key_first = g.s.first + g.t0 * kBN;
      // paged: the page ids of the segment's keys, 32 at a time, one per lane
      // (wcur: pages wbase .., wnxt: the next 32). Entries of pages that hold
      // no key to be read are not looked at; a copy there lands zeros (page -1)
      const int32_t* trow = PG ? p.block_table + static_cast<long long>(g.b) * p.max_pages : nullptr;
      const int lp_first = g.s.lo / ps, lp_end = (g.s.len + ps - 1) / ps;
      auto entry = [&](int lp) { return (PG && lp >= lp_first && lp < lp_end) ? __ldg(trow + lp) : -1; };
      int wbase = key_first / ps;
      int wcur = entry(wbase + lane), wnxt = entry(wbase + 32 + lane);
      for (int t = 0; t < g.nt && ok; ++t) {
        const int key0 = key_first + t * kBN;
        if (!waited && key0 + kBN > g.s.pos) {  // this tile holds a node's row, which the append writes
          grid_dependency_wait();
          waited = true;
        }
        for (int kv = 0; kv < 2; ++kv, ++u) {
          const int slot = u % kN, lap = u / kN;
          if (lane == 0) {
            if (lap > 0) ok = mbar_wait(bar(kE + slot), (lap - 1) & 1, p.wait_ns);
            if (!ok) fail(true);
            if (stop()) ok = false;
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          const CUtensorMap* map = kv ? &tmap_v : &tmap_k;
          const uint32_t dst = sbase + kRing + slot * kBytes;
          if constexpr (PG) {
            while (key0 / ps - wbase >= 32) {
              wcur = wnxt;
              wbase += 32;
              wnxt = entry(wbase + 32 + lane);
            }
            const int k = key0 + lane * rp, lp = k / ps, off = lp - wbase;  // off < 32 + 8
            const int pc = __shfl_sync(0xffffffffu, wcur, off & 31), pn = __shfl_sync(0xffffffffu, wnxt, off & 31);
            int page = off < 32 ? pc : pn;
            const bool needed = lane < copies && lp >= lp_first && lp < lp_end;
            if (needed && (page < 0 || page >= p.num_pages)) bad = true;
            if (!needed || page < 0 || page >= p.num_pages) page = -1;
            if (lane == 0) mbar_arrive_expect_tx(bar(kF + slot), kBytes);
            __syncwarp();
            if (lane < copies) {
              const uint32_t d = dst + lane * rp * (kByte ? 128 : 256);
              if constexpr (kByte) {
                tma_load_4d(d, map, 0, k & (ps - 1), g.j, page, bar(kF + slot));
              } else {
                tma_load_5d(d, map, 0, 0, 0, (k & (ps - 1)) >> 3, page < 0 ? -1 : page * p.h_kv + g.j, bar(kF + slot));
              }
            }
          } else if (lane == 0) {
            mbar_arrive_expect_tx(bar(kF + slot), kBytes);
            if constexpr (kByte)
              tma_load_3d(dst, map, 0, key0, row, bar(kF + slot));
            else
              tma_load_4d(dst, map, 0, key0, 0, row, bar(kF + slot));
          }
        }
      }
    }
    if (PG && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_PAGE_RANGE));
    // every copy this warp issued (u of them) lands before the block can exit
    if (lane == 0)
      for (int k = u > kN ? u - kN : 0; k < u; ++k) (void)mbar_wait(bar(kF + k % kN), (k / kN) & 1, kWaitLimitNs);
    __syncwarp();
  } else if (warp == 10) {
    regs_aux();
    // ------------------------------------------------------------ Q loader
    if (lane == 0) {
      if (p.early) grid_dependency_wait();
      TreeWalk walk = begin();
      TreeSegment g;
      bool ok = true, last_two = false;
      int seg = 0, n_two = 0;
      while (ok && walk.next(p, kBN, rows_per_block, g)) {
        // the Q area is free when the last segment's products with Q are done
        // or, with one row tile, when its accumulators have met there (a
        // barrier for each kind: every phase of it is waited for, so that a
        // parity never stands for an older phase)
        auto poll = [&](int id, int parity) {  // (a suspended wait wakes late, and the next S waits for it)
          const unsigned long long t0 = global_timer_ns();
          while (!mbar_test(bar(id), parity & 1))
            if (stop() || global_timer_ns() - t0 > p.wait_ns) return false;
          return true;
        };
        if (seg > 0) ok = last_two ? poll(C::kQFree, n_two - 1) : poll(C::kXFree, seg - n_two - 1);
        if (!ok) fail(true);
        if (!ok || stop()) break;
        last_two = is_two(g);
        n_two += last_two;
        const int tiles = last_two ? 2 : 1;
        // (tokens past the sequence's belong to the next: rows nobody uses)
        mbar_arrive_expect_tx(bar(C::kQFull), tiles * acc_rows * kD * 2);
        for (int q = 0; q < tiles; ++q)
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sbase + C::kQOff + q * kTileBytes + h * 16384, &tmap_q, 64 * h, g.j * G,
                        g.b * p.n + (g.rb * NT + q) * p.tokens_per_tile, bar(C::kQFull));
        ++seg;
      }
      if (seg > 0) (void)mbar_wait(bar(C::kQFull), (seg - 1) & 1, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 9) {
    regs_aux();
    // ----------------------------------------------------------- MMA issue
    // (the whole warp, converged; one elected lane issues)
    {
      constexpr uint32_t id_s = C::kHalf ? tc05::idesc_f16_f32(kBM, kBN, false, false)
                                           : tc05::idesc_bf16_f32(kBM, kBN, false, false);
      constexpr uint32_t id_o = C::kHalf ? tc05::idesc_f16_f32(kBM, kD, false, true)
                                           : tc05::idesc_bf16_f32(kBM, kD, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sb = __shfl_sync(0xffffffffu, sbase, 0);
      auto wait = [&](int id, int parity) {  // polls: a suspended wait wakes late
        if (__all_sync(0xffffffffu, mbar_test(bar(id), parity & 1))) return true;
        const unsigned long long t0 = global_timer_ns();
        while (!__all_sync(0xffffffffu, mbar_test(bar(id), parity & 1)))
          if (__any_sync(0xffffffffu, stop() || global_timer_ns() - t0 > p.wait_ns)) return false;
        return true;
      };
      int u0 = 0;            // the segment's first load
      int ps[2] = {0, 0};    // products P V issued into each accumulator
      auto full = [&](int u) { return wait(C::kFull + u % kSlots, u / kSlots); };
      auto issue_s = [&](int q, int t, int qt) {  // S_q = Q K(t)^T, Q's row tile qt
        tc05::fence_after_sync();
        mma_128<L::kHalf / 16>(tm + kColS + q * 128, tc05::smem_desc_sw128(sb + C::kQOff + qt * kTileBytes, 16, 1024),
                               tc05::smem_desc_sw128(sb + C::kRingOff + ((u0 + 2 * t) % kSlots) * kTileBytes, 16, L::kGroup),
                               id_s);
        commit_elect(bar(C::kSFull + q));
      };
      // O_q (+)= P_q V(t) of keys 64 h .. 64 h + 63: each half of P as soon as it is written
      auto issue_pv = [&](int q, int t, int h, bool add) {
        tc05::fence_after_sync();
        const uint64_t v = tc05::smem_desc_sw128(
            sb + C::kRingOff + ((u0 + 2 * t + 1) % kSlots) * kTileBytes + h * 8 * L::kGroup, L::kHalf, L::kGroup);
        const uint32_t a = tm + kColS + q * 128 + h * (C::kSplitP ? 64 : 32);
        mma_64<2 * L::kGroup / 16, C::kSplitP ? 32 : 16>(tm + kColO + q * 128, a, v, id_o, add || h > 0);
        if constexpr (C::kSplitP) mma_64<2 * L::kGroup / 16, 32>(tm + kColO + q * 128, a + 16, v, id_o, true);
      };
      auto pv = [&](int q, int t, bool add) {
        const int n = ps[q]++;
        if (!wait(C::kP + q, n) || !full(u0 + 2 * t + 1)) return false;
        issue_pv(q, t, 0, add);
        if (!wait(C::kPHi + q, n)) return false;
        issue_pv(q, t, 1, add);
        return true;
      };
      auto free_k = [&](int t) { commit_elect(bar(C::kEmpty + (u0 + 2 * t) % kSlots)); };
      auto free_v = [&](int t) { commit_elect(bar(C::kEmpty + (u0 + 2 * t + 1) % kSlots)); };
      bool ok = true;
      int seg = 0, n_two = 0;
      while (ok) {
        ok = wait(C::kSeg + (seg & 1), seg >> 1);
        if (!ok || !sh.more[seg & 1]) break;
        const int T = sh.seg[seg & 1].nt;
        const bool two = is_two(sh.seg[seg & 1]), last = sh.last[seg & 1] != 0;
        n_two += two;
        if constexpr (C::kHalf)
          ok = wait(C::kQReady + 0, seg) && (!two || wait(C::kQReady + 1, n_two - 1)) && full(u0);
        else
          ok = wait(C::kQFull, seg) && full(u0);
        if (!ok) break;
        issue_s(0, 0, 0);
        if (two) {
          issue_s(1, 0, 1);
          if (T == 1) commit_elect(bar(C::kQFree));
        }
        free_k(0);
        if (!two && T > 1) {
          ok = full(u0 + 2);
          if (!ok) break;
          issue_s(1, 1, 0);
          free_k(1);
        }
        // O of the last segment has been read (S, which P of the last segment
        // held, was free at its last product)
        if (seg > 0) ok = wait(C::kOFree, seg - 1);
        if (two) {
          for (int t = 0; ok && t < T; ++t) {
            ok = pv(0, t, t > 0);
            if (!ok) break;
            if (t + 1 < T) {
              ok = full(u0 + 2 * t + 2);
              if (!ok) break;
              issue_s(0, t + 1, 0);
            }
            ok = pv(1, t, t > 0);
            if (!ok) break;
            free_v(t);
            if (t + 1 < T) {
              issue_s(1, t + 1, 1);
              free_k(t + 1);
              if (t + 2 == T) commit_elect(bar(C::kQFree));
            }
          }
        } else {
          for (int t = 0; ok && t < T; ++t) {
            const int q = t & 1;
            ok = pv(q, t, t > 1);
            if (!ok) break;
            free_v(t);
            if (t + 2 < T) {
              ok = full(u0 + 2 * t + 4);
              if (!ok) break;
              issue_s(q, t + 2, 0);
              free_k(t + 2);
            }
          }
        }
        if (ok) commit_elect(bar(C::kODone));
        if (last) break;
        u0 += 2 * T;
        ++seg;
      }
      if (!ok) fail(lane == 0);
    }
    __syncwarp();
  } else if (warp == 11) {
    regs_aux();
    // ------------------------------------------------------------- segments
    // Segment k goes into place k & 1 when segment k - 2 has left it: found while
    // the softmax warps are at work (the walk's loads and divisions between two
    // segments cost them 2 us).
    // Of a block's segments only the first and the last can be parts of a
    // unit. The first one's partial, when others follow, is counted in here:
    // the softmax warps go on to the next unit meanwhile (waiting for their
    // writes and the counter cost them 2 us). Should the unit be complete with
    // it -- its other blocks as a rule end later -- the softmax warps merge it
    // after their last segment.
    bool complete = false;
    if (lane == 0) {
      TreeWalk walk = begin();
      for (int k = 0;; ++k) {
        if (k >= 2) {
          const bool ok = mbar_wait(bar(C::kSegFree + (k & 1)), ((k >> 1) - 1) & 1, p.wait_ns);
          if (!ok) fail(true);
          if (!ok || stop()) break;
        }
        TreeSegment& g = sh.seg[k & 1];
        const bool more = walk.next(p, kBN, rows_per_block, g), last = walk.at >= walk.end;
        sh.more[k & 1] = more;
        sh.last[k & 1] = last;
        if (k == 0) sh.first = g;
        mbar_arrive(bar(C::kSeg + (k & 1)));
        if (k == 1 && !(sh.first.head && sh.first.tail)) {
          const bool ok = mbar_wait(bar(C::kPart), 0, p.wait_ns);
          if (!ok) fail(true);
          if (!ok || stop()) break;
          const TreeMerge mg = tree_merge(plan, sh.first);
          __threadfence();  // the partial (seen through the barrier), before the count
          complete = atomicAdd(p.arrived + mg.ca, 1) == mg.m - 1;
          __threadfence();  // the other blocks' partials, after it
        }
        if (!more || last) break;
      }
    }
    __syncwarp();
    if (lane == 0) sh.pending = complete;
    named_bar_sync(3, 256 + 32);
  } else if (kByte && warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsConvert));
    // ---------------------------------------------------------- converters
    // Thread (r, h) widens the 64 dims of half h of row r (key key0 + r) of
    // every tile.
    if constexpr (kByte) {
      constexpr int kRaw = C::kRaw;
      const int r = (tid - 384) & 127, h = (tid - 384) >> 7;
      TreeWalk walk = begin();
      TreeSegment g;
      bool ok = true, waited = !p.early;
      int u = 0;
      while (ok && walk.next(p, kBN, rows_per_block, g)) {
        const int key_first = g.s.first + g.t0 * kBN;
        // uint8: the (scale, zero point) of this thread's row of a tile, zeros
        // where nothing may be read; requested a tile ahead
        auto scales = [&](int t, float2& k, float2& v) {
          k = v = make_float2(0.f, 0.f);
          const int key = key_first + t * kBN + r;
          if (DT != kDtypeU8 || t >= g.nt || key < g.s.lo || key >= g.s.len) return;
          long long row;
          if constexpr (PG) {
            const int page = __ldg(p.block_table + static_cast<long long>(g.b) * p.max_pages + key / p.page_size);
            if (page < 0 || page >= p.num_pages) return;
            row = (static_cast<long long>(page) * p.h_kv + g.j) * p.page_size + (key & (p.page_size - 1));
          } else {
            row = (static_cast<long long>(g.b) * p.h_kv + g.j) * p.capacity + key;
          }
          k = p.k_sz[row];  // (plain loads: the append of this step may have written them)
          v = p.v_sz[row];
        };
        auto appended = [&](int t) {  // before the scales of a tile that holds a node
          if (DT == kDtypeU8 && !waited && key_first + (t + 1) * kBN > g.s.pos) {
            grid_dependency_wait();
            waited = true;
          }
        };
        float2 k_now, v_now, k_next, v_next;
        appended(0);
        scales(0, k_now, v_now);
        for (int t = 0; t < g.nt && ok; ++t) {
          const int key = key_first + t * kBN + r;
          const bool live = key >= g.s.lo && key < g.s.len;
          appended(t + 1);
          scales(t + 1, k_next, v_next);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++u) {
            const int rs = u % kRaw, slot = u % kSlots;
            ok = mbar_wait(bar(C::kRFull + rs), (u / kRaw) & 1, p.wait_ns) &&
                 (u < kSlots || mbar_wait(bar(C::kEmpty + slot), (u / kSlots - 1) & 1, p.wait_ns));
            if (!ok) fail(true);
            ok = __all_sync(0xffffffffu, ok && !stop());
            if (!ok) break;
            const unsigned char* src = smem + C::kRawOff + rs * kRawBytes + r * 128;
            unsigned char* dst = smem + C::kRingOff + slot * kTileBytes + h * 16384 + r * 128;
            const float2 sz = kv ? v_now : k_now;
            const uint32_t z = u8_zero(sz.y);
            // (16 codes a pass, the next ones requested before this pass's stores.
            // Short code: all four passes unrolled, the uint8 kernel took a quarter
            // longer, as the instruction cache is shared with the softmax)
            auto codes = [&](int c) { return *reinterpret_cast<const uint4*>(src + (((4 * h + c) ^ (r & 7)) << 4)); };
            uint4 w = codes(0), next;
#pragma unroll(DT == kDtypeU8 ? 1 : 2)
            for (int c = 0; c < 4; ++c) {
              next = codes((c + 1) & 3);
              uint2 a, b, e, f;
              if constexpr (DT == kDtypeF8) {
                a = half_e5m2(w.x), b = half_e5m2(w.y), e = half_e5m2(w.z), f = half_e5m2(w.w);
              } else {
                a = widen_u8(w.x, z), b = widen_u8(w.y, z), e = widen_u8(w.z, z), f = widen_u8(w.w, z);
              }
              if (!live) a = b = e = f = make_uint2(0u, 0u);
              *reinterpret_cast<uint4*>(dst + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
              *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(e.x, e.y, f.x, f.y);
              w = next;
            }
            if (DT == kDtypeU8 && h == 0)
              reinterpret_cast<float*>(smem + C::kScaleOff)[(u % C::kScales) * kBN + r] = sz.x * kU8Unit;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(C::kFull + slot));
              mbar_arrive(bar(C::kREmpty + rs));
            }
          }
          k_now = k_next;
          v_now = v_next;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // ---------------------------- softmax of accumulator q, row r per thread
    const int q = warp >> 2, r = tid & (kBM - 1);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_base + kColS + q * 128, ocol = tmem + lane_base + kColO + q * 128;
    float c = p.scale_log2;  // (e5m2: over the factor that Q's row was scaled by)
    const bool warp_rows = (warp & 3) * 32 < acc_rows;  // some lane of this warp holds a row
    bool waited = !p.early;
    int u0 = 0, seg = 0, js = 0;  // first load of the segment; segments; tiles of this accumulator
    bool ok = true, aborted = false;
    while (true) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kSeg + (seg & 1)), (seg >> 1) & 1, p.wait_ns) && !stop());
      if (!ok) fail(lane == 0);
      aborted = bar_any(2, 256, !ok);  // (and no warp is at the last segment any more)
      if (aborted || !sh.more[seg & 1]) break;
      const TreeSegment& g = sh.seg[seg & 1];
      const bool two = is_two(g);
      const int step = two ? 1 : 2;
      const int gr = g.rb * rows_per_block + (two ? q * acc_rows : 0) + r;  // row of the unit's kv head
      const bool live = r < acc_rows && gr < g.s.nodes * G;
      const int node = live ? gr / G : -1;
      // this row's first key, the first key that not every row attends to
      const int ka = tree_first_key(p, g.b, g.s, node), pos = g.s.pos;
      const int nt = g.nt;
      int key0 = g.s.first + (g.t0 + (two ? 0 : q)) * kBN;
      if constexpr (C::kHalf) {
        // e5m2: Q's rows as f16, each scaled by a power of two to a largest magnitude
        // in [2^9, 2^10): exact for all but values 2^24 below the row's largest
        if (two || q == 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kQFull), seg & 1, p.wait_ns) && !stop());
          if (ok && r < acc_rows) {
            c = p.scale_log2 / half_row(smem + C::kQOff + (two ? q : 0) * kTileBytes, r);
            if (!two) sh.row[0][r] = c;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(bar(C::kQReady + (two ? q : 0)));
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kQReady + 0), seg & 1, p.wait_ns) && !stop());
          c = sh.row[0][r];
        }
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int t = two ? 0 : q; ok && t < nt; t += step, ++js, key0 += step * kBN) {
        // only tiles that reach a node, the end or the window are masked
        // (one answer for the warp: what follows has to stay converged)
        const bool masked = __any_sync(0xffffffffu, key0 + kBN > pos || key0 < ka);
        // (uint8: the bits where they are used, which suits that loop's registers:
        // 32 x 16 nodes over 4096 keys 136 -> 129 us)
        TreeRow row;
        uint32_t bits[4];  // bit x: the row attends to key key0 + x
        if (masked && warp_rows) {
          row = tree_row(p, g.b, g.s, node);
          if constexpr (DT != kDtypeU8) {
#pragma unroll
            for (int w = 0; w < 4; ++w) bits[w] = tree_bits(row, key0 + 32 * w);
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kSFull + q), js & 1, p.wait_ns) && !stop());
        if (!ok) break;
        tc05::fence_after_sync();
        const int vs = (u0 + 2 * t + 1) % kSlots;  // V's slot
        if (!kByte && (!two || q == 0) && (key0 + kBN > g.s.len || key0 < g.s.lo)) {
          // rows that no node reads may hold anything (NaN included): P = 0
          // there, and 0 * NaN would still poison O. Their V rows are zeroed
          // once the tile has landed, before P is published.
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kFull + vs), ((u0 + 2 * t + 1) / kSlots) & 1, p.wait_ns));
          if (!ok) break;
          if (key0 + r >= g.s.len || key0 + r < g.s.lo) {
            unsigned char* vrow = smem + C::kRingOff + vs * kTileBytes + tile_row<kGrouped>(r);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              *reinterpret_cast<uint4*>(vrow + x * 16) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(vrow + L::kHalf + x * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        if (warp_rows) {
          const float* sc = reinterpret_cast<const float*>(smem + C::kScaleOff);
          const float4* sk = reinterpret_cast<const float4*>(sc + ((u0 + 2 * t) % C::kScales) * kBN);
          const float4* sv = reinterpret_cast<const float4*>(sc + ((u0 + 2 * t + 1) % C::kScales) * kBN);
          constexpr bool kMaskS = DT != kDtypeU8;
          auto scores = [&](int x, float (&s)[32]) {  // keys 32 x .. 32 x + 31, masked ones -inf
            tc05::wait_ld();
            tc05::reg_fence(s);
            if constexpr (DT == kDtypeU8) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 f = sk[8 * x + i];
                const float2 a = mul2(make_float2(s[4 * i], s[4 * i + 1]), make_float2(f.x, f.y));
                const float2 b = mul2(make_float2(s[4 * i + 2], s[4 * i + 3]), make_float2(f.z, f.w));
                s[4 * i] = a.x, s[4 * i + 1] = a.y, s[4 * i + 2] = b.x, s[4 * i + 3] = b.y;
              }
            }
            if (!kMaskS && masked) {  // (past the scales, which may be anything in a masked row)
              const uint32_t w = tree_bits(row, key0 + 32 * x);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((w >> i) & 1u)) s[i] = -INFINITY;
            }
          };
          // bf16, e5m2: -inf into S itself, out of the way of the other tiles' code (32 x
          // 64 nodes over 4096 keys, bf16 169.3 -> 167.2 us, e5m2 157.3 -> 152)
          if (kMaskS && masked) {
#pragma unroll 1
            for (int x = 0; x < kBN / 16; ++x) {
              const uint32_t w = (x < 4 ? (x < 2 ? bits[0] : bits[1]) : (x < 6 ? bits[2] : bits[3])) >> (16 * (x & 1));
              float v[16];
              tc05::ld_32x32b_x16(scol + 16 * x, v);
              tc05::wait_ld();
              tc05::reg_fence(v);
              uint32_t m[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) m[i] = (w >> i) & 1u ? __float_as_uint(v[i]) : 0xff800000u;
              tc05::st_32x32b_x16_u(scol + 16 * x, m);
            }
            tc05::wait_st();
          }
          // A thread's scores pass through registers twice, for the maximum and
          // for the probabilities. (128 of them kept in registers between the two
          // need a loop body twice as long, which was slower.) P of 32 keys takes
          // columns of S that this thread has read already.
          float mt = -INFINITY;
#pragma unroll 1
          for (int x = 0; x < kBN / 32; x += 2) {
            float s0[32], s1[32];
            tc05::ld_32x32b_x32(scol + 32 * x, s0);
            tc05::ld_32x32b_x32(scol + 32 * x + 32, s1);
            scores(x, s0);
            scores(x + 1, s1);
            float mx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = max3(s0[i], s0[8 + i], s0[16 + i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = max3(mx[i], s0[24 + i], s1[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = max3(mx[i], s1[8 + i], s1[16 + i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], s1[24 + i]);
            mt = max3(mt, max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], max3(mx[5], mx[6], mx[7])));
          }
          // a new reference maximum only when the row's maximum grew by more than 2^8
          const bool grow = (mt - m_ref) * c > kRescaleLog2 || (m_ref == -INFINITY && mt != -INFINITY);
          const float m_new = grow ? mt : m_ref;
          if (__any_sync(0xffffffffu, grow && m_ref != -INFINITY)) {
            // O is rescaled. The last product into O_q is done: it was issued
            // before this S_q, whose completion this thread has seen
            const float alpha = (grow && m_ref != -INFINITY) ? fast_exp2((m_ref - m_new) * c) : 1.f;
#pragma unroll 1
            for (int x = 0; x < kD / 16; ++x) {  // (16 dims a pass: as fast as 32, in half the code)
              float v[16];
              tc05::ld_32x32b_x16(ocol + x * 16, v);
              tc05::wait_ld();
              tc05::reg_fence(v);
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i] * alpha);
              tc05::st_32x32b_x16_u(ocol + x * 16, w);
            }
            l *= alpha;
          }
          m_ref = m_new;
          const float e = m_ref == -INFINITY ? 0.f : (C::kHalf ? kHalfShift - m_ref * c : -m_ref * c);
          float2 sm4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          if (DT == kDtypeU8) {  // the V tile's scales
            ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kFull + vs), ((u0 + 2 * t + 1) / kSlots) & 1, p.wait_ns));
            if (!ok) break;
          }
          auto probs = [&](int x, const float (&s)[32]) {
            uint32_t pk[C::kSplitP ? 32 : 16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 d0 = fma2(make_float2(s[2 * i], s[2 * i + 1]), c, e);
              const float2 d1 = fma2(make_float2(s[2 * i + 2], s[2 * i + 3]), c, e);
              float2 p0 = make_float2(fast_exp2(d0.x), fast_exp2(d0.y)), p1 = make_float2(fast_exp2(d1.x), fast_exp2(d1.y));
              sm4[i & 3] = add2(sm4[i & 3], p0);
              sm4[(i + 1) & 3] = add2(sm4[(i + 1) & 3], p1);
              if constexpr (DT == kDtypeU8) {
                const float4 f = sv[8 * x + i / 2];
                p0 = mul2(p0, make_float2(f.x, f.y));
                p1 = mul2(p1, make_float2(f.z, f.w));
              }
              if constexpr (C::kSplitP) {
                split_p(p0, pk[i], pk[16 + i]);
                split_p(p1, pk[i + 1], pk[17 + i]);
              } else {
                pk[i] = pack_p<C::kHalf>(p0);
                pk[i + 1] = pack_p<C::kHalf>(p1);
              }
            }
            if constexpr (C::kSplitP)
              tc05::st_32x32b_x32_u(scol + 32 * x, pk);
            else
              tc05::st_32x32b_x16_u(scol + 16 * x, pk);
          };
#pragma unroll 1
          for (int x = 0; x < kBN / 32; ++x) {
            float s0[32];
            tc05::ld_32x32b_x32(scol + 32 * x, s0);
            scores(x, s0);
            probs(x, s0);
            if (!(x & 1)) continue;
            // these 64 keys' P is in tensor memory: their products may start
            tc05::wait_st();
            tc05::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar((x == 1 ? C::kP : C::kPHi) + q));
          }
          l += ((sm4[0].x + sm4[0].y) + (sm4[1].x + sm4[1].y)) + ((sm4[2].x + sm4[2].y) + (sm4[3].x + sm4[3].y));
        } else {  // no rows here: the arrivals that the products wait for
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::kP + q));
            mbar_arrive(bar(C::kPHi + q));
          }
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::kODone), seg & 1, p.wait_ns) && !stop());
      if (!ok && lane == 0) fail(true);
      // all eight warps agree whether the segment's result stands
      aborted = bar_any(2, 256, !ok);
      if (aborted) break;
      tc05::fence_after_sync();
      if (!waited) {  // the append clears the counters; out may still be read before it
        grid_dependency_wait();
        waited = true;
      }
      // ---- the segment's result, 32 dims at a time: a whole unit's goes out,
      // a part's into the workspace. (One copy of this code for every case:
      // fetching it costs more than running it.)
      const bool whole = g.head && g.tail, last = sh.last[seg & 1] != 0;
      // both accumulators hold these rows: each warpgroup hands the other's 64
      // dims over and puts out its own, through the Q area (free: every product
      // with Q is done; NT = 2: the second row tile's half), 16 KB a direction
      const bool both = !two && nt > 1;
      unsigned char* xbuf = smem + C::kQOff + (NT - 1) * kTileBytes;
      float m2 = m_ref == -INFINITY ? -INFINITY : (C::kHalf ? m_ref * c - kHalfShift : m_ref * c), w0 = 1.f, w1 = 0.f, mo = 0.f, lo = 0.f;
      if (both) {
        if (q == 1) {
          sh.row[0][r] = m2;
          sh.row[1][r] = l;
        }
        named_bar_sync(1, 256);
        if (q == 0) {
          mo = sh.row[0][r];
          lo = sh.row[1][r];
          sh.row[0][r] = m2;
          sh.row[1][r] = l;
        }
      }
      const bool writer = (two || both || q == 0) && warp_rows;
      const long long orow = live ? tree_out_row(p, g, gr) : 0;
      const int br = gr - g.rb * rows_per_block;  // row of the block
      float* part = tree_place(p, g, blockIdx.x, rows_per_block, kD);
      float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN score: NaN)
      auto weights = [&]() {  // of the two accumulators in what both hold
        const float mx = fmaxf(m2, mo);
        w0 = mx != -INFINITY ? exp2f(m2 - mx) : 0.f;
        w1 = mx != -INFINITY ? exp2f(mo - mx) : 0.f;
        l = w0 * l + w1 * lo;
        m2 = mx;
        inv = l != 0.f ? 1.f / l : 0.f;
      };
      // this thread's pieces of 32 dims
      const int x0 = both ? 2 * q : 0, x1 = both ? x0 + 2 : kD / 32;
#pragma unroll 1
      for (int x = x0; x < x1; ++x) {
        float v[32];
        auto piece = [&](int from, int i) {  // 16 bytes i of row r of accumulator `from`
          return reinterpret_cast<float4*>(xbuf + from * 16384 + r * 128 + ((i ^ (r & 7)) << 4));
        };
        if (both) {
          if (x > x0) named_bar_sync(1, 256);  // what was handed over has been read
          __syncwarp();
          if (warp_rows) {
            tc05::ld_32x32b_x32(ocol + (x ^ 2) * 32, v);
            tc05::wait_ld();
            tc05::reg_fence(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) *piece(q, i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
          named_bar_sync(1, 256);
        }
        __syncwarp();
        if (writer) {
          tc05::ld_32x32b_x32(ocol + x * 32, v);
          tc05::wait_ld();
          tc05::reg_fence(v);
        }
        if (both) {
          if (x == x0) {
            if (q == 1) {
              mo = sh.row[0][r];
              lo = sh.row[1][r];
            }
            weights();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 o = *piece(1 - q, i);
            v[4 * i] = fmaf(w1, o.x, w0 * v[4 * i]);
            v[4 * i + 1] = fmaf(w1, o.y, w0 * v[4 * i + 1]);
            v[4 * i + 2] = fmaf(w1, o.z, w0 * v[4 * i + 2]);
            v[4 * i + 3] = fmaf(w1, o.w, w0 * v[4 * i + 3]);
          }
        }
        if (x + 1 == x1) {  // O is read, the Q area, and the segment's place
          tc05::fence_before_sync();
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::kOFree));
            mbar_arrive(bar(C::kSegFree + (seg & 1)));
            if (!two) mbar_arrive(bar(C::kXFree));
          }
        }
        if (writer) {
          if (!whole) {
            if (live) {
              float4* dst = reinterpret_cast<float4*>(part) + static_cast<size_t>(8 * x) * rows_per_block + br;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[static_cast<size_t>(i) * rows_per_block] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
          } else if (p.out_dtype == kDtypeF32) {
            if (live) {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow * kD + 32 * x);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
            }
          } else {
            // bf16: four lanes exchange their rows' 16-byte pieces, so that
            // they write 64 bytes of one row together (a lane writing its own
            // row touches 32 lines with every store: 256 rows took 6 us)
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
            transpose4(w, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const long long to = __shfl_sync(0xffffffffu, live ? orow : -1ll, (lane & ~3) + k);
              if (to >= 0)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to * kD + 32 * x + 8 * (lane & 3)) =
                    make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
          }
        }
      }
      if (writer && live && (two || q == 0)) {
        if (!whole) {
          part[static_cast<size_t>(rows_per_block) * kD + br] = m2;
          part[static_cast<size_t>(rows_per_block) * (kD + 1) + br] = l;
        } else if (p.lse_out != nullptr) {
          p.lse_out[orow] = l != 0.f ? (m2 + log2f(l)) * 0.69314718055994530942f : -INFINITY;
        }
      }
      __syncwarp();
      if (lane == 0 && !whole && !last) mbar_arrive(bar(C::kPart));
      if (last) break;
      u0 += 2 * nt;
      ++seg;
    }
    // ---- parts of units: the last segment's is counted in here, the first
    // one's was by warp 11; a unit that is complete is merged
    named_bar_sync(3, 256 + 32);
    if (!aborted) {
      const TreeSegment& g = sh.seg[seg & 1];
      const bool part = sh.more[seg & 1] && !(g.head && g.tail);
      bool complete = false;
      if (part)
        complete = tree_arrive(p, tree_merge(plan, g), tid, &sh.flag, [] { named_bar_sync(1, 256); });
#pragma unroll 1
      for (int i = 0; i < 2; ++i)
        if (i == 0 ? complete : sh.pending != 0) {
          const TreeSegment& f = i == 0 ? g : sh.first;
          tree_merge_rows<kD>(p, tree_merge(plan, f), f, rows_per_block, tid, 256);
        }
    }
  }

  // a block without work ends behind the append all the same: what follows in
  // the stream may take this launch's end for the append's
  if (p.early && tid == 0) grid_dependency_wait();
  // ---- teardown: every role is done with tensor memory
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    if (*reinterpret_cast<volatile int*>(&sh.abort)) {
      // products may still be in flight after a timeout: wait (bounded) for
      // them before the columns are released
      commit_elect(bar(C::kDrain));  // (the lane that issued them)
      if (lane == 0) (void)mbar_wait(bar(C::kDrain), 0, kWaitLimitNs);
      __syncwarp();
    }
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int NT, bool PG, int DT>
cudaError_t launch_tree_tc05_t(const TreeParams& p, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CUtensorMap& tq, cudaStream_t stream) {
  using C = Cfg<NT, DT>;
  auto kern = attn_tree_tc05_kernel<NT, PG, DT>;
  // a build with another register count at launch would leave setmaxnreg.inc
  // waiting for registers that never come: it is not launched
  static const int launch_regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : -1;
  }();
  if (launch_regs != C::kRegsLaunch) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, tq, p);
}

template <int DT>
cudaError_t launch_tree_tc05_dt(const TreeParams& p, int tiles, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tq, cudaStream_t stream) {
  if constexpr (DT != kDtypeU8)
    if (tiles == 2)
      return p.paged ? launch_tree_tc05_t<2, true, DT>(p, ctas, tk, tv, tq, stream)
                     : launch_tree_tc05_t<2, false, DT>(p, ctas, tk, tv, tq, stream);
  if (tiles != 1) return cudaErrorInvalidValue;
  return p.paged ? launch_tree_tc05_t<1, true, DT>(p, ctas, tk, tv, tq, stream)
                 : launch_tree_tc05_t<1, false, DT>(p, ctas, tk, tv, tq, stream);
}

}  // namespace
}  // namespace mqa
