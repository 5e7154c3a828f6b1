// Attention of a tree of drafted tokens over the cache on warp-level tensor
// cores, for every cache the library reads on tensor cores: bf16, uint8 codes
// and fp8 e5m2, contiguous or paged, head_dim 64 or 128, any group.
// attn_tree_tc05.cuh takes head_dim 128 with up to 128 heads per kv head; this
// kernel the rest.
//
// Rows of kv head j are its (node i, query head h = j G + hl) pairs, row =
// i G + hl, in blocks of 64: four warps with 16 rows each share every 64-key
// tile. Per tile, with FlashAttention's running maximum and sum ("Arsitektur
// Inferensi LLM", section 5):
//   S = Q K^T, masked;  m' = max(m, max S);  P = 2^(c (S - m')), c = scale log2 e
//   O = 2^(c (m - m')) O + P V;  l = 2^(c (m - m')) l + sum P
// S, P and O live in registers (m16n8k16 fragments), K and V in shared memory
// as bf16 (two tiles each, four at head_dim 64: one is used while the others
// arrive). One-byte caches are widened on the way in, exactly: an e5m2 value
// has 3 significant bits, code - zero point is an integer of magnitude <= 255
// and has 8. The row's scale then multiplies the score (K) or the probability
// (V) in fp32. P enters its product as two bf16 terms (split_p, within 2^-15;
// one term, 2^-8, was more than half of the output's error).
//
// Keys that no row may read (past the sequence, before the window) land as
// zeros whatever the cache holds there.
//
// Bound: with few rows the HBM stream of K and V; the tiles' L2-to-SM copies
// and the 64-row MMA work from about 64 rows per kv head on (32 x 16 nodes on
// 4096 keys, 32 + 8 heads of 64 dims, 273 MB: a step takes 105 us, 2.6 TB/s;
// with P in one term 89 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mqa_decode.h"
#include "launch.h"
#include "ptx.cuh"
#include "tree.cuh"

namespace mqa {
namespace {

constexpr int kRows = 64;    // rows per block
constexpr int kKeys = 64;    // keys per tile
constexpr int kThreads = 128;

template <int D, bool BYTE>
struct Lay {
  static constexpr int kTile = kKeys * D * 2;          // one bf16 tile
  // bf16: four tiles in flight at d = 64 (two: half the rate); one-byte caches
  // hold the next tile in registers
  static constexpr int kStages = BYTE || D == 128 ? 2 : 4;
  static constexpr int kK = 0, kV = kStages * kTile;   // [kStages] each
  static constexpr int kScale = 2 * kStages * kTile;   // uint8: K, V scales [2][2][kKeys]
  static constexpr int kBytes = kScale + 4 * kKeys * 4;
};

// byte offset of 16-byte chunk c of row r
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  return r * (D * 2) + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// four codes (one word) as two bf16 pairs; z: u8_zero of the row's zero point
template <int DT>
__device__ __forceinline__ uint2 widen4(uint32_t w, uint32_t z) {
  if constexpr (DT == kDtypeU8) {
    return widen_u8(w, z);
  } else {  // an e5m2 code is the high byte of an IEEE half
    const uint32_t h01 = __byte_perm(w, 0u, 0x1404), h23 = __byte_perm(w, 0u, 0x3424);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h23));
    return make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3) attn_tree_kernel(const TreeParams p) {
  using Y = Lay<D, DT != kDtypeBf16>;
  constexpr int kStages = Y::kStages;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ TreePlan plan;
  __shared__ int s_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group;
  constexpr bool kByte = DT != kDtypeBf16;

  grid_dependency_wait();  // q_rot, the nodes' cache rows and the cleared counters
  if (warp == 0) tree_plan(p, kKeys, kRows, blockIdx.x, gridDim.x, &plan);
  __syncthreads();
  TreeWalk walk;
  walk.start(plan);
  const uint32_t sb = smem_u32(smem);
  const float c = p.scale_log2;

  TreeSegment g;
  while (walk.next(p, kKeys, kRows, g)) {
    const int b = g.b, j = g.j, row0 = g.rb * kRows, rows_unit = g.s.nodes * G;
    // ---- this lane's two rows: 16 warp + lane / 4, + 8
    const int ra = row0 + 16 * warp + (lane >> 2), rb = ra + 8;
    TreeRow tr[2];
    tr[0] = tree_row(p, b, g.s, ra < rows_unit ? ra / G : -1);
    tr[1] = tree_row(p, b, g.s, rb < rows_unit ? rb / G : -1);
    // ---- Q fragments
    uint32_t q[D / 16][4];
    {
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q_rot);
      const long long oa = tree_out_row(p, g, ra < rows_unit ? ra : row0) * D + (lane & 3) * 2;
      const long long ob = tree_out_row(p, g, rb < rows_unit ? rb : row0) * D + (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][0] = *reinterpret_cast<const uint32_t*>(qp + oa + 16 * k);
        q[k][1] = *reinterpret_cast<const uint32_t*>(qp + ob + 16 * k);
        q[k][2] = *reinterpret_cast<const uint32_t*>(qp + oa + 16 * k + 8);
        q[k][3] = *reinterpret_cast<const uint32_t*>(qp + ob + 16 * k + 8);
      }
    }
    // ---- loads. Thread t takes chunks t, t + 128, ... of a tile's rows (a
    // chunk is 16 bytes of the cache: 8 bf16 or 16 codes).
    constexpr int kEl = kByte ? 16 : 8, kPerRow = D / kEl, kN = kKeys * kPerRow / kThreads;
    uint4 kr[kByte ? kN : 1], vr[kByte ? kN : 1];
    float2 ksz[kByte ? kN : 1], vsz[kByte ? kN : 1];
    bool bad_page = false;
    // row (token) of the cache a key lives in, -1: none (or no valid page)
    auto row_of = [&](int key) -> long long {
      if (key < g.s.lo || key >= g.s.len) return -1;
      if (!p.paged) return (static_cast<long long>(b) * p.h_kv + j) * p.capacity + key;
      const int page = __ldg(p.block_table + static_cast<long long>(b) * p.max_pages + key / p.page_size);
      if (page < 0 || page >= p.num_pages) {
        bad_page = true;
        return -1;
      }
      return (static_cast<long long>(page) * p.h_kv + j) * p.page_size + (key & (p.page_size - 1));
    };
    auto request = [&](int t, int st) {  // tile t of the unit
      const int key0 = g.s.first + (g.t0 + t) * kKeys;
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        const int ch = tid + u * kThreads, r = ch / kPerRow, cc = ch - r * kPerRow;
        const long long row = row_of(key0 + r);
        const long long off = (row < 0 ? 0 : row * D + cc * kEl) * (kByte ? 1 : 2);
        const unsigned char* ks = static_cast<const unsigned char*>(p.k_cache) + off;
        const unsigned char* vs = static_cast<const unsigned char*>(p.v_cache) + off;
        if constexpr (!kByte) {
          copy16(sb + Y::kK + st * Y::kTile + chunk_at<D>(r, cc), ks, row >= 0);
          copy16(sb + Y::kV + st * Y::kTile + chunk_at<D>(r, cc), vs, row >= 0);
        } else {
          kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
          ksz[u] = vsz[u] = make_float2(0.f, 0.f);  // (scale, zero point): a missing row is zero
          if (row >= 0) {
            kr[u] = *reinterpret_cast<const uint4*>(ks);
            vr[u] = *reinterpret_cast<const uint4*>(vs);
            if constexpr (DT == kDtypeU8) {
              ksz[u] = p.k_sz[row];
              vsz[u] = p.v_sz[row];
            }
          }
        }
      }
      if constexpr (!kByte) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto land = [&](int st) {  // one-byte caches: the requested codes, widened, into shared memory
      if constexpr (kByte) {
#pragma unroll
        for (int u = 0; u < kN; ++u) {
          const int ch = tid + u * kThreads, r = ch / kPerRow, cc = ch - r * kPerRow;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint4 w = kv ? vr[u] : kr[u];
            const float2 sz = kv ? vsz[u] : ksz[u];
            const uint32_t z = DT == kDtypeU8 ? u8_zero(sz.y) : 0u;
            const uint2 a = widen4<DT>(w.x, z), e = widen4<DT>(w.y, z);
            const uint2 f = widen4<DT>(w.z, z), h = widen4<DT>(w.w, z);
            unsigned char* dst = smem + (kv ? Y::kV : Y::kK) + st * Y::kTile;
            *reinterpret_cast<uint4*>(dst + chunk_at<D>(r, 2 * cc)) = make_uint4(a.x, a.y, e.x, e.y);
            *reinterpret_cast<uint4*>(dst + chunk_at<D>(r, 2 * cc + 1)) = make_uint4(f.x, f.y, h.x, h.y);
            if (DT == kDtypeU8 && cc == 0)
              reinterpret_cast<float*>(smem + Y::kScale)[(kv * 2 + st) * kKeys + r] = sz.x * kU8Unit;
          }
        }
      }
    };

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    // (a group is committed for each tile, past the last one too: the count of
    // groups behind tile t is then always kStages - 1)
    auto ahead = [&](int t) {
      if (t < g.nt)
        request(t, t % kStages);
      else if constexpr (!kByte)
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (kByte) {
      ahead(0);
    } else {
      for (int t = 0; t < kStages - 1; ++t) ahead(t);
    }
    for (int t = 0; t < g.nt; ++t) {
      const int st = t % kStages;
      if constexpr (kByte) {
        land(st);
        ahead(t + 1);
      } else {
        ahead(t + kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      }
      __syncthreads();
      const uint32_t ks = sb + Y::kK + st * Y::kTile, vs = sb + Y::kV + st * Y::kTile;
      float s[kKeys / 8][4];
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int np = 0; np < kKeys / 16; ++np) {
          const int r = np * 16 + (lane & 7) + ((lane >> 4) << 3), cc = 2 * k + ((lane >> 3) & 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(ks + chunk_at<D>(r, cc), b0, b1, b2, b3);
          mma_bf16_16816(s[2 * np], q[k], b0, b1);
          mma_bf16_16816(s[2 * np + 1], q[k], b2, b3);
        }
      }
      if constexpr (DT == kDtypeU8) {
        const float* sc = reinterpret_cast<const float*>(smem + Y::kScale) + st * kKeys;
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) {
          const float2 f = *reinterpret_cast<const float2*>(sc + 8 * i + (lane & 3) * 2);
          s[i][0] *= f.x, s[i][1] *= f.y, s[i][2] *= f.x, s[i][3] *= f.y;
        }
      }
      // ---- mask: only tiles that reach a node, the window or the end
      const int key0 = g.s.first + (g.t0 + t) * kKeys;
      if (key0 + kKeys > g.s.pos || p.window > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = tree_bits(tr[h], key0), w1 = tree_bits(tr[h], key0 + 32);
#pragma unroll
          for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = 8 * i + (lane & 3) * 2 + e;
              if (!((col < 32 ? w0 >> col : w1 >> (col - 32)) & 1u)) s[i][2 * h + e] = -INFINITY;
            }
        }
      }
      // ---- softmax
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = m[h];
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) mx = fmaxf(mx, fmaxf(s[i][2 * h], s[i][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float e = mx == -INFINITY ? 0.f : mx;  // nothing attended yet: every probability 2^-inf = 0
        alpha[h] = fast_exp2((m[h] - e) * c);
        m[h] = mx;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float pr = fast_exp2((s[i][2 * h + x] - e) * c);
            s[i][2 * h + x] = pr;
            sum += pr;
          }
        }
        l[h] = l[h] * alpha[h] + sum;  // (of this lane's columns; the four lanes' sums meet at the end)
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= alpha[0], o[i][1] *= alpha[0];
          o[i][2] *= alpha[1], o[i][3] *= alpha[1];
        }
      }
      if constexpr (DT == kDtypeU8) {
        const float* sc = reinterpret_cast<const float*>(smem + Y::kScale) + (2 + st) * kKeys;
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) {
          const float2 f = *reinterpret_cast<const float2*>(sc + 8 * i + (lane & 3) * 2);
          s[i][0] *= f.x, s[i][1] *= f.y, s[i][2] *= f.x, s[i][3] *= f.y;
        }
      }
      // ---- O += P V
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k) {
        uint32_t a[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          split_p(make_float2(s[2 * k + (i >> 1)][2 * (i & 1)], s[2 * k + (i >> 1)][2 * (i & 1) + 1]), a[i], al[i]);
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          const int r = k * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, cc = 2 * dp + (lane >> 4);
          uint32_t b0, b1, b2, b3;
          ldsm_x4_trans(vs + chunk_at<D>(r, cc), b0, b1, b2, b3);
          mma_bf16_16816(o[2 * dp], a, b0, b1);
          mma_bf16_16816(o[2 * dp + 1], a, b2, b3);
          mma_bf16_16816(o[2 * dp], al, b0, b1);
          mma_bf16_16816(o[2 * dp + 1], al, b2, b3);
        }
      }
      __syncthreads();  // the tile is read: the next request may overwrite it
    }
    if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(p.err, static_cast<int>(MQA_DEVERR_PAGE_RANGE));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    // ---- the segment's result
    if (g.head && g.tail) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = h == 0 ? ra : rb;
        if (r >= rows_unit) continue;
        const float inv = l[h] != 0.f ? 1.f / l[h] : 0.f;  // (a NaN score: NaN)
        const long long orow = tree_out_row(p, g, r);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const long long at = orow * D + 8 * i + (lane & 3) * 2;
          const float x = o[i][2 * h] * inv, y = o[i][2 * h + 1] * inv;
          if (p.out_dtype == kDtypeBf16)
            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at) = pack_bf16x2(x, y);
          else
            *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(x, y);
        }
        if ((lane & 3) == 0 && p.lse_out != nullptr)
          p.lse_out[orow] = l[h] != 0.f ? (m[h] * c + log2f(l[h])) * 0.69314718055994530942f : -INFINITY;
      }
    } else {
      float* part = tree_place(p, g, blockIdx.x, kRows, D);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * warp + (lane >> 2) + 8 * h;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)  // columns 8 i + 2 (lane % 4): half of piece 2 i + (lane % 4) / 2
          *reinterpret_cast<float2*>(part + ((2 * i + ((lane & 3) >> 1)) * kRows + r) * 4 + (lane & 1) * 2) =
              make_float2(o[i][2 * h], o[i][2 * h + 1]);
        if ((lane & 3) == 0) {
          part[kRows * D + r] = m[h] == -INFINITY ? -INFINITY : m[h] * c;
          part[kRows * (D + 1) + r] = l[h];
        }
      }
      const TreeMerge mg = tree_merge(plan, g);
      if (tree_arrive(p, mg, tid, &s_flag, [] { __syncthreads(); }))
        tree_merge_rows<D>(p, mg, g, kRows, tid, kThreads);
    }
  }
}

template <int D, int DT>
cudaError_t launch_t(const TreeParams& p, int ctas, cudaStream_t stream) {
  auto kern = attn_tree_kernel<D, DT>;
  constexpr int smem = Lay<D, DT != kDtypeBf16>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

// (blocks per SM: what their registers allow, 255 and 168 a thread, the latter
// by the launch bounds: left alone, uint8 took more and 133 us instead of 109)
TreeShape tree_mma_shape(int head_dim) { return {kRows, head_dim == 128 ? 2 : 3}; }

cudaError_t launch_tree_mma(const TreeParams& p, int ctas, cudaStream_t stream) {
  if (p.head_dim == 128) {
    if (p.cache_dtype == kDtypeBf16) return launch_t<128, kDtypeBf16>(p, ctas, stream);
    if (p.cache_dtype == kDtypeU8) return launch_t<128, kDtypeU8>(p, ctas, stream);
    return launch_t<128, kDtypeF8>(p, ctas, stream);
  }
  if (p.cache_dtype == kDtypeBf16) return launch_t<64, kDtypeBf16>(p, ctas, stream);
  if (p.cache_dtype == kDtypeU8) return launch_t<64, kDtypeU8>(p, ctas, stream);
  return launch_t<64, kDtypeF8>(p, ctas, stream);
}

}  // namespace mqa
