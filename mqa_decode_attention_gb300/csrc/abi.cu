// The C ABI of libmqa_decode.so (declared in include/mqa_decode.h):
// host-side argument checks, split choice, TMA descriptor encoding, launches.
// Nothing here allocates device memory or synchronises.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/mqa_decode.h"
#include "launch.h"

namespace {
thread_local char g_cuda_error[256] = "";
}  // namespace

void mqa::record_cuda_error(cudaError_t e) {
  snprintf(g_cuda_error, sizeof(g_cuda_error), "%s: %s", cudaGetErrorName(e), cudaGetErrorString(e));
}

namespace {

using namespace mqa;

mqa_status fail_cuda(cudaError_t e) {
  record_cuda_error(e);
  return MQA_ERR_CUDA;
}

unsigned long long wait_limit(const mqa_kv_layout* L) {
  return L->wait_limit_ns > 0 ? static_cast<unsigned long long>(L->wait_limit_ns) : kWaitLimitNs;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_pow2(long long x) { return x > 0 && (x & (x - 1)) == 0; }

long long token_limit(const mqa_kv_layout* L) {
  return L->paged ? static_cast<long long>(L->max_pages_per_seq) * L->page_size : L->capacity;
}

mqa_status check_layout(const mqa_kv_layout* L) {
  if (L == nullptr) return MQA_ERR_INVALID_ARG;
  if (L->cache_dtype != MQA_BF16 && L->cache_dtype != MQA_F32 && L->cache_dtype != MQA_U8 &&
      L->cache_dtype != MQA_FP8_E5M2 && L->cache_dtype != MQA_U4)
    return MQA_ERR_UNSUPPORTED;
  if (L->cache_dtype == MQA_U8 || L->cache_dtype == MQA_U4) {
    if (L->k_scale_zero == nullptr || L->v_scale_zero == nullptr) return MQA_ERR_INVALID_ARG;
    if (!aligned(L->k_scale_zero, 16) || !aligned(L->v_scale_zero, 16)) return MQA_ERR_INVALID_ARG;
    // the (scale, zero) or (scale, minimum) rows of a kv head are copied in units of 16 bytes
    if (!L->paged && L->capacity % (L->cache_dtype == MQA_U8 ? 2 : 4) != 0) return MQA_ERR_UNSUPPORTED;
  }
  if (L->batch < 1 || L->h_q < 1 || L->h_kv < 1 || L->h_q % L->h_kv != 0) return MQA_ERR_INVALID_ARG;
  if (L->head_dim != 64 && L->head_dim != 128) return MQA_ERR_UNSUPPORTED;
  if (L->k_cache == nullptr || L->v_cache == nullptr) return MQA_ERR_INVALID_ARG;
  if (!aligned(L->k_cache, 16) || !aligned(L->v_cache, 16)) return MQA_ERR_INVALID_ARG;
  if (L->paged != 0 && L->paged != 1) return MQA_ERR_INVALID_ARG;
  if (L->window < 0) return MQA_ERR_INVALID_ARG;
  if (!L->paged) {
    if (L->capacity < 1 || L->capacity > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  } else {
    if (L->page_size < 16 || L->page_size > 256 || !is_pow2(L->page_size)) return MQA_ERR_UNSUPPORTED;
    if (L->num_pages < 1 || L->max_pages_per_seq < 1 || L->block_table == nullptr) return MQA_ERR_INVALID_ARG;
    if (!aligned(L->block_table, 4)) return MQA_ERR_INVALID_ARG;
    if (static_cast<long long>(L->max_pages_per_seq) * L->page_size > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  }
  // (token indexes of a few tiles past the last one are formed in 32 bits)
  if (L->cache_dtype == MQA_U4 && token_limit(L) > (1ll << 31) - 1024) return MQA_ERR_UNSUPPORTED;
  return MQA_OK;
}

int resolve_variant(const mqa_kv_layout* L, int variant) {
  if (variant == MQA_VARIANT_AUTO) return L->cache_dtype == MQA_F32 ? MQA_VARIANT_CUDA_CORE : MQA_VARIANT_TENSOR_CORE;
  return variant;
}

// Which cache dtypes a kernel family reads: tensor cores bf16, uint8, fp8
// e5m2 and 4 bit, CUDA cores bf16 and fp32.
bool variant_supports(int variant, int cache_dtype) {
  if (variant == MQA_VARIANT_TENSOR_CORE)
    return cache_dtype == MQA_BF16 || cache_dtype == MQA_U8 || cache_dtype == MQA_FP8_E5M2 || cache_dtype == MQA_U4;
  return cache_dtype == MQA_BF16 || cache_dtype == MQA_F32;
}

int dtype_code(int cache_dtype) {
  switch (cache_dtype) {
    case MQA_BF16: return kDtypeBf16;
    case MQA_F32: return kDtypeF32;
    case MQA_U8: return kDtypeU8;
    case MQA_U4: return kDtypeU4;
    default: return kDtypeF8;
  }
}

// one-byte caches: uint8 codes with (scale, zero) rows, or fp8 e5m2
bool byte_cache(int cache_dtype) { return cache_dtype == MQA_U8 || cache_dtype == MQA_FP8_E5M2; }

struct DeviceInfo {
  int sms = 0;
  int smem_per_sm = 0;
  int threads_per_sm = 0;
};

DeviceInfo device_info(int dev) {
  static std::mutex mu;
  static DeviceInfo cache[64];
  std::lock_guard<std::mutex> lock(mu);
  DeviceInfo& d = cache[dev & 63];
  if (d.sms == 0) {
    cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&d.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
    cudaDeviceGetAttribute(&d.threads_per_sm, cudaDevAttrMaxThreadsPerMultiProcessor, dev);
    if (d.sms <= 0) d.sms = 1;
  }
  return d;
}

// Query rows per kv head from which the tensor-memory (tcgen05) kernel takes
// the decode attention: 16-row mma.sync tiles run out of latency hiding there
// (MQA's G = 32, several new tokens per sequence).
constexpr int kTc05MinRows = 32;

// Contiguous bf16 caches; paged bf16 pools with several new tokens per
// sequence (a one-token paged step keeps the warp-MMA kernels); contiguous fp8
// e5m2 caches with several new tokens per sequence (the kernel's fp8 form: the
// code tiles enter the MMAs as they are; a one-token e5m2 MQA step takes
// attn_tc05_widen.cu, measured faster there).
bool use_tc05(const mqa_kv_layout* L, int variant, int n_new) {
  if (variant != MQA_VARIANT_TENSOR_CORE || L->head_dim != 128) return false;
  if ((L->h_q / L->h_kv) * n_new < kTc05MinRows) return false;
  if (L->cache_dtype == MQA_BF16) return !L->paged || n_new > 1;
  return L->cache_dtype == MQA_FP8_E5M2 && !L->paged && n_new > 1;
}


// n_new: query tokens per sequence; a kv head then has G x n_new query rows.
KernelShape decode_shape(const mqa_kv_layout* L, int variant, int n_new = 1) {
  const int G = L->h_q / L->h_kv;
  if (use_tc05(L, variant, n_new)) return tc05_shape();
  if (variant == MQA_VARIANT_TENSOR_CORE && byte_cache(L->cache_dtype))
    return !tc05_keys_applies(G, n_new, L->head_dim, L->paged)
               ? decode_u8_shape(L->head_dim, G * n_new, L->cache_dtype == MQA_FP8_E5M2)
               : (L->cache_dtype == MQA_U8 ? tc05_keys_shape() : tc05_widen_shape());
  if (variant == MQA_VARIANT_TENSOR_CORE) return decode_mma_shape(L->head_dim, G * n_new);
  return decode_fma_shape(L->cache_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32, L->head_dim, G);
}

int head_blocks(const mqa_kv_layout* L, const KernelShape& ks, int n_new = 1) {
  const int rows = (L->h_q / L->h_kv) * n_new;
  return (rows + ks.heads_per_cta - 1) / ks.heads_per_cta;
}


// Multi-token decode runs on the tensor-core kernels: bf16 (warp-MMA or
// tcgen05), uint8 and e5m2 (the one-byte warp-MMA kernel, or the tcgen05
// kernel's fp8 form for 32 or more rows per kv head over a contiguous e5m2
// cache).
bool multi_supported(const mqa_kv_layout* L, int variant, int n_new) {
  return n_new == 1 || (variant == MQA_VARIANT_TENSOR_CORE && (L->cache_dtype == MQA_BF16 || L->cache_dtype == MQA_U4 ||
                                                               byte_cache(L->cache_dtype)));
}

// A 4-bit cache: one block takes a unit (sequence, kv head, block of query rows),
// or all resident blocks share all tiles (attn_u4.cu); then the workspace holds
// a counter and two partial results for each block.
struct U4Plan {
  U4Shape shape;
  int row_blocks;
  int ctas;
  size_t counters;   // bytes at the start of the workspace
  size_t workspace;
};

constexpr int kWholeTiles = 128;  // (see choose_splits)

U4Plan u4_plan(const mqa_kv_layout* L, int n_new) {
  int dev = 0;
  cudaGetDevice(&dev);
  U4Plan c;
  const int rows = (L->h_q / L->h_kv) * n_new;
  c.shape = u4_shape(rows);
  c.row_blocks = (rows + c.shape.rows - 1) / c.shape.rows;
  c.ctas = device_info(dev).sms * c.shape.ctas_per_sm;
  c.counters = (static_cast<size_t>(c.ctas) * 4 + 255) / 256 * 256;
  c.workspace = c.counters + static_cast<size_t>(2) * c.ctas * u4_part_floats(c.shape.rows, L->head_dim) * 4;
  return c;
}

// Tokens one (sequence, kv head) may need read: the bound, or with a sliding
// window W the window plus the alignment of its start down to a tile.
int read_span(const mqa_kv_layout* L, int max_len, int n_new = 1) {
  if (L->window > 0 && L->window + kTile + n_new - 1 < max_len) return L->window + kTile + n_new - 1;
  return max_len;
}

// Token-axis split count. Blocks of one (sequence, kv head) are independent,
// so the only reasons to split are (a) too few units to fill the GPU in one
// wave, and (b) device-side lengths that may vary up to max_seq_len, where
// bounded chunks keep long sequences from finishing last. Measured on GB300:
// a single wave of equal blocks streams best (more, smaller blocks add
// partial-output traffic and a second wave), and 4096-token chunks balance a
// paged batch of lengths spread over [128, 16384].
int choose_splits(const mqa_kv_layout* L, int max_len_in, int variant, int n_new = 1) {
  if (L->cache_dtype == MQA_U4) {
    // One block for each unit, where the others' merging would cost more than its unequal load: for units of few tiles
    // (a tile's time goes with its dims and rows; head_dim 128 and 8 rows: 8 units of 16 tiles 10.0 us, shared 10.4, of 32
    // tiles 15.6 and 11.6; 160 units of 16 tiles 12.4 and 14.5), and for contiguous caches with units for more than half of
    // the blocks and a bound of up to kWholeTiles tiles (the lengths of a paged batch are taken as unequal). The lengths are
    // not known here. 32 x 8 units, equal / spread evenly up to the bound / one of the bound and the others of 1000 tokens, us:
    //   64 tiles    32 and 37 shared    29 and 42    27 and 25     .. of 32 rows    87 and 88    73 and 109     71 and 40 (others of 300)
    //   128 tiles   56 and 62           48 and 58    46 and 29                     161 and 163  152 and 204    132 and 53
    //   256 tiles  105 and 103          98 and 82    84 and 34                     304 and 305  296 and 218    245 and 60
    //   2048 tiles, one of the bound: 616 and 58. (16 rows are between; units past a whole number of waves, 464 of 64 tiles:
    //   65 and 58, 456 of them 46 and 48.)
    const U4Plan c = u4_plan(L, n_new);
    long long span = max_len_in;
    if (L->window > 0) span = std::min(span, static_cast<long long>(L->window) + n_new - 1 + kU4Tile - 1);
    const long long tiles = (span + kU4Tile - 1) / kU4Tile;
    if (tiles * L->head_dim * c.shape.rows <= 16 * 128 * 8) return 1;
    return !L->paged && tiles <= kWholeTiles && 2ll * L->batch * L->h_kv * c.row_blocks > c.ctas ? 1 : 2;
  }
  const int max_len = read_span(L, max_len_in);
  int dev = 0;
  cudaGetDevice(&dev);
  const DeviceInfo di = device_info(dev);
  const KernelShape ks = decode_shape(L, variant, n_new);
  const int by_smem = ks.smem_bytes > 0 ? di.smem_per_sm / (ks.smem_bytes + 1024) : 8;
  const int by_threads = di.threads_per_sm / ks.threads;
  int per_sm = std::max(1, std::min(by_smem, by_threads));
  if (ks.max_ctas_per_sm > 0) per_sm = std::min(per_sm, ks.max_ctas_per_sm);
  const long long slots = static_cast<long long>(di.sms) * per_sm;
  const long long units = static_cast<long long>(L->batch) * L->h_kv * head_blocks(L, ks, n_new);
  const int tiles = (max_len + kTile - 1) / kTile;
  int s = 1;
  if (L->paged) {
    const int chunk_tiles = 65;  // 4096 tokens, plus one tile for a window's unaligned start
    s = (tiles + chunk_tiles - 1) / chunk_tiles;
  } else if (units < slots) {
    s = static_cast<int>(slots / units);  // at most one wave
  }
  return std::max(1, std::min(s, tiles));
}

// Effective split count and chunk for a requested count (a 4-bit cache: one, or
// more than one, which stands for shared tiles).
void split_plan(const mqa_kv_layout* L, int requested, int max_len, int* splits, int* chunk) {
  if (L->cache_dtype == MQA_U4) {
    *splits = requested > 1 ? 2 : 1;
    *chunk = 0;
    return;
  }
  const int per = (max_len + requested - 1) / requested;
  const int c = ((per + kTile - 1) / kTile) * kTile;
  *chunk = c;
  *splits = (max_len + c - 1) / c;
}

size_t partial_bytes(const mqa_kv_layout* L, int splits, int n_new = 1) {
  if (splits <= 1) return 0;
  if (L->cache_dtype == MQA_U4) return u4_plan(L, n_new).workspace;
  const size_t rows = static_cast<size_t>(L->batch) * n_new * L->h_q;
  const size_t o_bytes = ((rows * splits * L->head_dim * 4) + 255) / 256 * 256;
  return o_bytes + rows * splits * 4;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// q_rot [batch n_new tokens][h_q][128] fp32 for the prefill kernel: a box is
// `rows` consecutive rows (group) of one kv head, i.e. rows / group tokens x
// the group's heads x 128 dims, unswizzled (512-byte rows).
bool make_q_map(CUtensorMap* map, const float* q_rot, int batch, int n_new, int h_q, int group, int rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(h_q), static_cast<cuuint64_t>(batch) * n_new};
  const cuuint64_t strides[2] = {128 * 4, static_cast<cuuint64_t>(h_q) * 128 * 4};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(rows / group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(q_rot), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// attn_tc05_kernel reading q_rot (not a fused step) with full 128-row blocks
// (prefill, many new tokens): when the group divides 64, a block's rows come
// as two boxes of 64 rows (p->q_tma set); else, and for fewer rows, the
// kernel reads them with plain loads. False only if the encoder fails.
bool tc05_q_map(Tc05Params* p, CUtensorMap* tq) {
  p->q_tma = 0;
  if (p->fuse || p->q_rot == nullptr || p->group > 64 || (p->group & (p->group - 1)) != 0 ||
      static_cast<long long>(p->group) * p->n_new < 128)
    return true;
  if (!make_q_map(tq, p->q_rot, p->batch, p->n_new, p->h_q, p->group, 64)) return false;
  p->q_tma = 1;
  return true;
}

// TMA descriptors for the tensor-core path: 128-byte swizzled boxes of
// 64 columns, kTile rows (contiguous) or one page (paged, pages shorter than
// a tile). With `merged`, head_dim 128 is described as 64 columns x 2 halves
// where the half dimension has the smaller stride (128 bytes) than the row
// (256 bytes): one box then carries both halves of its rows and lands in
// shared memory as two 64-column spans, so a tile needs half as many copies.
// `heads` > 1 (paged, merged only): a box also spans that many consecutive kv
// heads of one page, which are contiguous in the pool.
bool make_tensor_map(CUtensorMap* map, void* base, const mqa_kv_layout* L, bool merged, int heads = 1,
                     int box_rows = 0) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t D = L->head_dim;
  const cuuint64_t row_bytes = D * 2;
  cuuint64_t dims[5];
  cuuint64_t strides[4];
  cuuint32_t box[5];
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const cuuint32_t rows = box_rows > 0 ? static_cast<cuuint32_t>(box_rows)
                                       : static_cast<cuuint32_t>(L->paged ? (L->page_size < kTile ? L->page_size : kTile)
                                                                          : kTile);
  const cuuint64_t outer_rows = L->paged ? static_cast<cuuint64_t>(L->page_size) : static_cast<cuuint64_t>(L->capacity);
  cuuint32_t rank;
  if (merged) {
    dims[0] = 64;
    dims[1] = outer_rows;
    dims[2] = D / 64;
    strides[0] = row_bytes;
    strides[1] = 128;
    box[0] = 64;
    box[1] = rows;
    box[2] = static_cast<cuuint32_t>(D / 64);
    if (!L->paged) {
      rank = 4;
      dims[3] = static_cast<cuuint64_t>(L->batch) * L->h_kv;
      strides[2] = static_cast<cuuint64_t>(L->capacity) * row_bytes;
      box[3] = 1;
    } else {
      rank = 5;
      dims[3] = static_cast<cuuint64_t>(L->h_kv);
      dims[4] = static_cast<cuuint64_t>(L->num_pages);
      strides[2] = static_cast<cuuint64_t>(L->page_size) * row_bytes;
      strides[3] = static_cast<cuuint64_t>(L->h_kv) * L->page_size * row_bytes;
      box[3] = static_cast<cuuint32_t>(heads);
      box[4] = 1;
    }
  } else {
    dims[0] = D;
    dims[1] = outer_rows;
    strides[0] = row_bytes;
    box[0] = 64;
    box[1] = rows;
    if (!L->paged) {
      rank = 3;
      dims[2] = static_cast<cuuint64_t>(L->batch) * L->h_kv;
      strides[1] = static_cast<cuuint64_t>(L->capacity) * row_bytes;
      box[2] = 1;
    } else {
      rank = 4;
      dims[2] = static_cast<cuuint64_t>(L->h_kv);
      dims[3] = static_cast<cuuint64_t>(L->num_pages);
      strides[1] = static_cast<cuuint64_t>(L->page_size) * row_bytes;
      strides[2] = static_cast<cuuint64_t>(L->h_kv) * L->page_size * row_bytes;
      box[2] = 1;
      box[3] = 1;
    }
  }
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// TMA descriptors of a uint8 cache: maps[0], maps[1] the K / V codes (boxes
// of head_dim x `rows` rows x `heads` kv heads; 128-byte swizzle for 128-byte
// rows, 64-byte swizzle for 64-byte rows), maps[2], maps[3] their (scale,
// zero) rows as float32 runs of 2 x `rows` values per head. `heads` > 1 only
// for paged pools, where the heads of one page are consecutive.
bool make_u8_maps(CUtensorMap* maps, const mqa_kv_layout* L, int rows_in, int heads) {
  const bool f8 = L->cache_dtype == MQA_FP8_E5M2;  // codes only: the (scale, zero) maps repeat the code maps
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t D = L->head_dim;
  const cuuint32_t rows = static_cast<cuuint32_t>(rows_in);
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle swz = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  void* codes[2] = {L->k_cache, L->v_cache};
  void* sz[2] = {L->k_scale_zero, L->v_scale_zero};
  for (int i = 0; i < 2; ++i) {
    cuuint64_t dims[4], strides[3];
    cuuint32_t box[4];
    cuuint32_t rank;
    dims[0] = D;
    box[0] = static_cast<cuuint32_t>(D);
    box[1] = rows;
    strides[0] = D;
    if (!L->paged) {
      rank = 3;
      dims[1] = static_cast<cuuint64_t>(L->capacity);
      dims[2] = static_cast<cuuint64_t>(L->batch) * L->h_kv;
      strides[1] = static_cast<cuuint64_t>(L->capacity) * D;
      box[2] = 1;
    } else {
      rank = 4;
      dims[1] = static_cast<cuuint64_t>(L->page_size);
      dims[2] = static_cast<cuuint64_t>(L->h_kv);
      dims[3] = static_cast<cuuint64_t>(L->num_pages);
      strides[1] = static_cast<cuuint64_t>(L->page_size) * D;
      strides[2] = static_cast<cuuint64_t>(L->h_kv) * L->page_size * D;
      box[2] = static_cast<cuuint32_t>(heads);
      box[3] = 1;
    }
    if (fn(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, codes[i], dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  if (f8) {
    maps[2] = maps[0];
    maps[3] = maps[1];
    return true;
  }
  for (int i = 0; i < 2; ++i) {
    cuuint64_t dims[3], strides[2];
    cuuint32_t box[3];
    cuuint32_t rank;
    box[0] = 2 * rows;
    if (!L->paged) {
      rank = 2;
      dims[0] = 2 * static_cast<cuuint64_t>(L->capacity);
      dims[1] = static_cast<cuuint64_t>(L->batch) * L->h_kv;
      strides[0] = 2 * static_cast<cuuint64_t>(L->capacity) * 4;
      box[1] = 1;
    } else {
      rank = 3;
      dims[0] = 2 * static_cast<cuuint64_t>(L->page_size);
      dims[1] = static_cast<cuuint64_t>(L->h_kv);
      dims[2] = static_cast<cuuint64_t>(L->num_pages);
      strides[0] = 2 * static_cast<cuuint64_t>(L->page_size) * 4;
      strides[1] = static_cast<cuuint64_t>(L->h_kv) * strides[0];
      box[1] = static_cast<cuuint32_t>(heads);
      box[2] = 1;
    }
    if (fn(&maps[2 + i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, rank, sz[i], dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

// Tensor maps of the tcgen05 kernel's K / V tiles: bf16 tiles, or the fp8
// kernel's code tiles (t->f8 set).
// TMA descriptor of a paged bf16 pool for the tcgen05 kernel: dims (64 dims,
// page rows, the two 64-dim halves, kv heads, pages), box 64 x rp x 1 x 1 x 1
// with rp = min(page_size, 64), 128-byte swizzle: one copy per (page run,
// half), landing at the tile's half and row offset.
bool make_tc05_paged_map(CUtensorMap* map, void* base, const mqa_kv_layout* L) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t row_bytes = 256, ps = static_cast<cuuint64_t>(L->page_size);
  const cuuint64_t dims[5] = {64, ps, 2, static_cast<cuuint64_t>(L->h_kv), static_cast<cuuint64_t>(L->num_pages)};
  const cuuint64_t strides[4] = {row_bytes, 128, ps * row_bytes, static_cast<cuuint64_t>(L->h_kv) * ps * row_bytes};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(L->page_size < 64 ? L->page_size : 64), 1, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool tc05_maps(const mqa_kv_layout* L, Tc05Params* t, CUtensorMap* tk, CUtensorMap* tv) {
  if (L->paged) {
    t->paged = 1;
    t->page_size = L->page_size;
    t->max_pages = L->max_pages_per_seq;
    t->num_pages = L->num_pages;
    t->block_table = L->block_table;
    t->capacity = token_limit(L);
    return make_tc05_paged_map(tk, L->k_cache, L) && make_tc05_paged_map(tv, L->v_cache, L);
  }
  if (L->cache_dtype == MQA_FP8_E5M2) {
    CUtensorMap maps[4];
    if (!make_u8_maps(maps, L, tc05_f8_box_rows(), 1)) return false;
    *tk = maps[0];
    *tv = maps[1];
    t->f8 = 1;
    return true;
  }
  return make_tensor_map(tk, L->k_cache, L, true, 1, 128) && make_tensor_map(tv, L->v_cache, L, true, 1, 128);
}

void fill_theta(double* theta, int head_dim, double base) {
  for (int i = 0; i < head_dim / 2; ++i)
    theta[i] = std::pow(base, -2.0 * static_cast<double>(i) / static_cast<double>(head_dim));
}

mqa_status check_append_args(const mqa_kv_layout* layout, const void* q_new, const void* k_new, const void* v_new,
                             const int32_t* pos, double rope_base, const float* q_rot, const int32_t* err_word) {
  const mqa_status st = check_layout(layout);
  if (st != MQA_OK) return st;
  if (!q_new || !k_new || !v_new || !pos || !q_rot || !err_word) return MQA_ERR_INVALID_ARG;
  if (!aligned(q_new, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_rot, 16) ||
      !aligned(pos, 4) || !aligned(err_word, 4))
    return MQA_ERR_INVALID_ARG;
  if (!(rope_base > 0.0) || !std::isfinite(rope_base)) return MQA_ERR_INVALID_ARG;
  return MQA_OK;
}

// A tree's append: the nodes' depths and counts, and the counters to clear.
struct TreeAppend {
  const int32_t* depth;
  const int32_t* num_nodes;
  int32_t* zero;
  int zero_count;
};

// after the checks; options NULL: no norm, one position. zero: counters to
// clear for the attention launch that follows.
mqa_status norm_append(const mqa_kv_layout* layout, int n_new, const void* q_new, const void* k_new, const void* v_new,
                       const int32_t* pos, const mqa_norm_rope* options, double rope_base, float* q_rot, int32_t* zero,
                       int zero_count, int32_t* err_word, cudaStream_t stream) {
  // (a block's tokens are counted past the last one)
  if (static_cast<long long>(layout->batch) * n_new > (1ll << 31) - 64) return MQA_ERR_INVALID_ARG;
  NormAppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.batch = layout->batch;
  p.h_q = layout->h_q;
  p.h_kv = layout->h_kv;
  p.head_dim = layout->head_dim;
  p.cache_dtype = dtype_code(layout->cache_dtype);
  p.paged = layout->paged;
  p.n_new = n_new;
  p.q_new = q_new;
  p.k_new = k_new;
  p.v_new = v_new;
  p.pos = pos;
  p.eps = 1.f;
  if (options != nullptr) {
    p.q_weight = options->q_weight;
    p.k_weight = options->k_weight;
    if (p.q_weight || p.k_weight) p.eps = options->eps;
    if (options->n_axes > 0) {
      p.axis_pos = options->axis_pos;
      int end = 0;
      for (int a = 0; a < kMaxAxes; ++a) p.section_end[a] = end += a < options->n_axes ? options->section[a] : 0;
    }
  }
  p.k_cache = layout->k_cache;
  p.v_cache = layout->v_cache;
  p.capacity = layout->capacity;
  p.page_size = layout->page_size;
  p.num_pages = layout->num_pages;
  p.max_pages = layout->max_pages_per_seq;
  p.block_table = layout->block_table;
  p.k_sz = layout->k_scale_zero;
  p.v_sz = layout->v_scale_zero;
  p.q_rot = q_rot;
  p.err = err_word;
  p.zero = zero;
  p.zero_count = zero_count;
  fill_theta(p.theta, layout->head_dim, rope_base);
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = launch_append_norm(p, device_info(dev).sms, stream);
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

mqa_status append_impl(const mqa_kv_layout* layout, const void* q_new, const void* k_new, const void* v_new,
                       const int32_t* pos, double rope_base, float* q_rot, int32_t* err_word, mqa_stream_t stream,
                       int n_new = 1, const TreeAppend* tree = nullptr, int32_t* zero = nullptr, int zero_count = 0) {
  const mqa_status st = check_append_args(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word);
  if (st != MQA_OK) return st;
  if (n_new < 1 || static_cast<long long>(layout->batch) * n_new > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  if (layout->cache_dtype == MQA_U4)
    return norm_append(layout, n_new, q_new, k_new, v_new, pos, nullptr, rope_base, q_rot, zero, zero_count, err_word,
                       reinterpret_cast<cudaStream_t>(stream));
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.n_new = n_new;
  p.batch = layout->batch;
  p.h_q = layout->h_q;
  p.h_kv = layout->h_kv;
  p.head_dim = layout->head_dim;
  p.cache_dtype = dtype_code(layout->cache_dtype);
  p.paged = layout->paged;
  p.k_sz = static_cast<float2*>(layout->k_scale_zero);
  p.v_sz = static_cast<float2*>(layout->v_scale_zero);
  p.q_new = q_new;
  p.k_new = k_new;
  p.v_new = v_new;
  p.pos = pos;
  p.k_cache = layout->k_cache;
  p.v_cache = layout->v_cache;
  p.capacity = layout->capacity;
  p.page_size = layout->page_size;
  p.num_pages = layout->num_pages;
  p.max_pages = layout->max_pages_per_seq;
  p.block_table = layout->block_table;
  p.q_rot = q_rot;
  p.err = err_word;
  if (tree != nullptr) {
    p.depth = tree->depth;
    p.num_nodes = tree->num_nodes;
    p.zero = tree->zero;
    p.zero_count = tree->zero_count;
  }
  fill_theta(p.theta, layout->head_dim, rope_base);
  // few nodes: the blocks of append_rope.cu, which split a node's heads (a step of 8
  // nodes takes 17.0 us with them, 17.9 with append_tree.cu's; of 64 20.0 and 19.4, of
  // 256 40.2 and 39.8; the append alone of 2048 21.7 and 11.6)
  const bool wide = tree != nullptr && layout->cache_dtype == MQA_BF16 && p.batch * p.n_new >= kTreeAppendNodes;
  int dev = 0;
  if (wide) cudaGetDevice(&dev);
  const cudaError_t e = wide ? launch_append_tree(p, device_info(dev).sms, reinterpret_cast<cudaStream_t>(stream))
                            : launch_append_rope(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

// The raw new-token query and its positions, when the attention launch
// directly follows the append launch (fused step): the tensor-core kernels
// then rotate q themselves instead of waiting for q_rot.
struct RopeArgs {
  const void* q_new;
  const int32_t* pos;
  double rope_base;
  int fuse_append;  // 1: no append launch precedes; the decode kernel appends k_new / v_new itself
  const void* k_new;
  const void* v_new;
  float* q_rot;
};

// The tensor-core kernels can take the append over when one block sees all
// query heads of its kv head (warp-MMA kernels: G <= 32; tcgen05: one
// 128-row block). One-byte caches: the warp-MMA kernels (decode_u8_kernel
// with one head block, the paged head-group kernel) and the one-token MQA
// kernels (attn_tc05_keys.cu for uint8, attn_tc05_widen.cu for e5m2).
bool fusable(const mqa_kv_layout* L, int variant) {
  if (variant != MQA_VARIANT_TENSOR_CORE) return false;
  if (byte_cache(L->cache_dtype)) {
    const int G = L->h_q / L->h_kv;
    if (tc05_keys_applies(G, 1, L->head_dim, L->paged)) return true;
    return head_blocks(L, decode_shape(L, variant)) == 1;
  }
  if (L->cache_dtype != MQA_BF16) return false;
  if (use_tc05(L, variant, 1)) return L->h_q / L->h_kv <= 128;  // one row block
  return head_blocks(L, decode_shape(L, variant)) == 1;
}

// Several new tokens per sequence (bf16 cache): the attention kernel takes the
// appends over when one block sees all (token, head) rows of its kv head --
// tcgen05: at most 128 rows; warp-MMA: one head block, and the tokens' cos /
// sin tables fit (at most kMaxFusedNewTokens).
bool fusable_multi(const mqa_kv_layout* L, int variant, int n_new) {
  if (variant != MQA_VARIANT_TENSOR_CORE || L->cache_dtype != MQA_BF16 || n_new < 2) return false;
  // tcgen05: one row block of 128 (token, head) rows, and at most
  // kMaxFusedNewTokensTc05 tokens: the block's append warp turns every new
  // key pair with an fp64-reduced angle, which past that outlasts the stream
  // of keys it hides behind (gqa4k, step vs append + attention: n = 8 90.8 vs
  // 100.0 us, n = 16 100.4 vs 106.4, n = 32 148 vs 113.6)
  if (use_tc05(L, variant, n_new)) return (L->h_q / L->h_kv) * n_new <= 128 && n_new <= kMaxFusedNewTokensTc05;
  if (n_new > kMaxFusedNewTokens) return false;
  return head_blocks(L, decode_shape(L, variant, n_new), n_new) == 1;
}

// V codes of a 4-bit cache: boxes of whole rows x min(kU4Tile, page_size) tokens,
// swizzled over a row's bytes, so that the 8 rows of an ldmatrix lie in different banks.
bool make_u4_map(CUtensorMap* map, const mqa_kv_layout* L) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t row = L->head_dim / 2, rows = L->paged ? static_cast<cuuint64_t>(L->page_size) : static_cast<cuuint64_t>(L->capacity);
  const cuuint64_t heads = L->paged ? static_cast<cuuint64_t>(L->h_kv) : static_cast<cuuint64_t>(L->batch) * L->h_kv;
  const cuuint64_t dims[4] = {row, rows, heads, static_cast<cuuint64_t>(L->num_pages)};
  const cuuint64_t strides[3] = {row, rows * row, rows * row * heads};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(row), static_cast<cuuint32_t>(L->paged ? std::min(L->page_size, kU4Tile) : kU4Tile), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, L->paged ? 4 : 3, L->v_cache, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// after attention_impl's checks
mqa_status u4_attention(const mqa_kv_layout* L, int n_new, const float* q_rot, const int32_t* seq_lens, int max_seq_len,
                        float scale, bool whole, void* out, int out_dtype, float* lse_out, void* workspace,
                        int32_t* err_word, cudaStream_t stream, int early) {
  const U4Plan c = u4_plan(L, n_new);
  if (whole && static_cast<long long>(L->batch) * L->h_kv * c.row_blocks > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  U4Params p;
  std::memset(&p, 0, sizeof(p));
  p.batch = L->batch;
  p.h_q = L->h_q;
  p.h_kv = L->h_kv;
  p.group = L->h_q / L->h_kv;
  p.n_new = n_new;
  p.rows = p.group * n_new;
  p.head_dim = L->head_dim;
  p.row_blocks = c.row_blocks;
  p.paged = L->paged;
  p.page_size = L->page_size;
  p.num_pages = L->num_pages;
  p.max_pages = L->max_pages_per_seq;
  p.k_cache = static_cast<const uint8_t*>(L->k_cache);
  p.v_cache = static_cast<const uint8_t*>(L->v_cache);
  p.k_sm = static_cast<const uint32_t*>(L->k_scale_zero);
  p.v_sm = static_cast<const uint32_t*>(L->v_scale_zero);
  p.capacity = L->capacity;
  p.block_table = L->block_table;
  p.max_seq_len = max_seq_len;
  p.q_rot = q_rot;
  p.seq_lens = seq_lens;
  p.scale = scale;
  p.window = L->window;
  p.out = out;
  p.out_dtype = out_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  p.lse_out = lse_out;
  p.whole = whole;
  p.parts = static_cast<int>(c.ctas / (static_cast<long long>(L->batch) * L->h_kv * c.row_blocks));
  p.arrived = static_cast<int32_t*>(workspace);
  p.part = whole ? nullptr : reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + c.counters);
  p.err = err_word;
  p.early = early;
  p.wait_ns = wait_limit(L);
  CUtensorMap tv;
  if (!make_u4_map(&tv, L)) {
    snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
    return MQA_ERR_CUDA;
  }
  const cudaError_t e = launch_attn_u4(p, tv, c.ctas, /*clear=*/!whole && !early, stream);
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

mqa_status attention_impl(const mqa_kv_layout* layout, const float* q_rot, const int32_t* seq_lens, int32_t max_seq_len,
                          float scale, int32_t num_splits, void* out, int32_t out_dtype, float* lse_out,
                          void* workspace, size_t workspace_bytes, int32_t variant, int32_t* err_word,
                          mqa_stream_t stream, int early, const RopeArgs* rope, int n_new = 1, int prefill = 0) {
  const mqa_status st = check_layout(layout);
  if (st != MQA_OK) return st;
  // (prefill over a one-byte cache takes this path with the whole prompt)
  if (n_new < 1 || (!prefill && n_new > kMaxNewTokens)) return MQA_ERR_INVALID_ARG;
  if (static_cast<long long>(layout->batch) * n_new * layout->h_q > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  if (!q_rot || !seq_lens || !out || !err_word) return MQA_ERR_INVALID_ARG;
  if (!aligned(q_rot, 16) || !aligned(seq_lens, 4) || !aligned(out, 16) || !aligned(err_word, 4) ||
      (lse_out && !aligned(lse_out, 4)))
    return MQA_ERR_INVALID_ARG;
  if (max_seq_len < n_new || max_seq_len > token_limit(layout)) return MQA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || num_splits < 0) return MQA_ERR_INVALID_ARG;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  if (variant < MQA_VARIANT_AUTO || variant > MQA_VARIANT_TENSOR_CORE) return MQA_ERR_INVALID_ARG;
  const int v = resolve_variant(layout, variant);
  if (!variant_supports(v, layout->cache_dtype) || !multi_supported(layout, v, n_new)) return MQA_ERR_UNSUPPORTED;

  const int req = num_splits == 0 ? choose_splits(layout, max_seq_len, v, n_new) : num_splits;
  int splits, chunk;
  split_plan(layout, req, read_span(layout, max_seq_len, n_new), &splits, &chunk);
  const size_t need = partial_bytes(layout, splits, n_new);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return MQA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MQA_ERR_INVALID_ARG;
  }

  if (layout->cache_dtype == MQA_U4)
    return u4_attention(layout, n_new, q_rot, seq_lens, max_seq_len, scale, splits == 1, out, out_dtype, lse_out,
                        workspace, err_word, reinterpret_cast<cudaStream_t>(stream), early);

  const KernelShape ks = decode_shape(layout, v, n_new);
  bool merged = false;  // the attention launch merged its splits itself: no combine
  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.n_new = n_new;
  p.batch = layout->batch;
  p.h_q = layout->h_q;
  p.h_kv = layout->h_kv;
  p.group = layout->h_q / layout->h_kv;
  p.head_dim = layout->head_dim;
  p.cache_dtype = dtype_code(layout->cache_dtype);
  p.paged = layout->paged;
  p.k_cache = layout->k_cache;
  p.k_sz = static_cast<const float2*>(layout->k_scale_zero);
  p.v_sz = static_cast<const float2*>(layout->v_scale_zero);
  p.v_cache = layout->v_cache;
  p.capacity = layout->capacity;
  p.page_size = layout->page_size;
  p.num_pages = layout->num_pages;
  p.max_pages = layout->max_pages_per_seq;
  p.block_table = layout->block_table;
  p.q_rot = q_rot;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.num_splits = splits;
  p.chunk = chunk;
  p.head_blocks = head_blocks(layout, ks, n_new);
  p.window = layout->window;
  p.early = early;
  p.wait_ns = wait_limit(layout);
  // (one-byte caches and several new tokens: only in the fused step;
  // otherwise q_rot comes from the append launch)
  if (rope != nullptr && v == MQA_VARIANT_TENSOR_CORE &&
      ((n_new == 1 && (layout->cache_dtype == MQA_BF16 || (byte_cache(layout->cache_dtype) && rope->fuse_append))) ||
       (n_new > 1 && rope->fuse_append))) {
    p.rope_q = 1;
    p.q_new = rope->q_new;
    p.pos = rope->pos;
    fill_theta(p.theta, layout->head_dim, rope->rope_base);
    if (rope->fuse_append) {
      p.fuse_append = 1;
      p.early = 0;  // nothing of this step precedes the launch
      p.k_new = rope->k_new;
      p.v_new = rope->v_new;
      p.q_rot_out = rope->q_rot;
    }
  }
  p.out = out;
  p.out_dtype = out_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  p.lse_out = lse_out;
  p.err = err_word;
  if (splits > 1) {
    const size_t rows = static_cast<size_t>(layout->batch) * n_new * layout->h_q;
    const size_t o_bytes = ((rows * splits * layout->head_dim * 4) + 255) / 256 * 256;
    p.o_part = static_cast<float*>(workspace);
    p.lse_part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + o_bytes);
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (use_tc05(layout, v, n_new)) {
    Tc05Params t;
    std::memset(&t, 0, sizeof(t));
    t.batch = layout->batch;
    t.h_q = layout->h_q;
    t.h_kv = layout->h_kv;
    t.group = p.group;
    t.n_new = n_new;
    t.row_blocks = (p.group * n_new + 127) / 128;
    t.num_splits = splits;
    t.chunk = chunk;
    t.k_cache = layout->k_cache;
    t.v_cache = layout->v_cache;
    t.capacity = layout->capacity;
    t.max_seq_len = max_seq_len;
    t.seq_lens = seq_lens;
    t.q_rot = q_rot;
    t.scale_log2 = p.scale_log2;
    t.window = layout->window;
    t.out = out;
    t.out_dtype = p.out_dtype;
    t.lse_out = lse_out;
    t.o_part = p.o_part;
    t.lse_part = p.lse_part;
    t.err = err_word;
    t.early = early;
    t.wait_ns = p.wait_ns;
    if (rope != nullptr && rope->fuse_append) {  // (fusable: one row block)
      t.fuse = 1;
      t.early = 0;  // nothing of this step precedes the launch
      t.q_new = rope->q_new;
      t.k_new = rope->k_new;
      t.v_new = rope->v_new;
      t.pos = rope->pos;
      t.q_rot_out = rope->q_rot;
      fill_theta(t.theta, layout->head_dim, rope->rope_base);
    }
    CUtensorMap tk, tv, tq;
    if (!tc05_maps(layout, &t, &tk, &tv) || !tc05_q_map(&t, &tq)) {
      snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
      return MQA_ERR_CUDA;
    }
    e = launch_tc05_attention(t, tk, tv, &tq, s);
    if (e != cudaSuccess) return fail_cuda(e);
    merged = tc05_merges_splits(t);
    goto combine;
  }
  if (v == MQA_VARIANT_TENSOR_CORE && byte_cache(layout->cache_dtype) &&
      tc05_keys_applies(p.group, n_new, layout->head_dim, layout->paged)) {
    // one-byte MQA step on tcgen05. e5m2: the heads on the MMA rows, converter
    // warps widening the code tiles (attn_tc05_widen.cu); uint8: the keys on
    // the MMA rows (attn_tc05_keys.cu), measured faster for uint8
    CUtensorMap maps[4];
    if (!make_u8_maps(maps, layout, 128, 1)) {
      snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
      return MQA_ERR_CUDA;
    }
    Tc05Params t;
    std::memset(&t, 0, sizeof(t));
    t.batch = layout->batch;
    t.h_q = layout->h_q;
    t.h_kv = layout->h_kv;
    t.group = p.group;
    t.n_new = 1;
    t.row_blocks = 1;
    t.num_splits = splits;
    t.chunk = chunk;
    t.k_cache = layout->k_cache;
    t.v_cache = layout->v_cache;
    t.capacity = layout->capacity;
    t.max_seq_len = max_seq_len;
    t.seq_lens = seq_lens;
    t.q_rot = q_rot;
    t.scale_log2 = p.scale_log2;
    t.window = layout->window;
    t.out = out;
    t.out_dtype = p.out_dtype;
    t.lse_out = lse_out;
    t.o_part = p.o_part;
    t.lse_part = p.lse_part;
    t.err = err_word;
    t.early = early;
    t.wait_ns = p.wait_ns;
    if (rope != nullptr && rope->fuse_append) {
      // one launch: the kernel rotates q_new and encodes the new row itself
      t.fuse = 1;
      t.early = 0;
      t.q_new = rope->q_new;
      t.k_new = rope->k_new;
      t.v_new = rope->v_new;
      t.pos = rope->pos;
      t.q_rot_out = rope->q_rot;
      t.k_sz = static_cast<float2*>(layout->k_scale_zero);
      t.v_sz = static_cast<float2*>(layout->v_scale_zero);
      fill_theta(t.theta, layout->head_dim, rope->rope_base);
    }
    if (layout->cache_dtype == MQA_U8) {
      e = launch_tc05_keys_attention(t, kDtypeU8, maps, s);
    } else {
      e = launch_tc05_widen_attention(t, maps[0], maps[1], s);
      if (e != cudaSuccess) return fail_cuda(e);
      merged = tc05_widen_merges_splits(t);
      goto combine;
    }
  } else if (v == MQA_VARIANT_TENSOR_CORE && byte_cache(layout->cache_dtype)) {
    CUtensorMap maps[4];
    // Paged 16- / 32-token pages: blocks over groups of kv heads, one box per
    // page and head group (long contiguous runs of the pool).
    const int hg = decode_u8_heads_group(p);
    const int rows = hg > 0 ? layout->page_size : (layout->paged && layout->page_size < kTile ? layout->page_size : kTile);
    if (!make_u8_maps(maps, layout, rows, hg > 0 ? hg : 1)) {
      snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
      return MQA_ERR_CUDA;
    }
    e = hg > 0 ? launch_decode_u8_heads(p, hg, maps, s) : launch_decode_u8(p, maps, s);
  } else if (v == MQA_VARIANT_TENSOR_CORE) {
    CUtensorMap tk, tv;
    // Paged 16-token pages: blocks over groups of kv heads, one box per page
    // and head group (long contiguous runs of the pool).
    const int hg = decode_mma_heads_group(p);
    if (hg > 0 && make_tensor_map(&tk, layout->k_cache, layout, true, hg) &&
        make_tensor_map(&tv, layout->v_cache, layout, true, hg)) {
      p.merged_halves = 1;
      p.head_blocks = 1;
      e = launch_decode_mma_heads(p, hg, tk, tv, s);
      if (e != cudaSuccess) return fail_cuda(e);
      goto combine;
    }
    p.merged_halves = layout->head_dim == 128 && make_tensor_map(&tk, layout->k_cache, layout, true) &&
                      make_tensor_map(&tv, layout->v_cache, layout, true);
    if (!p.merged_halves &&
        (!make_tensor_map(&tk, layout->k_cache, layout, false) || !make_tensor_map(&tv, layout->v_cache, layout, false))) {
      snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
      return MQA_ERR_CUDA;
    }
    e = launch_decode_mma(p, tk, tv, s);
  } else {
    e = launch_decode_fma(p, s);
  }
  if (e != cudaSuccess) return fail_cuda(e);
combine:
  if (splits > 1 && !merged) {
    CombineParams c;
    c.o_part = p.o_part;
    c.lse_part = p.lse_part;
    c.rows = layout->batch * n_new * layout->h_q;
    c.num_splits = splits;
    c.head_dim = layout->head_dim;
    c.out = out;
    c.out_dtype = p.out_dtype;
    c.lse_out = lse_out;
    e = launch_combine(c, s);
    if (e != cudaSuccess) return fail_cuda(e);
  }
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

// Causal attention of the last n_new tokens of every sequence on tcgen05
// (prefill): contiguous bf16 cache, head_dim 128.
// Prefill over a uint8 cache, or a paged e5m2 pool: the one-byte warp-MMA
// kernel's multi-token form over the whole prompt (rows = (token, head) pairs,
// 32 per block; every block streams the keys up to its last row).
bool prefill_on_byte_kernel(const mqa_kv_layout* L) {
  return L->cache_dtype == MQA_U8 || (L->cache_dtype == MQA_FP8_E5M2 && L->paged);
}

// The cache types and shapes gqa_prefill_attention takes.
bool prefill_supported(const mqa_kv_layout* L) {
  if (prefill_on_byte_kernel(L)) return L->head_dim == 64 || L->head_dim == 128;
  return (L->cache_dtype == MQA_BF16 || L->cache_dtype == MQA_FP8_E5M2) && L->head_dim == 128;
}

mqa_status prefill_impl(const mqa_kv_layout* layout, int n_new, const float* q_rot, const int32_t* seq_lens,
                        int32_t max_seq_len, float scale, void* out, int32_t out_dtype, float* lse_out,
                        int32_t* err_word, mqa_stream_t stream, int early) {
  const mqa_status st = check_layout(layout);
  if (st != MQA_OK) return st;
  if (!prefill_supported(layout)) return MQA_ERR_UNSUPPORTED;
  if (prefill_on_byte_kernel(layout))
    return attention_impl(layout, q_rot, seq_lens, max_seq_len, scale, /*num_splits=*/1, out, out_dtype, lse_out,
                          nullptr, 0, MQA_VARIANT_TENSOR_CORE, err_word, stream, early, nullptr, n_new,
                          /*prefill=*/1);
  if (n_new < 1 || static_cast<long long>(layout->batch) * n_new > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  if (!q_rot || !seq_lens || !out || !err_word) return MQA_ERR_INVALID_ARG;
  if (!aligned(q_rot, 16) || !aligned(seq_lens, 4) || !aligned(out, 16) || !aligned(err_word, 4) ||
      (lse_out && !aligned(lse_out, 4)))
    return MQA_ERR_INVALID_ARG;
  if (max_seq_len < n_new || max_seq_len > token_limit(layout)) return MQA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return MQA_ERR_INVALID_ARG;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  const long long blocks = static_cast<long long>(layout->batch) * layout->h_kv *
                           ((static_cast<long long>(layout->h_q / layout->h_kv) * n_new + 127) / 128);
  if (blocks > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  Tc05Params p;
  std::memset(&p, 0, sizeof(p));
  p.batch = layout->batch;
  p.h_q = layout->h_q;
  p.h_kv = layout->h_kv;
  p.group = layout->h_q / layout->h_kv;
  p.n_new = n_new;
  p.row_blocks = static_cast<int>((static_cast<long long>(p.group) * n_new + 127) / 128);
  p.num_splits = 1;
  p.chunk = ((max_seq_len + 63) / 64) * 64;
  p.k_cache = layout->k_cache;
  p.v_cache = layout->v_cache;
  p.capacity = layout->capacity;
  p.max_seq_len = max_seq_len;
  p.seq_lens = seq_lens;
  p.q_rot = q_rot;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.window = layout->window;
  p.out = out;
  p.out_dtype = out_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  p.lse_out = lse_out;
  p.err = err_word;
  p.early = early;
  p.wait_ns = wait_limit(layout);
  CUtensorMap tk, tv;
  if (!tc05_maps(layout, &p, &tk, &tv)) {
    snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
    return MQA_ERR_CUDA;
  }
  cudaError_t e;
  {
    // two 128-row query tiles per block sharing every K / V tile (bf16, or
    // e5m2 code tiles in the kernel's fp8 form)
    const int rpb = tc05_prefill_rows_per_block();
    p.row_blocks = static_cast<int>((static_cast<long long>(p.group) * n_new + rpb - 1) / rpb);
    // a block's rows are whole tokens when the group divides them: then they
    // come as one TMA box ([tokens][heads][128] fp32)
    CUtensorMap tq = tk;
    if (p.group <= 256 && (p.group & (p.group - 1)) == 0) {
      if (!make_q_map(&tq, q_rot, layout->batch, n_new, layout->h_q, p.group, rpb)) {
        snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
        return MQA_ERR_CUDA;
      }
      p.q_tma = 1;
    }
    e = launch_tc05_prefill(p, tk, tv, tq, reinterpret_cast<cudaStream_t>(stream));
  }
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

}  // namespace

extern "C" {

mqa_status gqa_prefill_attention(const mqa_kv_layout* layout, int32_t n_new, const float* q_rot,
                                 const int32_t* seq_lens, int32_t max_seq_len, float scale, void* out,
                                 int32_t out_dtype, float* lse_out, int32_t* err_word, mqa_stream_t stream) {
  return prefill_impl(layout, n_new, q_rot, seq_lens, max_seq_len, scale, out, out_dtype, lse_out, err_word, stream,
                      /*early=*/0);
}

mqa_status mqa_prefill_step(const mqa_kv_layout* layout, int32_t n_new, const void* q_new, const void* k_new,
                            const void* v_new, const int32_t* pos, const int32_t* seq_lens, int32_t max_seq_len,
                            double rope_base, float scale, float* q_rot, void* out, int32_t out_dtype,
                            float* lse_out, int32_t* err_word, mqa_stream_t stream) {
  // the attention's own checks first, so nothing is launched for a call that fails
  const mqa_status st = check_layout(layout);
  if (st != MQA_OK) return st;
  if (!prefill_supported(layout)) return MQA_ERR_UNSUPPORTED;
  if (!seq_lens || !out || max_seq_len < n_new || max_seq_len > token_limit(layout)) return MQA_ERR_INVALID_ARG;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  const mqa_status a = append_impl(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word, stream, n_new);
  if (a != MQA_OK) return a;
  return prefill_impl(layout, n_new, q_rot, seq_lens, max_seq_len, scale, out, out_dtype, lse_out, err_word, stream,
                      /*early=*/1);
}

const char* mqa_status_string(mqa_status s) {
  switch (s) {
    case MQA_OK: return "ok";
    case MQA_ERR_INVALID_ARG: return "invalid argument";
    case MQA_ERR_UNSUPPORTED: return "unsupported configuration";
    case MQA_ERR_CUDA: return "CUDA error";
    case MQA_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

const char* mqa_last_cuda_error(void) { return g_cuda_error; }

mqa_status kv_append_rope(const mqa_kv_layout* layout, const void* q_new, const void* k_new, const void* v_new,
                          const int32_t* pos, double rope_base, float* q_rot, int32_t* err_word,
                          mqa_stream_t stream) {
  return append_impl(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word, stream);
}

int32_t mqa_choose_splits_multi(const mqa_kv_layout* layout, int32_t n_new, int32_t max_seq_len, int32_t variant) {
  if (check_layout(layout) != MQA_OK || max_seq_len < 1 || max_seq_len > token_limit(layout)) return -1;
  if (variant < MQA_VARIANT_AUTO || variant > MQA_VARIANT_TENSOR_CORE) return -1;
  if (n_new < 1 || n_new > kMaxNewTokens || max_seq_len < n_new) return -1;
  return choose_splits(layout, max_seq_len, resolve_variant(layout, variant), n_new);
}

int32_t mqa_choose_splits(const mqa_kv_layout* layout, int32_t max_seq_len, int32_t variant) {
  return mqa_choose_splits_multi(layout, 1, max_seq_len, variant);
}

size_t mqa_workspace_size_multi(const mqa_kv_layout* layout, int32_t n_new, int32_t max_seq_len, int32_t num_splits,
                                int32_t variant) {
  if (check_layout(layout) != MQA_OK || max_seq_len < 1 || max_seq_len > token_limit(layout) || num_splits < 0)
    return 0;
  if (variant < MQA_VARIANT_AUTO || variant > MQA_VARIANT_TENSOR_CORE) return 0;
  if (n_new < 1 || n_new > kMaxNewTokens || max_seq_len < n_new) return 0;
  const int v = resolve_variant(layout, variant);
  const int req = num_splits == 0 ? choose_splits(layout, max_seq_len, v, n_new) : num_splits;
  int splits, chunk;
  split_plan(layout, req, read_span(layout, max_seq_len, n_new), &splits, &chunk);
  return partial_bytes(layout, splits, n_new);
}

size_t mqa_workspace_size(const mqa_kv_layout* layout, int32_t max_seq_len, int32_t num_splits, int32_t variant) {
  return mqa_workspace_size_multi(layout, 1, max_seq_len, num_splits, variant);
}

int32_t mqa_step_launches(const mqa_kv_layout* layout, int32_t n_new, int32_t max_seq_len, int32_t num_splits,
                          int32_t variant, int32_t* fused_append) {
  if (check_layout(layout) != MQA_OK || max_seq_len < 1 || max_seq_len > token_limit(layout) || num_splits < 0)
    return -1;
  if (variant < MQA_VARIANT_AUTO || variant > MQA_VARIANT_TENSOR_CORE) return -1;
  if (n_new < 1 || n_new > kMaxNewTokens || max_seq_len < n_new) return -1;
  const int v = resolve_variant(layout, variant);
  if (!variant_supports(v, layout->cache_dtype) || !multi_supported(layout, v, n_new)) return -1;
  const int req = num_splits == 0 ? choose_splits(layout, max_seq_len, v, n_new) : num_splits;
  int splits, chunk;
  split_plan(layout, req, read_span(layout, max_seq_len, n_new), &splits, &chunk);
  // the decisions step_impl and attention_impl take
  const bool fused = (n_new == 1 && fusable(layout, v)) || fusable_multi(layout, v, n_new);
  bool merged = false;
  if (splits > 1) {
    Tc05Params t;
    std::memset(&t, 0, sizeof(t));
    t.group = layout->h_q / layout->h_kv;
    t.n_new = n_new;
    t.num_splits = splits;
    t.row_blocks = (t.group * n_new + 127) / 128;
    if (use_tc05(layout, v, n_new))
      merged = tc05_merges_splits(t);
    else if (v == MQA_VARIANT_TENSOR_CORE && layout->cache_dtype == MQA_FP8_E5M2 &&
             tc05_keys_applies(t.group, n_new, layout->head_dim, layout->paged))
      merged = tc05_widen_merges_splits(t);
  }
  if (layout->cache_dtype == MQA_U4) merged = true;
  if (fused_append) *fused_append = fused ? 1 : 0;
  return (fused ? 1 : 2) + (splits > 1 && !merged ? 1 : 0);
}

mqa_status splitkv_combine(const float* o_part, const float* lse_part, int32_t batch, int32_t h_q,
                           int32_t num_splits, int32_t head_dim, void* out, int32_t out_dtype, float* lse_out,
                           mqa_stream_t stream) {
  if (!o_part || !lse_part || !out) return MQA_ERR_INVALID_ARG;
  if (batch < 1 || h_q < 1 || num_splits < 1 || head_dim < 1) return MQA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MQA_ERR_UNSUPPORTED;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  if (!aligned(o_part, 4) || !aligned(lse_part, 4) || !aligned(out, 4) || (lse_out && !aligned(lse_out, 4)))
    return MQA_ERR_INVALID_ARG;
  CombineParams c;
  c.o_part = o_part;
  c.lse_part = lse_part;
  c.rows = batch * h_q;
  c.num_splits = num_splits;
  c.head_dim = head_dim;
  c.out = out;
  c.out_dtype = out_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  c.lse_out = lse_out;
  const cudaError_t e = launch_combine(c, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

mqa_status gqa_decode_attention(const mqa_kv_layout* layout, const float* q_rot, const int32_t* seq_lens,
                                int32_t max_seq_len, float scale, int32_t num_splits, void* out,
                                int32_t out_dtype, float* lse_out, void* workspace, size_t workspace_bytes,
                                int32_t variant, int32_t* err_word, mqa_stream_t stream) {
  return attention_impl(layout, q_rot, seq_lens, max_seq_len, scale, num_splits, out, out_dtype, lse_out, workspace,
                        workspace_bytes, variant, err_word, stream, /*early=*/0, /*rope=*/nullptr);
}

mqa_status kv_append_rope_multi(const mqa_kv_layout* layout, int32_t n_new, const void* q_new, const void* k_new,
                                const void* v_new, const int32_t* pos, double rope_base, float* q_rot,
                                int32_t* err_word, mqa_stream_t stream) {
  return append_impl(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word, stream, n_new);
}

mqa_status gqa_decode_attention_multi(const mqa_kv_layout* layout, int32_t n_new, const float* q_rot,
                                      const int32_t* seq_lens, int32_t max_seq_len, float scale, int32_t num_splits,
                                      void* out, int32_t out_dtype, float* lse_out, void* workspace,
                                      size_t workspace_bytes, int32_t variant, int32_t* err_word,
                                      mqa_stream_t stream) {
  return attention_impl(layout, q_rot, seq_lens, max_seq_len, scale, num_splits, out, out_dtype, lse_out, workspace,
                        workspace_bytes, variant, err_word, stream, /*early=*/0, /*rope=*/nullptr, n_new);
}

}  // extern "C"

namespace {

mqa_status step_impl(const mqa_kv_layout* layout, int n_new, const void* q_new, const void* k_new, const void* v_new,
                     const int32_t* pos, const int32_t* seq_lens, int32_t max_seq_len, double rope_base, float scale,
                     int32_t num_splits, float* q_rot, void* out, int32_t out_dtype, float* lse_out, void* workspace,
                     size_t workspace_bytes, int32_t variant, int32_t* err_word, mqa_stream_t stream) {
  // Check the attention's arguments too before anything is launched.
  const mqa_status st = check_layout(layout);
  if (st != MQA_OK) return st;
  if (n_new < 1 || n_new > kMaxNewTokens) return MQA_ERR_INVALID_ARG;
  if (!seq_lens || !out || max_seq_len < n_new || max_seq_len > token_limit(layout)) return MQA_ERR_INVALID_ARG;
  if (variant < MQA_VARIANT_AUTO || variant > MQA_VARIANT_TENSOR_CORE || num_splits < 0)
    return MQA_ERR_INVALID_ARG;
  if (!aligned(seq_lens, 4) || !aligned(out, 16) || !aligned(lse_out, 4) || !std::isfinite(scale) ||
      static_cast<long long>(layout->batch) * n_new * layout->h_q > (1ll << 31) - 1)
    return MQA_ERR_INVALID_ARG;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  const int v = resolve_variant(layout, variant);
  if (!variant_supports(v, layout->cache_dtype) || !multi_supported(layout, v, n_new)) return MQA_ERR_UNSUPPORTED;
  const int req = num_splits == 0 ? choose_splits(layout, max_seq_len, v, n_new) : num_splits;
  int splits, chunk;
  split_plan(layout, req, read_span(layout, max_seq_len, n_new), &splits, &chunk);
  const size_t need = partial_bytes(layout, splits, n_new);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MQA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return MQA_ERR_INVALID_ARG;
  const mqa_status ca = check_append_args(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word);
  if (ca != MQA_OK) return ca;
  if ((n_new == 1 && fusable(layout, v)) || fusable_multi(layout, v, n_new)) {
    // one launch: the attention kernel appends the new token(s) itself
    const RopeArgs rope{q_new, pos, rope_base, 1, k_new, v_new, q_rot};
    return attention_impl(layout, q_rot, seq_lens, max_seq_len, scale, num_splits, out, out_dtype, lse_out,
                          workspace, workspace_bytes, variant, err_word, stream, /*early=*/0, &rope, n_new);
  }
  // (a 4-bit cache whose tiles are shared: the append clears the attention's counters)
  const bool runs = layout->cache_dtype == MQA_U4 && need > 0;
  const mqa_status a = append_impl(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word, stream, n_new, nullptr,
                                   runs ? static_cast<int32_t*>(workspace) : nullptr,
                                   runs ? u4_plan(layout, n_new).ctas : 0);
  if (a != MQA_OK) return a;
  const RopeArgs rope{q_new, pos, rope_base, 0, nullptr, nullptr, nullptr};
  return attention_impl(layout, q_rot, seq_lens, max_seq_len, scale, num_splits, out, out_dtype, lse_out, workspace,
                        workspace_bytes, variant, err_word, stream, /*early=*/1, &rope, n_new);
}

}  // namespace

extern "C" {

mqa_status mqa_decode_step(const mqa_kv_layout* layout, const void* q_new, const void* k_new, const void* v_new,
                           const int32_t* pos, const int32_t* seq_lens, int32_t max_seq_len, double rope_base,
                           float scale, int32_t num_splits, float* q_rot, void* out, int32_t out_dtype,
                           float* lse_out, void* workspace, size_t workspace_bytes, int32_t variant,
                           int32_t* err_word, mqa_stream_t stream) {
  return step_impl(layout, 1, q_new, k_new, v_new, pos, seq_lens, max_seq_len, rope_base, scale, num_splits, q_rot,
                   out, out_dtype, lse_out, workspace, workspace_bytes, variant, err_word, stream);
}

mqa_status mqa_decode_step_multi(const mqa_kv_layout* layout, int32_t n_new, const void* q_new, const void* k_new,
                                 const void* v_new, const int32_t* pos, const int32_t* seq_lens, int32_t max_seq_len,
                                 double rope_base, float scale, int32_t num_splits, float* q_rot, void* out,
                                 int32_t out_dtype, float* lse_out, void* workspace, size_t workspace_bytes,
                                 int32_t variant, int32_t* err_word, mqa_stream_t stream) {
  return step_impl(layout, n_new, q_new, k_new, v_new, pos, seq_lens, max_seq_len, rope_base, scale, num_splits,
                   q_rot, out, out_dtype, lse_out, workspace, workspace_bytes, variant, err_word, stream);
}

}  // extern "C"

// ------------------------------------------------- a tree of drafted tokens
namespace {

mqa_status check_tree_layout(const mqa_kv_layout* L, int n) {
  const mqa_status st = check_layout(L);
  if (st != MQA_OK) return st;
  // tensor cores only, as the multi-token calls; no 4-bit form
  if (L->cache_dtype == MQA_F32 || L->cache_dtype == MQA_U4) return MQA_ERR_UNSUPPORTED;
  if (n < 1 || n > kMaxTreeNodes) return MQA_ERR_INVALID_ARG;
  if (static_cast<long long>(L->batch) * n * L->h_q > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  return MQA_OK;
}

struct TreeChoice {
  TreeShape shape;
  int tc05;          // row tiles of a block of the tcgen05 kernel, 0: the warp-MMA kernel
  int tokens;        // ... nodes of a row tile
  int ctas;          // blocks launched
  size_t counters;   // bytes of the counters at the start of the workspace
  size_t workspace;
};

TreeChoice tree_choice(const mqa_kv_layout* L, int n) {
  int dev = 0;
  cudaGetDevice(&dev);
  TreeChoice c;
  const int G = L->h_q / L->h_kv;
  c.shape = tree_mma_shape(L->head_dim);
  c.tc05 = c.tokens = 0;
  if (L->head_dim == 128 && G <= 128) {
    // (uint8: one row tile, the kernel has no room for a second beside the scales)
    c.tc05 = static_cast<long long>(G) * n > 128 && L->cache_dtype != MQA_U8 ? 2 : 1;
    c.tokens = std::min(128 / G, n);
    c.shape = {c.tc05 * c.tokens * G, 1};
  }
  c.ctas = device_info(dev).sms * c.shape.ctas_per_sm;
  c.counters = (static_cast<size_t>(c.ctas) * 4 + 255) / 256 * 256;
  c.workspace = c.counters + static_cast<size_t>(2) * c.ctas * tree_part_floats(c.shape.rows, L->head_dim) * 4;
  return c;
}

// A paged bf16 pool for the tcgen05 tree kernel: (64 dims, 8 rows, the two
// 64-dim halves, a page's groups of 8 rows, (page, kv head)), a box all of the
// first three and min(page_size, 64) rows: one copy per page run, landing as
// [groups][halves][8 rows][128 B].
bool make_tree_paged_map(CUtensorMap* map, void* base, const mqa_kv_layout* L) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t ps = static_cast<cuuint64_t>(L->page_size);
  const cuuint64_t dims[5] = {64, 8, 2, ps / 8, static_cast<cuuint64_t>(L->h_kv) * L->num_pages};
  const cuuint64_t strides[4] = {256, 128, 8 * 256, ps * 256};
  const cuuint32_t box[5] = {64, 8, 2, static_cast<cuuint32_t>(L->page_size < 64 ? L->page_size : 64) / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tcgen05 tree kernel's maps: K and V tiles, and q_rot [batch n tokens]
// [h_q][128] bf16 in boxes of 64 dims x the group x `tokens`.
bool make_tree_maps(const mqa_kv_layout* L, const void* q_rot, int n, int tokens, CUtensorMap* tk, CUtensorMap* tv,
                    CUtensorMap* tq) {
  if (L->cache_dtype == MQA_BF16) {
    if (!(L->paged ? make_tree_paged_map(tk, L->k_cache, L) && make_tree_paged_map(tv, L->v_cache, L)
                   : make_tensor_map(tk, L->k_cache, L, true, 1, kTreeTileKeys) &&
                         make_tensor_map(tv, L->v_cache, L, true, 1, kTreeTileKeys)))
      return false;
  } else {
    CUtensorMap maps[4];
    if (!make_u8_maps(maps, L, L->paged ? std::min(L->page_size, 64) : kTreeTileKeys, 1)) return false;
    *tk = maps[0];
    *tv = maps[1];
  }
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(L->h_q), static_cast<cuuint64_t>(L->batch) * n};
  const cuuint64_t strides[2] = {128 * 2, static_cast<cuuint64_t>(L->h_q) * 128 * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(L->h_q / L->h_kv), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q_rot), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

mqa_status check_tree_attention(const mqa_kv_layout* L, int n, const void* q_rot, const int32_t* pos,
                                const int32_t* depth, const int32_t* num_nodes, const uint32_t* mask, int max_seq_len,
                                float scale, const void* out, int out_dtype, const float* lse_out,
                                const void* workspace, size_t workspace_bytes, const int32_t* err_word) {
  const mqa_status st = check_tree_layout(L, n);
  if (st != MQA_OK) return st;
  if (!q_rot || !pos || !mask || !out || !err_word) return MQA_ERR_INVALID_ARG;
  if (L->window > 0 && !depth) return MQA_ERR_INVALID_ARG;
  if (!aligned(q_rot, 16) || !aligned(pos, 4) || !aligned(depth, 4) || !aligned(num_nodes, 4) || !aligned(mask, 4) ||
      !aligned(out, 16) || !aligned(lse_out, 4) || !aligned(err_word, 4))
    return MQA_ERR_INVALID_ARG;
  if (max_seq_len < 1 || max_seq_len > token_limit(L)) return MQA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MQA_ERR_INVALID_ARG;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < tree_choice(L, n).workspace) return MQA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MQA_ERR_INVALID_ARG;
  return MQA_OK;
}

// after the checks; early: the append launch, which clears the counters, directly precedes
mqa_status tree_attention_impl(const mqa_kv_layout* L, int n, const void* q_rot, const int32_t* pos,
                               const int32_t* depth, const int32_t* num_nodes, const uint32_t* mask, int max_seq_len,
                               float scale, void* out, int out_dtype, float* lse_out, void* workspace,
                               int32_t* err_word, cudaStream_t stream, int early) {
  const TreeChoice c = tree_choice(L, n);
  TreeParams p;
  std::memset(&p, 0, sizeof(p));
  p.batch = L->batch;
  p.h_q = L->h_q;
  p.h_kv = L->h_kv;
  p.group = L->h_q / L->h_kv;
  p.n = n;
  p.words = (n + 31) / 32;
  p.cache_dtype = dtype_code(L->cache_dtype);
  p.head_dim = L->head_dim;
  p.paged = L->paged;
  p.k_cache = L->k_cache;
  p.v_cache = L->v_cache;
  p.k_sz = static_cast<const float2*>(L->k_scale_zero);
  p.v_sz = static_cast<const float2*>(L->v_scale_zero);
  p.capacity = token_limit(L);
  p.page_size = L->page_size;
  p.num_pages = L->num_pages;
  p.max_pages = L->max_pages_per_seq;
  p.block_table = L->block_table;
  p.max_seq_len = max_seq_len;
  p.q_rot = q_rot;
  p.pos = pos;
  p.depth = depth;
  p.num_nodes = num_nodes;
  p.mask = mask;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.window = L->window;
  p.out = out;
  p.out_dtype = out_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  p.lse_out = lse_out;
  p.arrived = static_cast<int32_t*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + c.counters);
  p.err = err_word;
  // (2, 3, 4, 6 tiles measured: 8 kv heads, 8 nodes, 700 tokens 16.0, 17.0, 19.3, 17.6 us;
  // 3000 tokens 20.8, 20.6, 20.0, 21.0, over e5m2 22.9, 22.2, 22.8, 23.0, over uint8 24.9,
  // 23.6, 25.0, 27.1; 8000 tokens 33.0, 32.5, 33.1, 27.1)
  p.min_tiles = 3;
  p.tokens_per_tile = c.tokens;
  p.early = early;
  p.wait_ns = wait_limit(L);
  if (!early) {
    const cudaError_t ez = cudaMemsetAsync(workspace, 0, static_cast<size_t>(c.ctas) * 4, stream);
    if (ez != cudaSuccess) return fail_cuda(ez);
  }
  cudaError_t e;
  if (c.tc05) {
    CUtensorMap tk, tv, tq;
    if (!make_tree_maps(L, q_rot, n, c.tokens, &tk, &tv, &tq)) {
      snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed or is unavailable");
      return MQA_ERR_CUDA;
    }
    const auto launch = L->cache_dtype == MQA_BF16 ? launch_tree_tc05_bf16
                                                   : (L->cache_dtype == MQA_U8 ? launch_tree_tc05_u8 : launch_tree_tc05_f8);
    e = launch(p, c.tc05, c.ctas, tk, tv, tq, stream);
  } else {
    e = launch_tree_mma(p, c.ctas, stream);
  }
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

mqa_status check_tree_append(const mqa_kv_layout* L, int n, const void* q_new, const void* k_new, const void* v_new,
                             const int32_t* pos, const int32_t* depth, const int32_t* num_nodes, double rope_base,
                             const void* q_rot, const int32_t* err_word) {
  const mqa_status st = check_tree_layout(L, n);
  if (st != MQA_OK) return st;
  if (!depth || !aligned(depth, 4) || !aligned(num_nodes, 4)) return MQA_ERR_INVALID_ARG;
  return check_append_args(L, q_new, k_new, v_new, pos, rope_base, static_cast<const float*>(q_rot), err_word);
}

// Whether a K or V of one of kv_keep_path's layers holds rows of another's (or, a
// = b, its K those of its V): they would be moved more than once. Layers may share a
// pool, each with a table of its own.
bool same_rows(const mqa_kv_layout& a, const mqa_kv_layout& b) {
  if (a.paged && a.block_table != b.block_table) return false;
  if (&a == &b) return a.k_cache == a.v_cache;
  return a.k_cache == b.k_cache || a.k_cache == b.v_cache || a.v_cache == b.k_cache || a.v_cache == b.v_cache;
}

}  // namespace

extern "C" {

size_t mqa_tree_workspace_size(const mqa_kv_layout* layout, int32_t n_nodes) {
  return check_tree_layout(layout, n_nodes) == MQA_OK ? tree_choice(layout, n_nodes).workspace : 0;
}

mqa_status kv_append_rope_tree(const mqa_kv_layout* layout, int32_t n_nodes, const void* q_new, const void* k_new,
                               const void* v_new, const int32_t* pos, const int32_t* depth, const int32_t* num_nodes,
                               double rope_base, void* q_rot, int32_t* err_word, mqa_stream_t stream) {
  const mqa_status st =
      check_tree_append(layout, n_nodes, q_new, k_new, v_new, pos, depth, num_nodes, rope_base, q_rot, err_word);
  if (st != MQA_OK) return st;
  const TreeAppend tree{depth, num_nodes, nullptr, 0};
  return append_impl(layout, q_new, k_new, v_new, pos, rope_base, static_cast<float*>(q_rot), err_word, stream,
                     n_nodes, &tree);
}

mqa_status gqa_tree_attention(const mqa_kv_layout* layout, int32_t n_nodes, const void* q_rot, const int32_t* pos,
                              const int32_t* depth, const int32_t* num_nodes, const uint32_t* tree_mask,
                              int32_t max_seq_len, float scale, void* out, int32_t out_dtype, float* lse_out,
                              void* workspace, size_t workspace_bytes, int32_t* err_word, mqa_stream_t stream) {
  const mqa_status st = check_tree_attention(layout, n_nodes, q_rot, pos, depth, num_nodes, tree_mask, max_seq_len,
                                             scale, out, out_dtype, lse_out, workspace, workspace_bytes, err_word);
  if (st != MQA_OK) return st;
  return tree_attention_impl(layout, n_nodes, q_rot, pos, depth, num_nodes, tree_mask, max_seq_len, scale, out,
                             out_dtype, lse_out, workspace, err_word, reinterpret_cast<cudaStream_t>(stream),
                             /*early=*/0);
}

mqa_status mqa_tree_step(const mqa_kv_layout* layout, int32_t n_nodes, const void* q_new, const void* k_new,
                         const void* v_new, const int32_t* pos, const int32_t* depth, const int32_t* num_nodes,
                         const uint32_t* tree_mask, int32_t max_seq_len, double rope_base, float scale, void* q_rot,
                         void* out, int32_t out_dtype, float* lse_out, void* workspace, size_t workspace_bytes,
                         int32_t* err_word, mqa_stream_t stream) {
  // both calls' checks before the first launch
  mqa_status st = check_tree_append(layout, n_nodes, q_new, k_new, v_new, pos, depth, num_nodes, rope_base, q_rot,
                                    err_word);
  if (st != MQA_OK) return st;
  st = check_tree_attention(layout, n_nodes, q_rot, pos, depth, num_nodes, tree_mask, max_seq_len, scale, out,
                            out_dtype, lse_out, workspace, workspace_bytes, err_word);
  if (st != MQA_OK) return st;
  const TreeAppend tree{depth, num_nodes, static_cast<int32_t*>(workspace), tree_choice(layout, n_nodes).ctas};
  st = append_impl(layout, q_new, k_new, v_new, pos, rope_base, static_cast<float*>(q_rot), err_word, stream, n_nodes,
                   &tree);
  if (st != MQA_OK) return st;
  return tree_attention_impl(layout, n_nodes, q_rot, pos, depth, num_nodes, tree_mask, max_seq_len, scale, out,
                             out_dtype, lse_out, workspace, err_word, reinterpret_cast<cudaStream_t>(stream),
                             /*early=*/1);
}

mqa_status mqa_verify_tree(int32_t batch, int32_t n_nodes, int32_t vocab, const void* target_probs,
                           const void* draft_probs, int32_t probs_dtype, int64_t row_stride, const int32_t* tokens,
                           const int32_t* parents, const int32_t* num_nodes, const float* u_accept,
                           const float* u_next, int32_t* num_kept, int32_t* path, int32_t* next_token,
                           int32_t* err_word, mqa_stream_t stream) {
  if (batch < 1 || n_nodes < 1 || n_nodes > kMaxTreeNodes || vocab < 1) return MQA_ERR_INVALID_ARG;
  if (static_cast<long long>(batch) * n_nodes > (1ll << 31) - 1 || batch > (1 << 27)) return MQA_ERR_INVALID_ARG;
  if (vocab > (1 << 30) || row_stride < vocab || row_stride > (1ll << 31)) return MQA_ERR_INVALID_ARG;
  if (!target_probs || !tokens || !parents || !u_accept || !u_next || !num_kept || !path || !next_token || !err_word)
    return MQA_ERR_INVALID_ARG;
  if (!aligned(target_probs, 16) || !aligned(draft_probs, 16) || !aligned(tokens, 4) || !aligned(parents, 4) ||
      !aligned(num_nodes, 4) || !aligned(u_accept, 4) || !aligned(u_next, 4) || !aligned(num_kept, 4) ||
      !aligned(path, 4) || !aligned(next_token, 4) || !aligned(err_word, 4))
    return MQA_ERR_INVALID_ARG;
  if (probs_dtype != MQA_F32 && probs_dtype != MQA_BF16) return MQA_ERR_UNSUPPORTED;
  VerifyParams p;
  std::memset(&p, 0, sizeof(p));
  p.batch = batch;
  p.n = n_nodes;
  p.vocab = vocab;
  p.dtype = probs_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  p.row_stride = row_stride;
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = tokens;
  p.parents = parents;
  p.num_nodes = num_nodes;
  p.u_accept = u_accept;
  p.u_next = u_next;
  p.num_kept = num_kept;
  p.path = path;
  p.next_token = next_token;
  p.err = err_word;
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = launch_verify_tree(p, device_info(dev).sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

mqa_status kv_keep_path(const mqa_kv_layout* layouts, int32_t n_layers, int32_t n_nodes, const int32_t* pos,
                        const int32_t* path, const int32_t* num_kept, int32_t* err_word, mqa_stream_t stream) {
  if (layouts == nullptr || n_layers < 1 || n_nodes < 1 || n_nodes > kMaxTreeNodes) return MQA_ERR_INVALID_ARG;
  const mqa_kv_layout& f = layouts[0];
  for (int i = 0; i < n_layers; ++i) {
    const mqa_kv_layout& L = layouts[i];
    const mqa_status st = check_layout(&L);
    if (st != MQA_OK) return st;
    if (L.cache_dtype == MQA_U4) return MQA_ERR_UNSUPPORTED;
    if (L.cache_dtype != f.cache_dtype || L.batch != f.batch || L.h_kv != f.h_kv || L.head_dim != f.head_dim ||
        L.paged != f.paged)
      return MQA_ERR_INVALID_ARG;
    if (L.paged ? L.page_size != f.page_size || L.num_pages != f.num_pages ||
                      L.max_pages_per_seq != f.max_pages_per_seq
                : L.capacity != f.capacity)
      return MQA_ERR_INVALID_ARG;
    for (int j = 0; j <= i; ++j)
      if (same_rows(layouts[j], L)) return MQA_ERR_INVALID_ARG;
  }
  if (!pos || !path || !num_kept || !err_word) return MQA_ERR_INVALID_ARG;
  if (!aligned(pos, 4) || !aligned(path, 4) || !aligned(num_kept, 4) || !aligned(err_word, 4))
    return MQA_ERR_INVALID_ARG;
  if (f.h_kv > 65535) return MQA_ERR_UNSUPPORTED;  // grid limit
  KeepParams p;
  std::memset(&p, 0, sizeof(p));
  p.batch = f.batch;
  p.h_kv = f.h_kv;
  p.n = n_nodes;
  p.paged = f.paged;
  p.row_bytes = f.head_dim * (f.cache_dtype == MQA_F32 ? 4 : (f.cache_dtype == MQA_BF16 ? 2 : 1));
  p.capacity = token_limit(&f);
  p.page_size = f.page_size;
  p.num_pages = f.num_pages;
  p.max_pages = f.max_pages_per_seq;
  p.pos = pos;
  p.path = path;
  p.num_kept = num_kept;
  p.err = err_word;
  int dev = 0;
  cudaGetDevice(&dev);
  for (int i0 = 0; i0 < n_layers; i0 += kMaxKeepLayers) {
    const int m = std::min(kMaxKeepLayers, n_layers - i0);
    for (int i = 0; i < m; ++i) {
      const mqa_kv_layout& L = layouts[i0 + i];
      const bool u8 = L.cache_dtype == MQA_U8;
      p.layer[i] = {L.k_cache, L.v_cache, u8 ? static_cast<float2*>(L.k_scale_zero) : nullptr,
                    u8 ? static_cast<float2*>(L.v_scale_zero) : nullptr, L.block_table};
    }
    const cudaError_t e = launch_keep_path(p, m, device_info(dev).sms, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail_cuda(e);
  }
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

mqa_status kv_append_norm_rope(const mqa_kv_layout* layout, int32_t n_new, const void* q_new, const void* k_new,
                               const void* v_new, const int32_t* pos, const mqa_norm_rope* options, double rope_base,
                               float* q_rot, int32_t* err_word, mqa_stream_t stream) {
  const mqa_status st = check_append_args(layout, q_new, k_new, v_new, pos, rope_base, q_rot, err_word);
  if (st != MQA_OK) return st;
  if (n_new < 1 || static_cast<long long>(layout->batch) * n_new > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  if (options != nullptr) {
    if (!aligned(options->q_weight, 16) || !aligned(options->k_weight, 16)) return MQA_ERR_INVALID_ARG;
    if ((options->q_weight || options->k_weight) && (!(options->eps > 0.f) || !std::isfinite(options->eps)))
      return MQA_ERR_INVALID_ARG;
    if (options->n_axes < 0 || options->n_axes > kMaxAxes) return MQA_ERR_INVALID_ARG;
    if (options->n_axes > 0) {
      if (options->axis_pos == nullptr || !aligned(options->axis_pos, 4)) return MQA_ERR_INVALID_ARG;
      long long pairs = 0;
      for (int a = 0; a < options->n_axes; ++a) {
        if (options->section[a] < 0) return MQA_ERR_INVALID_ARG;
        pairs += options->section[a];
      }
      if (pairs != layout->head_dim / 2) return MQA_ERR_INVALID_ARG;
    }
  }
  return norm_append(layout, n_new, q_new, k_new, v_new, pos, options, rope_base, q_rot, nullptr, 0, err_word,
                     reinterpret_cast<cudaStream_t>(stream));
}

mqa_status kv_read_rows(const mqa_kv_layout* layout, int32_t n_rows, const int32_t* start, const int32_t* num_rows,
                        void* k_out, void* v_out, int32_t out_dtype, int32_t* err_word, mqa_stream_t stream) {
  const mqa_status st = check_layout(layout);
  if (st != MQA_OK) return st;
  if (!k_out || !v_out || !err_word) return MQA_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(start, 4) || !aligned(num_rows, 4) || !aligned(err_word, 4))
    return MQA_ERR_INVALID_ARG;
  if (n_rows < 1 || n_rows > token_limit(layout)) return MQA_ERR_INVALID_ARG;
  if (out_dtype != MQA_BF16 && out_dtype != MQA_F32) return MQA_ERR_UNSUPPORTED;
  // (at least 64 rows to a block)
  if ((static_cast<long long>(n_rows) + 63) / 64 * layout->batch * layout->h_kv > (1ll << 31) - 1) return MQA_ERR_INVALID_ARG;
  ReadParams p;
  std::memset(&p, 0, sizeof(p));
  p.batch = layout->batch;
  p.h_kv = layout->h_kv;
  p.head_dim = layout->head_dim;
  p.cache_dtype = dtype_code(layout->cache_dtype);
  p.paged = layout->paged;
  p.k_cache = layout->k_cache;
  p.v_cache = layout->v_cache;
  p.k_sz = layout->k_scale_zero;
  p.v_sz = layout->v_scale_zero;
  p.capacity = layout->capacity;
  p.limit = token_limit(layout);
  p.page_size = layout->page_size;
  p.num_pages = layout->num_pages;
  p.max_pages = layout->max_pages_per_seq;
  p.block_table = layout->block_table;
  p.start = start;
  p.num_rows = num_rows;
  p.n_rows = n_rows;
  p.k_out = k_out;
  p.v_out = v_out;
  p.out_dtype = out_dtype == MQA_BF16 ? kDtypeBf16 : kDtypeF32;
  p.err = err_word;
  const cudaError_t e = launch_read_rows(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  const cudaError_t e2 = cudaGetLastError();
  return e2 == cudaSuccess ? MQA_OK : fail_cuda(e2);
}

}  // extern "C"
