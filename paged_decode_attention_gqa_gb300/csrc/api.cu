// C-ABI front end: argument validation, split plan (grid size), TMA tensor
// maps, workspace layout, launches. Declared in include/zl_decode_attn.h.
#include "../../include/zl_decode_attn.h"
#include "gqa_wide.h"
#include "kernels.h"
#include "q4_host.h"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

namespace {

using zl::GqaParams;

constexpr double kLog2e = 1.4426950408889634;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// cuTensorMapEncodeTiled from the driver, fetched once through the runtime so
// the library links against cudart only.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A different nonzero tag for every GQA call in this process: the in-kernel
// split merge counts arrivals per tag, so counters left behind by a call that
// stopped early (a device error) are ignored by the next call. The call
// number goes through an invertible 32-bit mix (odd multiplier, xor-shifts),
// so consecutive tags are far apart and unlike small integers or float bits
// that other data may have left in the buffer.
uint32_t next_epoch() {
  static std::atomic<uint32_t> counter{0};
  uint32_t e = 0;
  while (e == 0) {
    uint32_t x = counter.fetch_add(1, std::memory_order_relaxed) + 1;
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    x ^= x >> 16;
    e = x;
  }
  return e;
}

struct DeviceInfo {
  int device = -1;
  int sms = 0;
};

zl_status current_device(DeviceInfo* info) {
  static int sm_count[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZL_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZL_ERR_UNSUPPORTED;
  if (sm_count[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return ZL_ERR_CUDA;
    sm_count[dev] = n;
  }
  info->device = dev;
  info->sms = sm_count[dev];
  return ZL_OK;
}

}  // namespace

// For the entry points of other files (q4_host.h).
zl_status zl::sm_count(int* sms) {
  DeviceInfo dev;
  const zl_status st = current_device(&dev);
  if (st == ZL_OK) *sms = dev.sms;
  return st;
}
CUresult zl::encode_tiled(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, void* base,
                          const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  auto encode = tensor_map_encoder();
  if (!encode) return CUDA_ERROR_NOT_INITIALIZED;
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return encode(map, type, rank, base, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

namespace {

// ------------------------------------------------------------------ GQA plan
struct GqaPlan {
  int hpc = 0, nhg = 0, g = 0, grid = 0;
  bool fused = false;
  // shared-prefix calls: prefix tiles, sequences per group, groups
  int prefix_tiles = 0, sgs = 0, ng = 0;
  int q_group = 1;  // query tokens per row group
  int gh = 0, hchunks = 1;  // query heads per row group, head chunks per kv head
  int ngroups = 1;          // row groups: ceil(q_len / q_group) x hchunks
  int tg = 1;       // token groups per CTA (2: both groups of a two-group call in every CTA)
  bool unit_cut = false;  // one CTA per (sequence, head group): no cut unit, no merge
  size_t off_lse = 0, off_o = 0, off_pre_lse = 0, off_pre_o = 0;
  size_t off_suf_lse = 0, off_suf_o = 0, bytes = 0;
  // modified scores with weights: each row's base and 1 / sum, then its scores
  size_t off_stat = 0, off_scores = 0;
  int64_t score_stride = 0;
  // modified scores with many rows: the tcgen05 kernel (gqa_wide.cu)
  bool wide = false;
  int tpt = 1, mt = 1, nblk = 1;
};

// Query rows per kv head above which a modified-score call runs the tcgen05
// kernel; with at most kFewUnits (sequence, kv head) units only above
// kWideRowsFew. Both sides measured, drafted trees, 4 heads to a kv head: 512
// units of 512-4096 tokens, 16 rows 120 us by either kernel, 20 rows 122 by the
// tcgen05 one and 166 by the other, 36 rows 123 and 230; 16 units of 200 tokens
// and 32 rows 13.7 and 16.2, of 16000 tokens 43 and 52; 8 units of 200 tokens and
// 20 or 32 rows 13.3 and 12.4 to 13.0, of 4000 tokens 24 and 21 to 23.
// A call with weights always runs the other one, which stores the scores that the
// weights are summed from. That is meant for few rows: 64 sequences of 512-4096
// tokens, 32 heads on 8 kv heads, with weights 16 drafted tokens take 487 us and
// 0.56 GB of scratch (135 us without weights, from a cold L2), 64 drafted tokens
// 1877 us and 2.2 GB (171 without).
constexpr int kWideRows = 16;
constexpr int kWideRowsFew = 32;
constexpr int kFewUnits = 8;

// Query tokens per sequence one call takes, and query heads per kv head (the
// GQA path takes the (token, head) rows of a kv head in groups of at most 16).
constexpr int kMaxQueryTokens = 128;
constexpr int kMaxGroupHeads = 128;
// A call whose longest (sequence, head group) unit has at most
// zl::kGqaUnitCutTiles tiles (known from max_seq_len) gives each unit a
// CTA of its own and skips the merge launch. Without max_seq_len the kernels
// take the same decision on the device (GqaParams::auto_cut).

zl_status gqa_validate_shape(const zl_decode_attn_params* a) {
  if (!a || a->struct_size != sizeof(zl_decode_attn_params)) return ZL_ERR_INVALID_ARG;
  if (a->B < 1 || a->Hq < 1 || a->Hkv < 1 || a->q_len < 1 || a->page_size < 1 ||
      a->num_pages < 1 || a->block_table_stride < 1 || a->D_qk < 1 || a->D_v < 1 ||
      a->num_ctas < 0 || a->max_seq_len < 0)
    return ZL_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0) return ZL_ERR_INVALID_ARG;
  if (a->flags & ~uint32_t(ZL_DECODE_SINGLE_LAUNCH | ZL_DECODE_TEST_STALL))
    return ZL_ERR_INVALID_ARG;
  if (a->num_ctas > 65535) return ZL_ERR_UNSUPPORTED;  // the tile cut needs G^2 < 2^32
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return ZL_ERR_INVALID_ARG;
  if (a->D_qk != zl::kGqaHeadDim || a->D_v != zl::kGqaHeadDim) return ZL_ERR_UNSUPPORTED;
  // (query token, head) rows of one kv head share an m16 tile: at most 16 per
  // row group. A call with g * q_len > 16 takes its query tokens in groups of
  // 16 / g, or with g > 16 each token's heads in ceil(g / 16) chunks (side by
  // side in one launch; one launch per group in single-launch mode). A
  // shared-prefix call keeps all its rows in one group.
  if (a->Hq / a->Hkv > kMaxGroupHeads || a->q_len > kMaxQueryTokens) return ZL_ERR_UNSUPPORTED;
  if (a->shared_prefix_pages > 0 && a->Hq / a->Hkv * a->q_len > 16) return ZL_ERR_UNSUPPORTED;
  if (a->page_size % zl::kGqaTile != 0 || a->page_size > 1024) return ZL_ERR_UNSUPPORTED;
  if (a->B > zl::kMaxBatch) return ZL_ERR_UNSUPPORTED;
  if (a->shared_prefix_pages < 0 || a->shared_prefix_pages > a->block_table_stride)
    return ZL_ERR_INVALID_ARG;
  if (a->shared_prefix_pages > 0 && (a->flags & ZL_DECODE_SINGLE_LAUNCH))
    return ZL_ERR_UNSUPPORTED;
  return ZL_OK;
}

// Score modifications (zl_decode_attn_ex): what does not depend on the call's pointers.
zl_status mods_validate(const zl_decode_attn_params* a, const zl_score_params* m) {
  if (!m || m->struct_size != sizeof(zl_score_params)) return ZL_ERR_INVALID_ARG;
  if (!(m->softcap >= 0.f) || !std::isfinite(m->softcap) || m->window < 0)
    return ZL_ERR_INVALID_ARG;
  // scale / c and c * log2(e) must be normal numbers
  if (m->softcap > 0.f && (m->softcap < 1e-6f || m->softcap > 1e6f ||
                           !std::isnormal(float(double(a->scale) / m->softcap))))
    return ZL_ERR_UNSUPPORTED;
  if (!aligned(m->alibi_slopes, 4) || !aligned(m->tree_mask, 4) || !aligned(m->weights, 4))
    return ZL_ERR_INVALID_ARG;
  if (m->weights) {
    if (m->weights_tokens < 1 || !std::isfinite(m->weights_decay) || m->weights_decay < 0.f)
      return ZL_ERR_INVALID_ARG;
    if (!zl::rows_distinct(a->B, a->Hkv, m->weights_seq_stride, m->weights_head_stride,
                           m->weights_tokens))
      return ZL_ERR_INVALID_ARG;
    // (the grid that sums them: whole blocks of tokens in 32 bits, a kv head each in y)
    if (m->weights_tokens > zl::kMaxWeightsTokens || a->Hkv > 65535) return ZL_ERR_UNSUPPORTED;
  }
  if (a->flags || a->shared_prefix_pages != 0) return ZL_ERR_UNSUPPORTED;
  return ZL_OK;
}

zl_status gqa_plan(const zl_decode_attn_params* a, GqaPlan* plan,
                   const zl_score_params* mods = nullptr) {
  zl_status st = gqa_validate_shape(a);
  if (st != ZL_OK) return st;
  if (mods && (st = mods_validate(a, mods)) != ZL_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != ZL_OK) return st;
  plan->g = a->Hq / a->Hkv;
  plan->tpt = 128 / plan->g;
  const int row_tiles = (a->q_len + plan->tpt - 1) / plan->tpt;
  plan->mt = row_tiles > 1 ? 2 : 1;
  plan->nblk = (row_tiles + plan->mt - 1) / plan->mt;
  // (the tcgen05 kernel counts tiles, and each unit's fixed cost, in 32 bits)
  const double most_tiles = double(a->B) * a->Hkv * plan->nblk *
                            (double(a->block_table_stride) * a->page_size / zl::kWideTile + 1 +
                             zl::kWideUnitCost);
  const int head_rows = plan->g * a->q_len;
  if (mods && !mods->weights && most_tiles < 2e9 &&
      head_rows > (int64_t(a->B) * a->Hkv <= kFewUnits ? kWideRowsFew : kWideRows)) {
    plan->wide = true;
    plan->grid = a->num_ctas > 0 ? a->num_ctas : dev.sms;
    if (a->num_ctas == 0 && a->max_seq_len > 0) {
      int64_t len = a->max_seq_len;
      if (mods->window > 0) len = std::min(len, int64_t(mods->window) + a->q_len + zl::kWideTile);
      const int64_t units = int64_t(a->B) * a->Hkv * plan->nblk;
      const int64_t tiles = (len + zl::kWideTile - 1) / zl::kWideTile;
      if (units <= plan->grid && tiles <= zl::kWideWholeTiles) {
        plan->unit_cut = true;  // one CTA per unit, no merge
        plan->grid = int(units);
      } else {
        plan->grid = int(std::min(int64_t(plan->grid), std::max<int64_t>(units * tiles, 1)));
      }
    }
    const size_t slots = size_t(plan->grid) * 2 * plan->mt * 128;
    plan->off_lse = round_up(size_t(plan->grid) * sizeof(int4), 256);
    plan->off_o = plan->off_lse + round_up(slots * sizeof(float), 256);
    plan->bytes = plan->off_o + slots * zl::kGqaHeadDim * sizeof(float);
    return ZL_OK;
  }
  plan->fused = (a->flags & ZL_DECODE_SINGLE_LAUNCH) != 0;
  plan->hpc = zl::gqa_heads_per_cta(a->Hkv);
  plan->nhg = a->Hkv / plan->hpc;
  if (plan->g <= 16) {  // every head of a token in one group
    plan->gh = plan->g;
    plan->hchunks = 1;
    plan->q_group = std::min(a->q_len, 16 / plan->g);
  } else {  // one token per group, its heads in chunks of at most 16
    plan->hchunks = (plan->g + 15) / 16;
    plan->gh = (plan->g + plan->hchunks - 1) / plan->hchunks;
    plan->q_group = 1;
  }
  plan->ngroups = (a->q_len + plan->q_group - 1) / plan->q_group * plan->hchunks;
  // Exactly two row groups, side by side: every CTA takes both (half the kv
  // heads per CTA, the same number of warps), so that one shared-memory stage
  // serves both groups and each K/V tile crosses from L2 once.
  if (plan->ngroups == 2 && !plan->fused && a->shared_prefix_pages == 0) {
    plan->tg = 2;
    plan->hpc = std::max(1, plan->hpc / 2);
    plan->nhg = a->Hkv / plan->hpc;
  }
  const int rps = plan->gh * plan->q_group;
  if (a->shared_prefix_pages > 0) {
    plan->prefix_tiles = a->shared_prefix_pages * a->page_size / zl::kGqaTile;
    plan->sgs = 16 / rps > 0 ? 16 / rps : 1;
    plan->ng = (a->B + plan->sgs - 1) / plan->sgs;
    if (plan->ng + a->B > zl::kMaxBatch) return ZL_ERR_UNSUPPORTED;  // one tile-count table
  }
  const int rows_per_warp = plan->prefix_tiles > 0 ? plan->sgs * rps : rps;
  int grid = a->num_ctas;
  if (grid == 0) {
    // the kernel's tile-offset table: one entry per unit (prefix groups and
    // sequences) plus the total; the launch takes the same layout
    const bool small = (plan->prefix_tiles > 0 ? plan->ng : 0) + a->B + 1 <= zl::kSmallTable;
    const int per_sm =
        mods ? zl::gqa_mod_ctas_per_sm(plan->hpc, rps > 8, plan->tg, small, dev.device)
        : plan->prefix_tiles > 0
            ? zl::gqa_shared_ctas_per_sm(plan->hpc, rows_per_warp > 8, a->q_len > 1, small,
                                         dev.device)
            : zl::gqa_ctas_per_sm(plan->hpc, rps > 8, a->q_len > 1, plan->fused, plan->tg, small,
                                  dev.device);
    if (per_sm < 1) return ZL_ERR_CUDA;
    grid = dev.sms * per_sm;
    if (a->max_seq_len > 0 && plan->prefix_tiles == 0) {
      // a window bounds what a sequence reads: the tiles from its oldest
      // token on (which may start inside a tile)
      int64_t max_len = a->max_seq_len;
      if (mods && mods->window > 0)
        max_len = std::min(max_len, int64_t(mods->window) + a->q_len + zl::kGqaTile);
      const int64_t max_tiles = (max_len + zl::kGqaTile - 1) / zl::kGqaTile;
      const int64_t units = int64_t(a->B) * plan->nhg;
      if (units <= grid && max_tiles <= zl::kGqaUnitCutTiles) {
        // Short contexts: one CTA per whole unit. Streaming the longest unit
        // alone costs less than cutting units and merging their pieces.
        plan->unit_cut = true;
        plan->fused = false;
        grid = int(units);
      } else {
        // No more CTAs than tiles: B * head groups * ceil(max_seq_len / 16).
        const int64_t tiles = units * max_tiles;
        if (tiles < grid) grid = int(tiles < 1 ? 1 : tiles);
      }
    }
  }
  plan->grid = grid;
  // partial slots: 2 per (token group, CTA) pair and consumer warp
  const size_t rows = size_t(grid) * plan->tg * 2 * plan->hpc * rows_per_warp;
  const size_t store_rows = plan->prefix_tiles > 0 ? size_t(a->B) * a->q_len * a->Hq : 0;
  // [0, off_lse): one arrival counter (8 bytes) per (sequence, kv head); then
  // the partials' lse and outputs; then (shared prefix) each query row's
  // result over its prefix part and over its suffix part when one CTA had the
  // whole unit: base-2 lse and normalised fp32 output.
  plan->off_lse = round_up(size_t(a->B) * a->Hkv * sizeof(unsigned long long), 256);
  plan->off_o = plan->off_lse + round_up(rows * sizeof(float), 256);
  plan->off_pre_lse = plan->off_o + round_up(rows * zl::kGqaHeadDim * sizeof(float), 256);
  plan->off_pre_o = plan->off_pre_lse + round_up(store_rows * sizeof(float), 256);
  plan->off_suf_lse =
      plan->off_pre_o + round_up(store_rows * zl::kGqaHeadDim * sizeof(float), 256);
  plan->off_suf_o = plan->off_suf_lse + round_up(store_rows * sizeof(float), 256);
  plan->bytes = plan->off_suf_o + store_rows * zl::kGqaHeadDim * sizeof(float);
  if (mods && mods->weights) {
    const size_t qrows = size_t(a->B) * a->q_len * a->Hq;
    plan->score_stride = int64_t(round_up(size_t(mods->weights_tokens), zl::kGqaTile));
    plan->off_stat = round_up(plan->bytes, 256);
    plan->off_scores = plan->off_stat + round_up(qrows * sizeof(float2), 256);
    plan->bytes = plan->off_scores + qrows * size_t(plan->score_stride) * sizeof(float);
  }
  return ZL_OK;
}

// A call with several groups of query tokens runs them in one launch, side by
// side, unless it merges inside the attention kernel (its arrival counters
// are per sequence and kv head) or has a shared prefix (one group only).
bool groups_together(const GqaPlan& plan) {
  return plan.ngroups > 1 && !plan.fused && plan.prefix_tiles == 0;
}

// ------------------------------------------------------------------ MLA plan
struct MlaPlan {
  int clusters = 0;
  size_t off_split = 0, off_span = 0, off_lse = 0, off_o = 0, bytes = 0;
};

zl_status mla_validate_shape(const zl_decode_attn_params* a) {
  if (!a || a->struct_size != sizeof(zl_decode_attn_params)) return ZL_ERR_INVALID_ARG;
  if (a->B < 1 || a->Hq < 1 || a->Hkv < 1 || a->q_len < 1 || a->page_size < 1 ||
      a->num_pages < 1 || a->block_table_stride < 1 || a->D_qk < 1 || a->D_v < 1 ||
      a->num_ctas < 0 || a->max_seq_len < 0)
    return ZL_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return ZL_ERR_INVALID_ARG;
  if (a->Hkv != 1) return ZL_ERR_INVALID_ARG;
  if (a->flags & ~uint32_t(ZL_DECODE_SINGLE_LAUNCH | ZL_DECODE_TEST_STALL))
    return ZL_ERR_INVALID_ARG;
  if (a->flags) return ZL_ERR_UNSUPPORTED;  // neither flag exists for MLA
  if (a->shared_prefix_pages != 0) return ZL_ERR_UNSUPPORTED;
  if (a->D_qk != zl::kMlaDqk || a->D_v != zl::kMlaDv) return ZL_ERR_UNSUPPORTED;
  if (a->Hq != zl::kMlaHeads) return ZL_ERR_UNSUPPORTED;
  if (a->page_size % zl::kMlaTile != 0 || a->page_size > 1024) return ZL_ERR_UNSUPPORTED;
  if (int64_t(a->B) * a->q_len > zl::kMlaMaxBatch) return ZL_ERR_UNSUPPORTED;
  return ZL_OK;
}

zl_status mla_plan(const zl_decode_attn_params* a, MlaPlan* plan) {
  zl_status st = mla_validate_shape(a);
  if (st != ZL_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != ZL_OK) return st;
  int clusters = a->num_ctas > 0 ? (a->num_ctas + 1) / 2 : dev.sms / 2;
  if (a->num_ctas == 0 && a->max_seq_len > 0) {
    const int64_t tiles =
        int64_t(a->B) * a->q_len *
        ((int64_t(a->max_seq_len) + zl::kMlaTile - 1) / zl::kMlaTile);
    if (tiles < clusters) clusters = int(tiles < 1 ? 1 : tiles);
  }
  if (clusters < 1) clusters = 1;
  plan->clusters = clusters;
  const size_t rows = size_t(clusters) * 2 * zl::kMlaHeads;
  // tile prefix sums per (sequence, query token) | first tile of each cluster |
  // first and last cluster of each unit | partial lse | partial outputs
  const size_t units = size_t(a->B) * a->q_len;
  plan->off_split = round_up((units + 1) * sizeof(int32_t), 256);
  plan->off_span = plan->off_split + round_up((size_t(clusters) + 1) * sizeof(int32_t), 256);
  plan->off_lse = plan->off_span + round_up(units * 2 * sizeof(int32_t), 256);
  plan->off_o = plan->off_lse + round_up(rows * sizeof(float), 256);
  plan->bytes = plan->off_o + rows * zl::kMlaDv * sizeof(float);
  return ZL_OK;
}

// Tensor maps this thread encoded recently, so a decode loop over the same
// pools skips the driver call (the map is a plain 128-byte value).
struct PoolMapKey {
  const void* pool;
  int64_t page_stride, token_stride, head_stride;
  int32_t D, page_size, Hkv, num_pages, box_heads, box_tokens;
  bool operator==(const PoolMapKey& o) const {
    return pool == o.pool && page_stride == o.page_stride && token_stride == o.token_stride &&
           head_stride == o.head_stride && D == o.D && page_size == o.page_size &&
           Hkv == o.Hkv && num_pages == o.num_pages && box_heads == o.box_heads &&
           box_tokens == o.box_tokens;
  }
};
constexpr int kMapCache = 8;
thread_local PoolMapKey t_map_keys[kMapCache];
thread_local CUtensorMap t_maps[kMapCache];
thread_local int t_map_used = 0, t_map_next = 0;

zl_status encode_pool_map(CUtensorMap* map, const void* pool, const zl_decode_attn_params* a,
                          int box_heads, int box_tokens = zl::kGqaTile) {
  const PoolMapKey key{pool, a->page_stride, a->token_stride, a->head_stride, a->D_qk,
                       a->page_size, a->Hkv, a->num_pages, box_heads, box_tokens};
  for (int i = 0; i < t_map_used; ++i)
    if (t_map_keys[i] == key) {
      *map = t_maps[i];
      return ZL_OK;
    }
  auto encode = tensor_map_encoder();
  if (!encode) return ZL_ERR_CUDA;
  const cuuint64_t dims[4] = {cuuint64_t(a->D_qk), cuuint64_t(a->page_size), cuuint64_t(a->Hkv),
                              cuuint64_t(a->num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(a->token_stride) * 2, cuuint64_t(a->head_stride) * 2,
                                 cuuint64_t(a->page_stride) * 2};
  const cuuint32_t box[4] = {64, cuuint32_t(box_tokens), cuuint32_t(box_heads), 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool),
                            dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return ZL_ERR_UNSUPPORTED;
  t_map_keys[t_map_next] = key;
  t_maps[t_map_next] = *map;
  t_map_next = (t_map_next + 1) % kMapCache;
  if (t_map_used < kMapCache) ++t_map_used;
  return ZL_OK;
}

// Query rows [B, q_len, Hq, 128] in boxes of g heads x tpt tokens.
zl_status encode_query_map(CUtensorMap* map, const zl_decode_attn_params* a, int g, int tpt) {
  auto encode = tensor_map_encoder();
  if (!encode) return ZL_ERR_CUDA;
  const cuuint64_t row = cuuint64_t(a->D_qk) * 2;
  const cuuint64_t dims[4] = {cuuint64_t(a->D_qk), cuuint64_t(a->Hq), cuuint64_t(a->q_len),
                              cuuint64_t(a->B)};
  const cuuint64_t strides[3] = {row, row * a->Hq, row * a->Hq * a->q_len};
  const cuuint32_t box[4] = {64, cuuint32_t(g), cuuint32_t(tpt), 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a->q),
                            dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ZL_OK : ZL_ERR_UNSUPPORTED;
}

zl_status validate_pointers(const zl_decode_attn_params* a, bool need_v) {
  if (!a->q || !a->k_pool || !a->block_table || !a->seq_lens || !a->out)
    return ZL_ERR_INVALID_ARG;
  if (need_v && !a->v_pool) return ZL_ERR_INVALID_ARG;
  if (!need_v && a->v_pool) return ZL_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->k_pool, 16) || !aligned(a->out, 16) ||
      (a->v_pool && !aligned(a->v_pool, 16)) || !aligned(a->block_table, 4) ||
      !aligned(a->seq_lens, 4) || (a->lse && !aligned(a->lse, 4)) ||
      (a->err_flags && !aligned(a->err_flags, 4)))
    return ZL_ERR_INVALID_ARG;
  if (a->page_stride <= 0 || a->token_stride <= 0 || a->head_stride <= 0 ||
      a->page_stride % 8 || a->token_stride % 8 || a->head_stride % 8)
    return ZL_ERR_INVALID_ARG;
  // fused KV append: GQA takes k_new and v_new together, MLA k_new alone
  if (!a->k_new && a->v_new) return ZL_ERR_INVALID_ARG;
  if (a->k_new && (need_v != (a->v_new != nullptr))) return ZL_ERR_INVALID_ARG;
  if ((a->k_new && !aligned(a->k_new, 16)) || (a->v_new && !aligned(a->v_new, 16)))
    return ZL_ERR_INVALID_ARG;
  return ZL_OK;
}

}  // namespace

namespace {

// Longest valid length of a sequence under modified scores (the kernels' sums of
// a length and a tile stay in 32 bits), and the window as the kernels take it:
// one that no sequence fills hides nothing, and its differences could leave 32
// bits.
int64_t mods_len_cap(const zl_decode_attn_params* a) {
  return std::min<int64_t>(a->block_table_stride * int64_t(a->page_size), INT32_MAX - 4096);
}
int mods_window(const zl_decode_attn_params* a, const zl_score_params& m) {
  return m.window >= mods_len_cap(a) ? 0 : m.window;
}

// The kernels' cap fields (kernels.h, gqa_wide.h) for scores c tanh(s / c).
template <class Params>
void set_cap(float scale, float c, Params* p) {
  if (!(c > 0.f)) return;
  p->cap_in = float(double(scale) / c);
  p->cap_out = float(double(c) * kLog2e);
  // coefficients and bound in the dot product's own units; where they leave
  // the range of normal 32-bit numbers, every score takes the full function
  const double in = double(scale) / c, poly[4] = ZL_CAP_POLYNOMIAL;
  bool normal = true;
  double f = in * c * kLog2e;
  for (int i = 0; i < 4; ++i, f *= in * in) {
    p->cap_f[i] = float(poly[i] * f);
    normal = normal && std::isnormal(p->cap_f[i]);
  }
  p->cap_z = float(0.25 / (in * in));
  if (!normal || !std::isnormal(p->cap_z)) {
    std::memset(p->cap_f, 0, sizeof(p->cap_f));
    p->cap_z = -1.f;
  }
}

// The modified-score launches: every row group in one attention launch, its
// merge, and the weights kernel when the call accumulates weights.
zl_status mods_run(const zl_decode_attn_params* a, const zl_score_params& m, const GqaPlan& plan,
                   GqaParams& p, char* ws, cudaStream_t s) {
  set_cap(a->scale, m.softcap, &p);
  p.slopes = m.alibi_slopes;
  p.window = mods_window(a, m);
  p.tree = m.tree_mask;
  p.tree_words = (a->q_len + 31) / 32;
  p.len_cap = mods_len_cap(a);
  if (m.weights) {
    p.len_cap = std::min(p.len_cap, int64_t(m.weights_tokens));
    p.row_stat = reinterpret_cast<float2*>(ws + plan.off_stat);
    p.scores = reinterpret_cast<float*>(ws + plan.off_scores);
    p.score_stride = plan.score_stride;
  }
  // one row group, two that share every CTA, or more side by side (see gqa_run)
  p.q_tok0 = 0;
  p.q_len = plan.q_group;
  p.ngroups = plan.ngroups;
  p.tg = plan.tg;
  p.group_ctas = plan.unit_cut || plan.tg == 2 ? plan.grid : std::max(1, plan.grid / plan.ngroups);
  const int grid = plan.tg == 2 ? plan.grid : p.group_ctas * plan.ngroups;
  DeviceInfo dev;
  const zl_status st = current_device(&dev);
  if (st != ZL_OK) return st;
  // eight warps to a merged row while that is about one wave of blocks: 256 rows
  // (8 sequences, 32 heads) 29.7 -> 24.1 us, one sequence of 60000 tokens 72 ->
  // 51; 512 rows 39.7 -> 40.6, 1024 rows 57.2 -> 62.3
  p.split_merge = int64_t(plan.ngroups) * a->B * a->Hkv * plan.gh * plan.q_group <= 2 * dev.sms;
  cudaError_t e = zl::gqa_mod_launch(p, grid, s, reinterpret_cast<cudaEvent_t>(a->attn_begin),
                                     reinterpret_cast<cudaEvent_t>(a->attn_end));
  if (e == cudaSuccess && m.weights) {
    zl::WeightsParams w;
    std::memset(&w, 0, sizeof(w));
    w.scores = p.scores;
    w.score_stride = p.score_stride;
    w.row_stat = p.row_stat;
    w.seq_lens = a->seq_lens;
    w.weights = m.weights;
    w.seq_stride = m.weights_seq_stride;
    w.head_stride = m.weights_head_stride;
    w.decay = m.weights_decay;
    w.B = a->B;
    w.q_total = a->q_len;
    w.Hq = a->Hq;
    w.Hkv = a->Hkv;
    w.g = plan.g;
    w.window = p.window;
    w.len_cap = p.len_cap;
    w.max_tokens = m.weights_tokens;
    e = zl::weights_launch(w, s);
  }
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

// A modified-score call with many rows per kv head (gqa_wide.cu). A fused
// append is a launch of its own here.
zl_status wide_run(const zl_decode_attn_params* a, const zl_score_params& m, const GqaPlan& plan,
                   cudaStream_t s) {
  zl::WideParams p;
  std::memset(&p, 0, sizeof(p));
  p.box = a->page_size % 128 == 0 ? 128 : a->page_size % 64 == 0 ? 64
          : a->page_size % 32 == 0 ? 32 : 16;
  zl_status st;
  if ((st = encode_pool_map(&p.tmap_k, a->k_pool, a, 1, p.box)) != ZL_OK) return st;
  if ((st = encode_pool_map(&p.tmap_v, a->v_pool, a, 1, p.box)) != ZL_OK) return st;
  if ((st = encode_query_map(&p.tmap_q, a, plan.g, plan.tpt)) != ZL_OK) return st;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.block_table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.bt_stride = a->block_table_stride;
  char* ws = static_cast<char*>(a->workspace);
  p.ws_cut = reinterpret_cast<int4*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + plan.off_lse);
  p.ws_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.err_flags = a->err_flags;
  p.B = a->B;
  p.q_total = a->q_len;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = plan.g;
  p.page_size = a->page_size;
  p.num_pages = a->num_pages;
  p.tpt = plan.tpt;
  p.mt = plan.mt;
  p.nblk = plan.nblk;
  p.whole_units = plan.unit_cut ? 2 : a->num_ctas == 0 ? 1 : 0;
  p.len_cap = mods_len_cap(a);
  p.scale_log2 = float(double(a->scale) * kLog2e);
  set_cap(a->scale, m.softcap, &p);
  p.slopes = m.alibi_slopes;
  p.window = mods_window(a, m);
  p.tree = m.tree_mask;
  p.tree_words = (a->q_len + 31) / 32;
  if (a->k_new) {
    zl_kv_append_params ap;
    std::memset(&ap, 0, sizeof(ap));
    ap.struct_size = sizeof(ap);
    ap.k_new = a->k_new;
    ap.v_new = a->v_new;
    ap.k_pool = const_cast<void*>(a->k_pool);
    ap.v_pool = const_cast<void*>(a->v_pool);
    ap.page_stride = a->page_stride;
    ap.token_stride = a->token_stride;
    ap.head_stride = a->head_stride;
    ap.block_table = a->block_table;
    ap.block_table_stride = a->block_table_stride;
    ap.seq_lens = a->seq_lens;
    ap.B = a->B;
    ap.q_len = a->q_len;
    ap.Hkv = a->Hkv;
    ap.D_k = a->D_qk;
    ap.D_v = a->D_v;
    ap.page_size = a->page_size;
    ap.num_pages = a->num_pages;
    ap.err_flags = a->err_flags;
    if ((st = zl::kv_append_run(&ap, false, s)) != ZL_OK) return st;
  }
  const cudaError_t e = zl::gqa_wide_launch(p, plan.grid, plan.unit_cut, s,
                                            reinterpret_cast<cudaEvent_t>(a->attn_begin),
                                            reinterpret_cast<cudaEvent_t>(a->attn_end));
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

// zl_decode_attn (mods = nullptr) and zl_decode_attn_ex.
zl_status gqa_run(const zl_decode_attn_params* a, const zl_score_params* mods,
                  zl_stream_t stream) {
  zl_status st = gqa_validate_shape(a);
  if (st != ZL_OK) return st;
  if (mods && (st = mods_validate(a, mods)) != ZL_OK) return st;
  if ((st = validate_pointers(a, true)) != ZL_OK) return st;
  GqaPlan plan;
  if ((st = gqa_plan(a, &plan, mods)) != ZL_OK) return st;
  if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < plan.bytes)
    return ZL_ERR_WORKSPACE;

  if (plan.wide) return wide_run(a, *mods, plan, reinterpret_cast<cudaStream_t>(stream));

  GqaParams p;
  std::memset(&p, 0, sizeof(p));
  if ((st = encode_pool_map(&p.tmap_k, a->k_pool, a, plan.hpc)) != ZL_OK) return st;
  if ((st = encode_pool_map(&p.tmap_v, a->v_pool, a, plan.hpc)) != ZL_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.block_table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.bt_stride = a->block_table_stride;
  char* ws = static_cast<char*>(a->workspace);
  p.ws_count = reinterpret_cast<unsigned long long*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + plan.off_lse);
  p.ws_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.err_flags = a->err_flags;
  p.epoch = next_epoch();
  p.test_stall = (a->flags & ZL_DECODE_TEST_STALL) ? 1 : 0;
  p.B = a->B;
  p.unit_cut = plan.unit_cut ? 1 : 0;
  p.auto_cut = (a->num_ctas == 0 && !plan.unit_cut && plan.prefix_tiles == 0) ? 1 : 0;
  p.q_total = a->q_len;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = plan.g;
  p.gh = plan.gh;
  p.hchunks = plan.hchunks;
  p.hc0 = 0;
  p.page_size = a->page_size;
  p.num_pages = a->num_pages;
  p.hpc = plan.hpc;
  p.nhg = plan.nhg;
  p.scale_log2 = float(double(a->scale) * kLog2e);
  p.prefix_tiles = plan.prefix_tiles;
  p.sgs = plan.sgs;
  p.ng = plan.ng;
  p.pre_lse = reinterpret_cast<float*>(ws + plan.off_pre_lse);
  p.pre_o = reinterpret_cast<float*>(ws + plan.off_pre_o);
  p.suf_lse = reinterpret_cast<float*>(ws + plan.off_suf_lse);
  p.suf_o = reinterpret_cast<float*>(ws + plan.off_suf_o);
  if (a->k_new) {  // the attention launch stores the new tokens' rows first
    p.k_new = static_cast<const uint4*>(a->k_new);
    p.v_new = static_cast<const uint4*>(a->v_new);
    p.k_pool = static_cast<uint4*>(const_cast<void*>(a->k_pool));
    p.v_pool = static_cast<uint4*>(const_cast<void*>(a->v_pool));
    p.page_stride16 = a->page_stride / 8;
    p.token_stride16 = a->token_stride / 8;
    p.head_stride16 = a->head_stride / 8;
  }

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (mods) return mods_run(a, *mods, plan, p, ws, s);
  const int ngroups = plan.ngroups;
  if (groups_together(plan)) {
    // Every row group (q_group query tokens, gh heads of each kv head) in one
    // launch, side by side: two share every CTA; more split the grid's CTAs
    // between them, and each cuts the same tile line, so the groups read each
    // K/V tile at about the same time (all but the first read are served by
    // L2). One merge launch covers every group.
    p.q_tok0 = 0;
    p.q_len = plan.q_group;
    p.ngroups = ngroups;
    p.tg = plan.tg;
    // two groups per CTA: each group has every CTA; else the grid is split.
    // The partial slots are sized for plan.grid (group, CTA) pairs: with
    // floor(grid / ngroups) >= 1 CTAs per group the pairs are at most that; a
    // group with one CTA (more groups than CTAs) takes the whole tile line,
    // so it cuts no unit and writes no partial (nor does a unit-cut launch).
    p.group_ctas = plan.unit_cut || plan.tg == 2 ? plan.grid : std::max(1, plan.grid / ngroups);
    const int launch_grid = plan.tg == 2 ? plan.grid : p.group_ctas * ngroups;
    const cudaError_t e = zl::gqa_decode_launch(
        p, launch_grid, false, s, reinterpret_cast<cudaEvent_t>(a->attn_begin),
        reinterpret_cast<cudaEvent_t>(a->attn_end));
    return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
  }
  // One launch (attention, then its merge) per row group: group gg is query
  // tokens from (gg / hchunks) * q_group, head chunk gg % hchunks. attn_begin
  // is recorded before the first, attn_end after the last attention launch.
  // The launches share the workspace: each reads it only after the one before
  // has finished (programmatic dependent launches).
  p.ngroups = 1;
  p.tg = 1;
  p.group_ctas = plan.grid;
  for (int gg = 0; gg < ngroups; ++gg) {
    const int tok0 = gg / plan.hchunks * plan.q_group;
    p.q_tok0 = tok0;
    p.q_len = std::min(plan.q_group, a->q_len - tok0);
    p.hc0 = gg % plan.hchunks;
    if (gg > 0) p.epoch = next_epoch();
    const bool first = gg == 0, last = gg == ngroups - 1;
    cudaEvent_t begin = first ? reinterpret_cast<cudaEvent_t>(a->attn_begin) : nullptr;
    cudaEvent_t end = last ? reinterpret_cast<cudaEvent_t>(a->attn_end) : nullptr;
    const cudaError_t e = plan.prefix_tiles > 0
                              ? zl::gqa_shared_launch(p, plan.grid, s, begin, end)
                              : zl::gqa_decode_launch(p, plan.grid, plan.fused, s, begin, end);
    if (e != cudaSuccess) return ZL_ERR_CUDA;
  }
  return ZL_OK;
}

}  // namespace

extern "C" {

const char* zl_status_string(zl_status s) {
  switch (s) {
    case ZL_OK: return "ok";
    case ZL_ERR_INVALID_ARG: return "invalid argument";
    case ZL_ERR_UNSUPPORTED: return "unsupported shape or layout";
    case ZL_ERR_WORKSPACE: return "workspace missing or too small";
    case ZL_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

zl_status zl_decode_attn_workspace_size(const zl_decode_attn_params* a, size_t* bytes) {
  if (!bytes) return ZL_ERR_INVALID_ARG;
  GqaPlan plan;
  const zl_status st = gqa_plan(a, &plan);
  if (st != ZL_OK) return st;
  *bytes = plan.bytes;
  return ZL_OK;
}

zl_status zl_decode_attn_launches(const zl_decode_attn_params* a, int32_t* launches) {
  if (!launches) return ZL_ERR_INVALID_ARG;
  GqaPlan plan;
  const zl_status st = gqa_plan(a, &plan);
  if (st != ZL_OK) return st;
  const int per_launch = (plan.fused || plan.unit_cut) ? 1 : 2;
  *launches = groups_together(plan) ? per_launch : plan.ngroups * per_launch;
  return ZL_OK;
}

zl_status zl_decode_attn(const zl_decode_attn_params* a, zl_stream_t stream) {
  return gqa_run(a, nullptr, stream);
}

zl_status zl_decode_attn_ex_workspace_size(const zl_decode_attn_params* a,
                                           const zl_score_params* mods, size_t* bytes) {
  if (!bytes || !mods) return ZL_ERR_INVALID_ARG;
  GqaPlan plan;
  const zl_status st = gqa_plan(a, &plan, mods);
  if (st != ZL_OK) return st;
  *bytes = plan.bytes;
  return ZL_OK;
}

zl_status zl_decode_attn_ex(const zl_decode_attn_params* a, const zl_score_params* mods,
                            zl_stream_t stream) {
  if (!mods) return ZL_ERR_INVALID_ARG;
  return gqa_run(a, mods, stream);
}

zl_status zl_decode_attn_mla_workspace_size(const zl_decode_attn_params* a, size_t* bytes) {
  if (!bytes) return ZL_ERR_INVALID_ARG;
  MlaPlan plan;
  const zl_status st = mla_plan(a, &plan);
  if (st != ZL_OK) return st;
  *bytes = plan.bytes;
  return ZL_OK;
}

zl_status zl_decode_attn_mla(const zl_decode_attn_params* a, zl_stream_t stream) {
  zl_status st = mla_validate_shape(a);
  if (st != ZL_OK) return st;
  if ((st = validate_pointers(a, false)) != ZL_OK) return st;
  MlaPlan plan;
  if ((st = mla_plan(a, &plan)) != ZL_OK) return st;
  if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < plan.bytes)
    return ZL_ERR_WORKSPACE;
  auto encode = tensor_map_encoder();
  if (!encode) return ZL_ERR_CUDA;

  zl::MlaParams p;
  std::memset(&p, 0, sizeof(p));
  {
    const cuuint64_t dims[3] = {cuuint64_t(zl::kMlaDqk), cuuint64_t(a->page_size),
                                cuuint64_t(a->num_pages)};
    const cuuint64_t strides[2] = {cuuint64_t(a->token_stride) * 2, cuuint64_t(a->page_stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(zl::kMlaTile), 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    if (encode(&p.tmap_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a->k_pool), dims,
               strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return ZL_ERR_UNSUPPORTED;
  }
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.block_table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.bt_stride = a->block_table_stride;
  char* ws = static_cast<char*>(a->workspace);
  p.ws_prefix = reinterpret_cast<int32_t*>(ws);
  p.ws_split = reinterpret_cast<int32_t*>(ws + plan.off_split);
  p.ws_span = reinterpret_cast<int32_t*>(ws + plan.off_span);
  p.ws_lse = reinterpret_cast<float*>(ws + plan.off_lse);
  p.ws_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.err_flags = a->err_flags;
  p.B = a->B;
  p.q_len = a->q_len;
  p.page_size = a->page_size;
  p.num_pages = a->num_pages;
  p.scale_log2 = float(double(a->scale) * kLog2e);
  p.out_align32 = aligned(a->out, 32) ? 1 : 0;
  if (a->k_new) {  // the attention launch stores the new tokens' latent rows first
    p.kv_new = static_cast<const uint4*>(a->k_new);
    p.kv_pool = static_cast<uint4*>(const_cast<void*>(a->k_pool));
    p.page_stride16 = a->page_stride / 8;
    p.token_stride16 = a->token_stride / 8;
  }
  const cudaError_t e = zl::mla_decode_launch(p, plan.clusters,
                                              reinterpret_cast<cudaStream_t>(stream),
                                              reinterpret_cast<cudaEvent_t>(a->attn_begin),
                                              reinterpret_cast<cudaEvent_t>(a->attn_end));
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

}  // extern "C"
