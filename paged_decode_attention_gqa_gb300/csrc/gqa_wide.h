// Interface between the C-ABI front end and the many-row kernel (gqa_wide.cu).
#pragma once

#include "kernels.h"

namespace zl {

constexpr int kWideTile = 128;  // tokens per tile
// What a unit costs beside its tiles, in tiles, for the cut between CTAs.
// (64 sequences of 512-4096 tokens, 64 drafted tokens: 196, 177, 172, 172, 178 us
// at 0, 1, 2, 3 and 5; 16 drafted tokens: 137, 128, 129, 130, 132 us.)
constexpr int kWideUnitCost = 2;
// Units of at most this many tiles are not cut: a CTA each, or the line is cut
// at the nearest unit's start. (256 units of 128-512 tokens, 16 drafted tokens, 4 heads:
// 29.9 us cut, 28.7 whole, 512 units 47.9 and 43.9, with 64 drafted tokens 65.6
// and 58.4; with 8 tiles allowed, 160 units of 512-1024 tokens 28.8 and 32.9.)
constexpr int kWideWholeTiles = 4;

// tanh(y) / y for z = y^2 in [0, 1/4]: the cubic in z that interpolates it at
// the 4 Chebyshev nodes of the interval, within 5.5e-7 (6.3e-7
// evaluated in 32 bits): a score c tanh(s / c) is then off by 3e-7 of c at most.
#define ZL_CAP_POLYNOMIAL {0.999999451, -0.333262842, 0.131899394, -0.0443927384}

struct WideParams {
  CUtensorMap tmap_k;  // 4-D {D, page_size, Hkv, num_pages}, box {64, box, 1, 1}, 128B swizzle
  CUtensorMap tmap_v;
  CUtensorMap tmap_q;  // 4-D {D, Hq, q_total, B}, box {64, g, tpt, 1}, 128B swizzle
  __nv_bfloat16* out;
  float* lse;              // natural log, or nullptr
  const int32_t* block_table;
  const int32_t* seq_lens;
  int64_t bt_stride;
  int4* ws_cut;        // [CTAs] the unit each boundary cuts first, for the merge
  float* ws_lse;       // [CTAs][2][mt * 128] base-2 lse of partials (NaN bad, +inf NaN)
  float* ws_o;         // [..][128] normalised partial outputs
  uint32_t* err_flags;
  int B, q_total, Hq, Hkv, g, page_size, num_pages;
  int box;   // tokens per bulk copy: the largest of 128, 64, 32, 16 dividing page_size
  int tpt;   // query tokens per row tile: 128 / g
  int mt;    // row tiles per row block: 1 (the call has only one) or 2
  int nblk;  // row blocks per kv head
  // 2: a CTA per unit (the host knows a length bound and launches no merge); 1:
  // the default grid, the kernel decides by kWideWholeTiles; 0: units are cut
  int whole_units;
  int64_t len_cap;
  float scale_log2, cap_in, cap_out;  // as in GqaParams
  // The capped score in base 2 as x (cap_f[0] + cap_f[1] z + ..), z = x^2, of the
  // dot product x; right where z <= cap_z (-1: nowhere)
  float cap_f[4], cap_z;
  const float* slopes;
  int window;
  const uint32_t* tree;
  int tree_words;
};

// The attention kernel on `grid` CTAs, then the merge of the units it cut
// (no_merge: the caller knows that there are none).
cudaError_t gqa_wide_launch(const WideParams& p, int grid, bool no_merge, cudaStream_t stream,
                            cudaEvent_t attn_begin, cudaEvent_t attn_end);

}  // namespace zl
