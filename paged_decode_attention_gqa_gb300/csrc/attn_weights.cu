// Accumulated attention weights: how much each cached token was attended to.
//
//   weights[b, kh, t] <- decay weights[b, kh, t] + sum over the sequence's
//   query tokens i and the g query heads of kv head kh of softmax_t(scores),
//
// for t < seq_lens[b]. The attention kernel keeps every base-2 score x it
// computed and, per query row, the final softmax base m and 1 / l, so a weight
// is 2^(x - m) / l: 4 bytes written and read per (row, token) instead of a
// second pass over K (256 bytes per token and kv head). Up to 32 rows per kv
// head those are the fewer bytes; with more (drafted trees) it is the form there
// is, not the cheapest one. Each weight is summed in a fixed order: no atomics,
// the same bits every time.
#include "kernels.h"
#include "ptx.cuh"

#include <math_constants.h>

namespace zl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kQuad = 128;  // tokens of a warp: four per lane, one 16-byte load per row
constexpr int kRows = 4;    // query rows whose scores a warp reads together

// RW warps share 128 tokens and divide the query rows between them (their sums
// are added in the order of the warps); the block's kWarps / RW groups of warps
// have tokens of their own. RW grows with the rows, so that a warp has about
// kRows of them: with one thread per token and all rows in turn, 32 rows of
// 7493 tokens took 65 us.
template <int RW>
__global__ void __launch_bounds__(kThreads)
attn_weights_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int kTokens = kWarps / RW * kQuad;  // of the block
  __shared__ float4 part[RW > 1 ? kWarps : 1][32];
  // A programmatic dependent of the attention launch's last kernel.
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int L = p.seq_lens[b];
  if (L < 0 || int64_t(L) > p.len_cap) return;  // flagged by the attention
  const int t0 = int(blockIdx.x) * kTokens;
  if (t0 >= L) return;
  // Scores are stored for whole tiles of 16 tokens from the oldest window's on;
  // within them the ones a row does not see are -inf.
  const int lo = p.window ? max(L - p.q_total - p.window + 1, 0) / kGqaTile * kGqaTile : 0;
  const int t = t0 + warp / RW * kQuad + lane * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const int rows = p.q_total * p.g;
  if (t >= lo && t < L) {
    for (int r0 = warp % RW; r0 < rows; r0 += RW * kRows) {
      float2 stat[kRows];
      float4 x[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {  // loads of four rows in flight
        const int r = r0 + k * RW;
        stat[k] = make_float2(0.f, 0.f);  // (0, 0): no weight, or over a bad page
        if (r < rows) {
          const int64_t row =
              (int64_t(b) * p.q_total + r / p.g) * p.Hq + int64_t(h) * p.g + r % p.g;
          stat[k] = __ldg(p.row_stat + row);
          x[k] = __ldcs(reinterpret_cast<const float4*>(p.scores + row * p.score_stride + t));
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (stat[k].y == 0.f) continue;
        if (isnan(stat[k].y)) {  // a NaN row: every token that it sees
          sum.x += x[k].x == -CUDART_INF_F ? 0.f : CUDART_NAN_F;
          sum.y += x[k].y == -CUDART_INF_F ? 0.f : CUDART_NAN_F;
          sum.z += x[k].z == -CUDART_INF_F ? 0.f : CUDART_NAN_F;
          sum.w += x[k].w == -CUDART_INF_F ? 0.f : CUDART_NAN_F;
          continue;
        }
        sum.x += ex2_approx(x[k].x - stat[k].x) * stat[k].y;
        sum.y += ex2_approx(x[k].y - stat[k].x) * stat[k].y;
        sum.z += ex2_approx(x[k].z - stat[k].x) * stat[k].y;
        sum.w += ex2_approx(x[k].w - stat[k].x) * stat[k].y;
      }
    }
  }
  if constexpr (RW > 1) {
    part[warp][lane] = sum;
    __syncthreads();
    if (warp % RW != 0) return;
#pragma unroll
    for (int k = 1; k < RW; ++k) {
      const float4 o = part[warp + k][lane];
      sum.x += o.x;
      sum.y += o.y;
      sum.z += o.z;
      sum.w += o.w;
    }
  }
  float* w = p.weights + int64_t(b) * p.seq_stride + int64_t(h) * p.head_stride + t;
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (t + k >= L) continue;
    // decay 0 starts over: what the buffer held before (NaN even) does not count
    w[k] = p.decay == 0.f ? v[k] : fmaf(p.decay, w[k], v[k]);
  }
}

template <int RW>
cudaError_t launch(const WeightsParams& p, cudaStream_t stream) {
  constexpr int kTokens = kWarps / RW * kQuad;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.max_tokens + kTokens - 1) / kTokens), unsigned(p.Hkv),
                     unsigned(p.B));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_weights_kernel<RW>, p);
}

}  // namespace

cudaError_t weights_launch(const WeightsParams& p, cudaStream_t stream) {
  const int rows = p.q_total * p.g;
  if (rows <= kRows) return launch<1>(p, stream);
  if (rows <= 2 * kRows) return launch<2>(p, stream);
  if (rows <= 4 * kRows) return launch<4>(p, stream);
  return launch<8>(p, stream);
}

}  // namespace zl
