// Accumulated attention weights: how much each cached token was attended to.
//
//   weights[b, kh, t] <- decay weights[b, kh, t] + sum over the sequence's
//   query tokens i and the g query heads of kv head kh of softmax_t(scores),
//
// for t < seq_lens[b]. The attention kernel keeps every base-2 score x it
// computed and, per query row, the final softmax base m and 1 / l, so a weight
// is 2^(x - m) / l: 4 bytes written and read per (row, token) instead of a
// second pass over K (256 bytes per token and kv head). Each weight is summed
// by one thread in row order: no atomics, the same bits every time.
#include "kernels.h"
#include "ptx.cuh"

namespace zl {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;    // tokens per thread, kThreads apart
constexpr int kRows = 4;   // query rows whose scores are read together

__global__ void __launch_bounds__(kThreads)
attn_weights_kernel(const __grid_constant__ WeightsParams p) {
  // A programmatic dependent of the attention launch's last kernel.
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.y, b = blockIdx.z;
  const int L = p.seq_lens[b];
  if (L < 0 || int64_t(L) > p.len_cap) return;  // flagged by the attention
  const int t0 = int(blockIdx.x) * (kThreads * kPer);
  if (t0 >= L) return;
  // tokens before the oldest window have no stored score
  const int lo = p.window ? max(L - p.q_total - p.window + 1, 0) : 0;
  float sum[kPer] = {0.f, 0.f, 0.f, 0.f};
  const int t = t0 + threadIdx.x;
  if (t0 + kThreads * kPer > lo) {
    for (int i = 0; i < p.q_total; ++i) {
      const int64_t row0 = (int64_t(b) * p.q_total + i) * p.Hq + int64_t(h) * p.g;
      // 16 loads in flight per thread (one row at a time took twice as long)
      for (int j = 0; j < p.g; j += kRows) {
        float2 stat[kRows];
        float x[kRows][kPer];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          // (0, 0): a row without weight, or over a bad page, or past the last
          stat[r] = j + r < p.g ? __ldg(p.row_stat + row0 + j + r) : make_float2(0.f, 0.f);
          const float* s = p.scores + (row0 + min(j + r, p.g - 1)) * p.score_stride;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int tk = t + k * kThreads;
            x[r][k] = tk >= lo && tk < L ? __ldcs(s + tk) : 0.f;
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (stat[r].y == 0.f) continue;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int tk = t + k * kThreads;
            if (tk >= lo && tk < L) sum[k] += ex2_approx(x[r][k] - stat[r].x) * stat[r].y;
          }
        }
      }
    }
  }
  float* w = p.weights + int64_t(b) * p.seq_stride + int64_t(h) * p.head_stride;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int tk = t + k * kThreads;
    if (tk >= L) continue;
    // decay 0 starts over: what the buffer held before (NaN even) does not count
    w[tk] = p.decay == 0.f ? sum[k] : fmaf(p.decay, w[tk], sum[k]);
  }
}

}  // namespace

cudaError_t weights_launch(const WeightsParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.max_tokens + kThreads * kPer - 1) / (kThreads * kPer)),
                     unsigned(p.Hkv), unsigned(p.B));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_weights_kernel, p);
}

}  // namespace zl
