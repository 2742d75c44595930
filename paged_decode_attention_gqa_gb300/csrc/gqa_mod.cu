// GQA decode with modified scores: kernel instances and launches.
//
// For query row (token i, head h) at position pos_i and cached token t at
// position pos_t, with the scaled score s = scale q.k_t:
//   cap     s <- c tanh(s / c)
//   bias    s <- s - slope_h (pos_i - pos_t)
//   window  token t is seen only if pos_i - pos_t < window
//   tree    drafted token j (the j-th of the last q_len) is seen only if bit j
//           of row i's ancestor mask is set; positions then count ancestors
// The kernel is gqa_decode_kernel (gqa_kernel.cuh) in its kModeMod instances: the
// same tile line, TMA ring and online softmax, with every row masked on its
// own. Tiles wholly before the oldest row's window are left out of the line,
// so a windowed call reads only what it sees.
#include "gqa_kernel.cuh"

namespace zl {

namespace {

// The merge of a modified-score call with few rows: a block per row, its
// kSplitWarps warps taking the unit's pieces in equal runs; the runs' results
// are then merged like pieces, in order. With a warp per row, 64 KB per SM of
// partials wait on one chain of reads (8 sequences cut into 19 pieces each: 8
// us; one sequence of 60000 tokens: 16).
constexpr int kSplitWarps = 8;

__global__ void __launch_bounds__(kSplitWarps * 32)
gqa_merge_split_kernel(const __grid_constant__ GqaParams p, int G) {
  __shared__ float s_lse[kSplitWarps];
  __shared__ float4 s_o[kSplitWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rmax = p.gh * p.q_len;
  const int64_t per_group = int64_t(p.B) * p.Hkv * rmax, item = blockIdx.x;
  const int tg = int(item / per_group);
  const int64_t gitem = item - tg * per_group;
  const int unit = int(gitem / rmax), r0 = int(gitem % rmax);
  const int b = unit / p.Hkv, kvh = unit % p.Hkv;
  const RowGroup rg = row_group(p, tg);
  int before = 0, all = 0, nmax = 0;
  for (int s = lane; s < p.B; s += 32) {
    const int t = seq_unit_tiles<kModeMod>(p, p.seq_lens[s]);
    all += t;
    before += s < b ? t : 0;
    nmax = max(nmax, t);
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  nmax = __reduce_max_sync(0xffffffffu, nmax);
  const int n = seq_unit_tiles<kModeMod>(p, p.seq_lens[b]);
  griddep_wait();
  griddep_launch_dependents();
  if (r0 >= rg.gh * rg.qlen || n == 0) return;
  if (p.auto_cut && short_units(int64_t(p.B) * p.nhg, nmax, G)) return;
  const int hg = kvh / p.hpc, w = kvh % p.hpc;
  const int64_t W = int64_t(p.nhg) * all;
  const TileCut cut(W, cut_ctas(p, W, int64_t(p.B) * p.nhg, G));
  const int64_t U0 = int64_t(p.nhg) * before + int64_t(hg) * n;
  const int c_lo = cut.owner(U0), c_hi = cut.owner(U0 + n - 1);
  if (c_lo == c_hi) return;
  const int per = (c_hi - c_lo + kSplitWarps) / kSplitWarps;  // pieces of a warp
  const int from = c_lo + warp * per, to = min(c_hi, from + per - 1);
  MergeAcc<1> m;
  m.init();
  if (from <= to)
    merge_add_pieces<1, 8>(m, p, cut, tg * G, U0, c_lo, to, w, rmax, 0, r0, 1, lane, from);
  {
    const bool some = !no_weight<kModeMod>(m.den[0]);
    const float inv = some ? __frcp_rn(m.den[0]) : 0.f;
    s_o[warp][lane] = make_float4(m.acc[0].x * inv, m.acc[0].y * inv, m.acc[0].z * inv,
                                  m.acc[0].w * inv);
    if (lane == 0)
      s_lse[warp] = m.bad              ? CUDART_NAN_F
                    : isnan(m.den[0]) ? CUDART_INF_F
                    : some            ? m.mx[0] + log2f(m.den[0])
                                      : -CUDART_INF_F;
  }
  __syncthreads();
  if (warp != 0) return;
  m.init();
#pragma unroll
  for (int k = 0; k < kSplitWarps; ++k) m.add(0, s_lse[k], s_o[k][lane]);
  merge_write_out<kModeMod>(m, p, b, rg.tok0, kvh * p.g + rg.hoff, rg.gh, r0, 1, lane);
}

template <int HPC, bool R16, int TG>
struct ModInstance {
  static cudaError_t launch(const GqaParams& p, int grid, cudaStream_t stream) {
    return launch_attn<HPC, R16, true, false, kModeMod, TG>(p, grid, stream);
  }
  static int ctas_per_sm(bool small, int device) {
    return occupancy<HPC, R16, true, false, kModeMod, TG>(device, small);
  }
};

// The instance for (heads per CTA, 16 rows, row groups per CTA); two row
// groups per CTA come with at most 4 heads (api.cu halves them).
template <class F>
auto with_instance(int hpc, bool r16, int tg, F&& f) -> decltype(f(ModInstance<1, false, 1>())) {
  switch ((hpc * 2 + (r16 ? 1 : 0)) * 4 + tg) {
#define ZL_CASE(H, S, T) \
  case (H * 2 + S) * 4 + T: return f(ModInstance<H, bool(S), T>());
    ZL_CASE(1, 0, 1) ZL_CASE(1, 1, 1) ZL_CASE(2, 0, 1) ZL_CASE(2, 1, 1)
    ZL_CASE(4, 0, 1) ZL_CASE(4, 1, 1) ZL_CASE(8, 0, 1) ZL_CASE(8, 1, 1)
    ZL_CASE(1, 0, 2) ZL_CASE(1, 1, 2) ZL_CASE(2, 0, 2) ZL_CASE(2, 1, 2)
    ZL_CASE(4, 0, 2) ZL_CASE(4, 1, 2)
#undef ZL_CASE
    default: return {};
  }
}

}  // namespace

int gqa_mod_ctas_per_sm(int hpc, bool rows16, int tg, bool small, int device) {
  return with_instance(hpc, rows16, tg,
                       [&](auto inst) -> int { return inst.ctas_per_sm(small, device); });
}

cudaError_t gqa_mod_launch(const GqaParams& p, int grid, cudaStream_t stream,
                           cudaEvent_t attn_begin, cudaEvent_t attn_end) {
  cudaError_t e = cudaSuccess;
  const bool known = p.hpc == 1 || p.hpc == 2 || p.hpc == 4 || (p.hpc == 8 && p.tg == 1);
  if (!known || p.tg < 1 || p.tg > 2) return cudaErrorInvalidValue;
  if (attn_begin && (e = cudaEventRecord(attn_begin, stream)) != cudaSuccess) return e;
  e = with_instance(p.hpc, p.gh * p.q_len > 8, p.tg, [&](auto inst) -> cudaError_t {
    return inst.launch(p, grid, stream);
  });
  if (e != cudaSuccess) return e;
  if (attn_end && (e = cudaEventRecord(attn_end, stream)) != cudaSuccess) return e;
  if (p.unit_cut) return cudaSuccess;  // nothing to merge
  if (!p.split_merge) return launch_merge<kModeMod>(p, stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(int64_t(p.ngroups) * p.B * p.Hkv * p.gh * p.q_len));
  cfg.blockDim = dim3(kSplitWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gqa_merge_split_kernel, p, p.group_ctas);
}

}  // namespace zl
