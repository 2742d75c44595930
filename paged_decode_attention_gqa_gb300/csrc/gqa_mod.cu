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
  return launch_merge<kModeMod>(p, stream);
}

}  // namespace zl
