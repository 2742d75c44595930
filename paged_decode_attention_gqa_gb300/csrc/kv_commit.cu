// Commit of a drafted tree's accepted path (zl_kv_commit in the header): the K
// and V rows of drafted token path[j] move to position ctx + j, ctx =
// seq_lens[b] - q_len.
//
// One block per (sequence, kv head, 256-byte column part of K or V): at most
// 128 rows of 256 bytes, 8 chunks of 16 bytes per thread, all read before any
// is written, so any path is safe in place. The first block of a (sequence, kv
// head) also moves the tokens' sums of weights, the same way. The whole call is
// a few hundred KB: it is bound by the chain of dependent reads (length, path,
// page, row), which all blocks walk at once.
#include "kv_move.cuh"
#include "kernels.h"
#include "ptx.cuh"

#include <cstddef>
#include <cstring>

namespace zl {
namespace {

constexpr int kThreads = 256;
constexpr int kPart = 16;                       // 16-byte chunks per column part
constexpr int kRowsPerPass = kThreads / kPart;  // 16
constexpr int kPasses = 8;
constexpr int kMaxDrafted = kRowsPerPass * kPasses;  // 128

struct CommitParams {
  MovePools pools;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* path;
  int64_t path_stride;
  const int32_t* accepted;
  int32_t* new_lens;
  uint32_t* err_flags;
  int q_len, max_accepted, k_parts;
  float* weights;  // [B][Hkv][w_tokens], strides in elements; nullptr: none
  int64_t w_seq, w_head;
  int w_tokens;
};

__global__ void __launch_bounds__(kThreads)
kv_commit_kernel(const __grid_constant__ CommitParams p) {
  griddep_launch_dependents();
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const bool is_v = int(blockIdx.x) >= p.k_parts;
  const int part = is_v ? int(blockIdx.x) - p.k_parts : int(blockIdx.x);
  const int width = is_v ? p.pools.cv : p.pools.ck;
  uint4* pool = is_v ? p.pools.v : p.pools.k;
  const int col = part * kPart + tid % kPart, r0 = tid / kPart;
  const bool first = blockIdx.x == 0 && h == 0;  // reports for the sequence

  const int L = __ldg(p.seq_lens + b), n = __ldg(p.accepted + b);
  const bool len_ok = L >= p.q_len && int64_t(L) <= p.bt_stride * p.pools.page_size &&
                      (!p.weights || L <= p.w_tokens);
  bool path_ok = n >= 0 && n <= p.max_accepted;
  int src[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int j = i * kRowsPerPass + r0;
    src[i] = path_ok && j < n ? __ldg(p.path + int64_t(b) * p.path_stride + j) : 0;
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) path_ok = path_ok && src[i] >= 0 && src[i] < p.q_len;
  path_ok = !__syncthreads_or(!path_ok);
  if (!len_ok || !path_ok) {
    if (first && tid == 0) {
      p.new_lens[b] = L;
      if (p.err_flags) atomicOr(p.err_flags, (len_ok ? 0u : 2u) | (path_ok ? 0u : 16u));
    }
    return;
  }
  const int ctx = L - p.q_len;
  if (first && tid == 0) p.new_lens[b] = ctx + n;
  const int32_t* bt = p.block_table + int64_t(b) * p.bt_stride;
  // sums of the drafted tokens, from ctx on
  float* w = p.weights && blockIdx.x == 0
                 ? p.weights + int64_t(b) * p.w_seq + int64_t(h) * p.w_head + ctx
                 : nullptr;
  float sum = 0.f;
  if (w && tid < n) sum = w[__ldg(p.path + int64_t(b) * p.path_stride + tid)];
  uint4 data[kPasses];
  uint4* dst[kPasses];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int j = i * kRowsPerPass + r0;
    dst[i] = nullptr;
    if (j >= n || src[i] == j || col >= width) continue;
    const int ts = ctx + src[i], td = ctx + j;
    const int ps = __ldg(bt + ts / p.pools.page_size), pd = __ldg(bt + td / p.pools.page_size);
    if (ps < 0 || ps >= p.pools.num_pages || pd < 0 || pd >= p.pools.num_pages) {
      bad = true;
      continue;
    }
    data[i] = pool[p.pools.row(ps, ts % p.pools.page_size, h) + col];
    dst[i] = pool + p.pools.row(pd, td % p.pools.page_size, h) + col;
  }
  __syncthreads();  // every row of this part is read, and every sum
  if (w && tid < p.q_len) w[tid] = sum;  // 0 behind the accepted ones
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (dst[i]) *dst[i] = data[i];
  if (bad && p.err_flags) atomicOr(p.err_flags, 1u);
}

}  // namespace
}  // namespace zl

extern "C" zl_status zl_kv_commit(const zl_kv_commit_params* params, zl_stream_t stream) {
  zl_kv_commit_params given;
  if (!zl::take_params(params, offsetof(zl_kv_commit_params, weights), &given))
    return ZL_ERR_INVALID_ARG;
  const zl_kv_commit_params* a = &given;
  zl::CommitParams p;
  std::memset(&p, 0, sizeof(p));
  const zl_status st = zl::move_pools(a, &p.pools);
  if (st != ZL_OK) return st;
  if (!a->path || !a->accepted || !zl::aligned_to(a->path, 4) || !zl::aligned_to(a->accepted, 4))
    return ZL_ERR_INVALID_ARG;
  if (a->q_len < 1 || a->path_len < 1 || a->path_stride < a->path_len)
    return ZL_ERR_INVALID_ARG;
  if (a->weights &&
      (!zl::aligned_to(a->weights, 4) || a->weights_tokens < 1 ||
       !zl::rows_distinct(a->B, a->Hkv, a->weights_seq_stride, a->weights_head_stride,
                          a->weights_tokens)))
    return ZL_ERR_INVALID_ARG;
  // (one block writes a sequence's new length while others still read its
  // accepted count and path)
  if (zl::overlaps(a->new_lens, a->B, a->accepted, a->B) ||
      zl::overlaps(a->new_lens, a->B, a->path, (a->B - 1) * a->path_stride + a->path_len))
    return ZL_ERR_INVALID_ARG;
  if (a->q_len > zl::kMaxDrafted) return ZL_ERR_UNSUPPORTED;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.seq_lens = a->seq_lens;
  p.path = a->path;
  p.path_stride = a->path_stride;
  p.accepted = a->accepted;
  p.new_lens = a->new_lens;
  p.err_flags = a->err_flags;
  p.q_len = a->q_len;
  p.weights = a->weights;
  p.w_seq = a->weights_seq_stride;
  p.w_head = a->weights_head_stride;
  p.w_tokens = a->weights_tokens;
  p.max_accepted = a->path_len < a->q_len ? a->path_len : a->q_len;
  p.k_parts = (p.pools.ck + zl::kPart - 1) / zl::kPart;
  const int parts = p.k_parts + (p.pools.cv + zl::kPart - 1) / zl::kPart;
  const dim3 grid(parts, a->Hkv, a->B);
  zl::kv_commit_kernel<<<grid, zl::kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
