// Eviction by accumulated weights (zl_kv_evict in the header), in two launches.
//
// select: one block per (sequence, kv head) finds the K-th largest weight of
// the tokens between the sinks and the recent ones by a radix select on 32-bit
// keys that order as the floats do (11 + 11 + 10 bits, a histogram in shared
// memory each), then lists the kept positions in order: a token is kept if its
// key is above the threshold, or equals it and fewer than the missing number
// of equal ones came before it. Each warp owns a contiguous stretch, counts
// it, and after a scan over the warps writes its places; no atomics decide an
// order, so the result is always the same. The same block moves the weights.
//
// move: rows are 16-byte chunks. In place, kept[j] >= j, so the rows of one
// (sequence, kv head, column part) may move in ascending chunks: a chunk's
// sources lie at or above its first destination, and nothing later reads what
// an earlier chunk overwrote, but a chunk has to be read in full before it is
// written, and before any later chunk is. One block walks one column part;
// the next chunk's loads are in flight while this one is stored. Into other
// pages there is no such order and the rows are cut into segments as well.
#include "kv_move.cuh"
#include "kernels.h"
#include "ptx.cuh"

#include <cstring>

namespace zl {
namespace {

struct EvictParams {
  MovePools pools;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* dst_table;  // == block_table in place
  int64_t dst_stride;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* kept;             // [B, Hkv, budget]
  const float* weights;
  int64_t w_seq, w_head;
  float* weights_out;        // == weights in place
  int64_t wo_seq, wo_head;
  uint32_t* err_flags;
  int w_tokens, Hkv, budget, sink, recent;
  // move launch: column parts of K (then of V) of `part` chunks, segments of
  // kSegment rows (out of place; 1 in place)
  int part, k_parts, parts, segments;
};

__device__ __forceinline__ bool evict_len_ok(const EvictParams& p, int L) {
  const int64_t reach = p.bt_stride * p.pools.page_size;
  const int64_t dst_reach = p.dst_stride * p.pools.page_size;
  return L >= 0 && int64_t(L) <= reach && L <= p.w_tokens && int64_t(min(L, p.budget)) <= dst_reach;
}

// ------------------------------------------------------------------- select
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// A key that orders as the weights do: larger weight, larger key; -0 as +0,
// NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[kSelWarps], warp_eq[kSelWarps];
  __shared__ uint32_t s_prefix, s_need;
  griddep_wait();
  const int h = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = p.seq_lens[b];
  int32_t* kept = p.kept + (int64_t(b) * p.Hkv + h) * p.budget;
  const float* w = p.weights + int64_t(b) * p.w_seq + int64_t(h) * p.w_head;
  float* wo = p.weights_out + int64_t(b) * p.wo_seq + int64_t(h) * p.wo_head;
  if (!evict_len_ok(p, L)) {
    if (h == 0 && tid == 0 && p.err_flags) atomicOr(p.err_flags, 2u);
    for (int j = tid; j < p.budget; j += kSelThreads) kept[j] = -1;
    return;
  }
  if (L <= p.budget) {
    for (int j = tid; j < p.budget; j += kSelThreads) kept[j] = j < L ? j : -1;
    if (wo != w)
      for (int j = tid; j < L; j += kSelThreads) wo[j] = w[j];
    return;
  }
  const int M = L - p.sink - p.recent;                 // candidates
  const int K = p.budget - p.sink - p.recent;          // kept of them: K < M
  const float* c = w + p.sink;
  for (int j = tid; j < p.sink; j += kSelThreads) kept[j] = j;
  for (int j = tid; j < p.recent; j += kSelThreads)
    kept[p.budget - p.recent + j] = L - p.recent + j;
  if (K > 0) {
    // the K-th largest key, most significant digits first: `prefix` holds the
    // digits found, `need` how many of the keys that share them are kept
    uint32_t prefix = 0, need = uint32_t(K);
    int shift = 21;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      const uint32_t nb = 1u << bits;
      for (uint32_t i = tid; i < nb; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const int high = shift + bits;  // 32 in the first pass
      for (int i0 = 0; i0 < M; i0 += kSelThreads * 4) {
        uint32_t key[4];
        bool in[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * kSelThreads + tid;
          in[u] = i < M;
          key[u] = in[u] ? weight_key(c[i]) : 0u;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool take = in[u] && (high == 32 || (key[u] >> high) == prefix);
          const uint32_t bin = (key[u] >> shift) & (nb - 1u);
          // many equal weights (tokens nobody attended to): one add for a warp
          const uint32_t m = __ballot_sync(0xffffffffu, take);
          if (!m) continue;
          const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(m) - 1);
          const uint32_t same = __ballot_sync(0xffffffffu, take && bin == lead);
          if (take && bin != lead) atomicAdd(&hist[bin], 1u);
          if (lane == __ffs(m) - 1) atomicAdd(&hist[lead], __popc(same));
        }
      }
      __syncthreads();
      // the digit: the largest one with at least `need` keys at or above it.
      // Thread i owns bins [2i, 2i + 1]; suffix sums over the threads.
      const uint32_t per = nb / kSelThreads;  // 2 or 1
      uint32_t mine = 0;
      for (uint32_t k = 0; k < per; ++k) mine += hist[tid * per + k];
      uint32_t suf = mine;  // over lanes >= this one
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_down_sync(0xffffffffu, suf, off);
        if (lane + off < 32) suf += x;
      }
      if (lane == 0) warp_sum[warp] = suf;
      __syncthreads();
      uint32_t above = suf - mine;  // keys in bins above this thread's
      for (int k = warp + 1; k < kSelWarps; ++k) above += warp_sum[k];
      if (above < need && need <= above + mine) {
        for (int k = int(per) - 1; k >= 0; --k) {
          const uint32_t cnt = hist[tid * per + k];
          if (need <= above + cnt) {
            s_prefix = (prefix << bits) | uint32_t(tid * per + k);
            s_need = need - above;
            break;
          }
          above += cnt;
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      shift -= pass == 0 ? 11 : 10;
    }
    // `prefix` is the threshold key: every key above it is kept, and the first
    // `need` of those that equal it
    const uint32_t T = prefix;
    const int seg = ((M + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;  // a warp's stretch
    const int a0 = min(M, warp * seg), a1 = min(M, a0 + seg);
    uint32_t gt = 0, eq = 0;
    for (int i = a0 + lane; i < a1; i += 32) {
      const uint32_t key = weight_key(c[i]);
      gt += key > T ? 1u : 0u;
      eq += key == T ? 1u : 0u;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      gt += __shfl_xor_sync(0xffffffffu, gt, off);
      eq += __shfl_xor_sync(0xffffffffu, eq, off);
    }
    if (lane == 0) {
      warp_sum[warp] = gt;
      warp_eq[warp] = eq;
    }
    __syncthreads();
    uint32_t gt0 = 0, eq0 = 0;  // before this warp's stretch
    for (int k = 0; k < warp; ++k) {
      gt0 += warp_sum[k];
      eq0 += warp_eq[k];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = a0; i0 < a1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < a1 ? weight_key(c[i]) : 0u;
      const uint32_t g = __ballot_sync(0xffffffffu, i < a1 && key > T);
      const uint32_t e = __ballot_sync(0xffffffffu, i < a1 && key == T);
      const uint32_t gb = gt0 + __popc(g & below), eb = eq0 + __popc(e & below);
      const bool take = ((g >> lane) & 1u) || (((e >> lane) & 1u) && eb < need);
      if (take) kept[p.sink + gb + min(eb, need)] = p.sink + i;
      gt0 += __popc(g);
      eq0 += __popc(e);
    }
  }
  __syncthreads();
  // Weights move like the rows: ascending, a chunk read before it is written.
  for (int j0 = 0; j0 < p.budget; j0 += kSelThreads) {
    const int j = j0 + tid;
    float x = 0.f;
    if (j < p.budget) x = w[kept[j]];
    __syncthreads();
    if (j < p.budget) wo[j] = x;
  }
}

// --------------------------------------------------------------------- move
constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;       // chunks of 16 bytes per thread and step
constexpr int kSegment = 1024;   // rows whose places are looked up together

// Column part q of a row: chunks [c0, c0 + part) of K or V.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int64_t s_src[kSegment], s_dst[kSegment];  // row starts in chunks; -1: no move
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int seg = IN_PLACE ? 0 : int(blockIdx.x) / p.parts;
  const int q = IN_PLACE ? int(blockIdx.x) : int(blockIdx.x) % p.parts;
  const bool is_v = q >= p.k_parts;
  const int width = is_v ? p.pools.cv : p.pools.ck;
  const int col = (is_v ? q - p.k_parts : q) * p.part + tid % p.part;
  uint4* pool = is_v ? p.pools.v : p.pools.k;
  const int32_t* kept = p.kept + (int64_t(b) * p.Hkv + h) * p.budget;
  if (blockIdx.x == 0 && h == 0 && tid == 0) {
    const int L = p.seq_lens[b];
    p.new_lens[b] = evict_len_ok(p, L) ? min(L, p.budget) : L;
  }
  const int step_rows = kMoveThreads / p.part * kUnroll;  // rows of one step of the block
  const int32_t* sbt = p.block_table + int64_t(b) * p.bt_stride;
  const int32_t* dbt = p.dst_table + int64_t(b) * p.dst_stride;
  bool bad = false;
  const int first = seg * kSegment;
  const int last = IN_PLACE ? p.budget : min(p.budget, first + kSegment);
  for (int base = first; base < last; base += kSegment) {
    const int rows = min(kSegment, last - base);
    bool more = false;  // some row of the segment is kept
    for (int r = tid; r < rows; r += kMoveThreads) {
      const int j = base + r, t = kept[j];
      int64_t src = -1, dst = -1;
      if (t >= 0) {
        more = true;
        if (!IN_PLACE || t != j) {
          const int ps = __ldg(sbt + t / p.pools.page_size);
          const int pd = __ldg(dbt + j / p.pools.page_size);
          if (ps < 0 || ps >= p.pools.num_pages || pd < 0 || pd >= p.pools.num_pages) {
            bad = true;
          } else {
            src = p.pools.row(ps, t % p.pools.page_size, h);
            dst = p.pools.row(pd, j % p.pools.page_size, h);
          }
        }
      }
      s_src[r] = src;
      s_dst[r] = dst;
    }
    if (!__syncthreads_or(more)) break;  // kept entries end before this segment
    // steps of step_rows rows: load the next step before storing this one
    uint4 cur[kUnroll], nxt[kUnroll];
    auto load = [&](int r0, uint4 (&v)[kUnroll]) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * (kMoveThreads / p.part) + tid / p.part;
        if (r < rows && col < width && s_src[r] >= 0) v[u] = pool[s_src[r] + col];
      }
    };
    load(0, cur);
    for (int r0 = 0; r0 < rows; r0 += step_rows) {
      load(r0 + step_rows, nxt);
      if (IN_PLACE) __syncthreads();  // this step's rows are read by every thread
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * (kMoveThreads / p.part) + tid / p.part;
        if (r < rows && col < width && s_src[r] >= 0) pool[s_dst[r] + col] = cur[u];
        cur[u] = nxt[u];
      }
    }
    // the next segment's rows lie above every row stored here, and its places
    // go into the same shared arrays
    __syncthreads();
  }
  if (bad && q == 0 && p.err_flags) atomicOr(p.err_flags, 1u);
}

cudaError_t evict_launch(EvictParams& p, int B, cudaStream_t stream) {
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
    return e;
  evict_select_kernel<<<dim3(p.Hkv, B), kSelThreads, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const bool in_place = p.dst_table == p.block_table;
  p.segments = in_place ? 1 : (p.budget + kSegment - 1) / kSegment;
  // A row's 16-byte chunks in parts of 16 (256 bytes); in place with few
  // (sequence, kv head) pairs narrower parts, down to a 32-byte sector, so
  // that there are two blocks per SM.
  p.part = 16;
  auto count = [&] {
    p.k_parts = (p.pools.ck + p.part - 1) / p.part;
    p.parts = p.k_parts + (p.pools.cv + p.part - 1) / p.part;
    return int64_t(p.parts) * p.Hkv * B;
  };
  while (count() < 2 * sms && in_place && p.part > 2) p.part /= 2;
  const dim3 grid(p.parts * p.segments, p.Hkv, B);
  if (in_place)
    evict_move_kernel<true><<<grid, kMoveThreads, 0, stream>>>(p);
  else
    evict_move_kernel<false><<<grid, kMoveThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace zl

extern "C" zl_status zl_kv_evict(const zl_kv_evict_params* a, zl_stream_t stream) {
  if (!a || a->struct_size != sizeof(zl_kv_evict_params)) return ZL_ERR_INVALID_ARG;
  zl::EvictParams p;
  std::memset(&p, 0, sizeof(p));
  const zl_status st = zl::move_pools(a, &p.pools);
  if (st != ZL_OK) return st;
  if (!a->kept || !a->weights || !zl::aligned_to(a->kept, 4) || !zl::aligned_to(a->weights, 4) ||
      !zl::aligned_to(a->weights_out, 4) || !zl::aligned_to(a->dst_block_table, 4))
    return ZL_ERR_INVALID_ARG;
  if (a->budget < 1 || a->sink < 0 || a->recent < 0 ||
      int64_t(a->sink) + a->recent > a->budget || a->weights_tokens < 1)
    return ZL_ERR_INVALID_ARG;
  if (a->dst_block_table && a->dst_block_table_stride < 1) return ZL_ERR_INVALID_ARG;
  // rows of different sequences and heads must not overlap
  if ((a->B > 1 && a->weights_seq_stride < a->weights_tokens) ||
      (a->Hkv > 1 && a->weights_head_stride < a->weights_tokens))
    return ZL_ERR_INVALID_ARG;
  const int64_t out_tokens = a->budget < a->weights_tokens ? a->budget : a->weights_tokens;
  if (a->weights_out && ((a->B > 1 && a->weights_out_seq_stride < out_tokens) ||
                         (a->Hkv > 1 && a->weights_out_head_stride < out_tokens)))
    return ZL_ERR_INVALID_ARG;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.dst_table = a->dst_block_table ? a->dst_block_table : a->block_table;
  p.dst_stride = a->dst_block_table ? a->dst_block_table_stride : a->block_table_stride;
  p.seq_lens = a->seq_lens;
  p.new_lens = a->new_lens;
  p.kept = a->kept;
  p.weights = a->weights;
  p.w_seq = a->weights_seq_stride;
  p.w_head = a->weights_head_stride;
  p.weights_out = a->weights_out ? a->weights_out : a->weights;
  p.wo_seq = a->weights_out ? a->weights_out_seq_stride : a->weights_seq_stride;
  p.wo_head = a->weights_out ? a->weights_out_head_stride : a->weights_head_stride;
  p.err_flags = a->err_flags;
  p.w_tokens = a->weights_tokens;
  p.Hkv = a->Hkv;
  p.budget = a->budget;
  p.sink = a->sink;
  p.recent = a->recent;
  const cudaError_t e = zl::evict_launch(p, a->B, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
