// Eviction by accumulated weights (zl_kv_evict in the header), in two launches.
//
// select: one cluster of CTAs per (sequence, kv head) finds the K-th largest
// weight of the tokens between the sinks and the recent ones by a radix select
// on 32-bit keys that order as the floats do (a histogram of the keys' next
// digit in each CTA's shared memory, summed over the cluster), then lists the
// kept positions in order: a token is kept if its key is above the threshold,
// or equals it and fewer than the missing number of equal ones came before it.
// Each CTA owns a contiguous part of the row, each thread 16 tokens of it in a
// row (32 in long rows): its counts and a scan over threads and CTAs give the
// place of every kept token, so no atomic decides an order and the result is
// always the same. A CTA keeps its part of the weights in shared memory; they
// are read from memory once. What bounds it is the chain of passes and their
// barriers and the instructions per token, not the 4 bytes. The instance goes by the length of
// the weights rows, which is all the host knows: rows far longer than the
// sequences cost passes over nothing (64 x 8 rows of 2049-4096 tokens to 2048,
// both launches: 200 us in rows of 4096, 249 of 32768, 464 of 131072, and 607
// just above, where no cluster holds a row). With one CTA per row, ballots per
// token and the weights read again in every pass it took 209 us for 64 rows of
// 32k-131k tokens and 31 us for 512 rows of 2k-4k.
//
// move: rows are 16-byte chunks. In place, kept[j] >= j, so the rows of one
// (sequence, kv head, column part) may move in ascending chunks: a chunk's
// sources lie at or above its first destination, and nothing later reads what
// an earlier chunk overwrote, but a chunk has to be read in full before it is
// written, and before any later chunk is. One block walks one column part, or
// with few of them a cluster of up to 8 (7 sequences of 25k-55k tokens, 2 kv
// heads: 200 us with one block, 114 so); the next chunk's loads are in flight
// while this one is stored. Into other pages there is no such order and the rows
// are cut into segments as well.
#include "kv_move.cuh"
#include "kernels.h"
#include "ptx.cuh"

#include <cstddef>
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
  // 0: the weights behind the new length stay as they are; else they become 0,
  // in place up to the old length, in weights_out up to this many
  int w_clear;
  int cluster;    // CTAs per row of the select launch
  // move launch: column parts of K (then of V) of `part` chunks, segments of
  // kSegment rows (out of place; 1 in place), CTAs that share a part (in place)
  int part, k_parts, parts, segments, move_cluster;
};

__device__ __forceinline__ bool evict_len_ok(const EvictParams& p, int L) {
  const int64_t reach = p.bt_stride * p.pools.page_size;
  const int64_t dst_reach = p.dst_stride * p.pools.page_size;
  return L >= 0 && int64_t(L) <= reach && L <= p.w_tokens && int64_t(min(L, p.budget)) <= dst_reach;
}

// ------------------------------------------------------------------- select
constexpr int kSelCluster = 8;    // CTAs per row at most (the portable cluster size)

// A key that orders as the weights do: larger weight, larger key; -0 as +0,
// NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  const uint32_t k = u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
  return isnan(w) ? 0u : k;
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kBins = 256;        // of a digit: 4 digits of 8 bits
constexpr int kHistBytes = kBins * 32 * 4;

// T threads of kRun consecutive tokens each, kBlocks blocks per SM.
// Every lane counts in a histogram of its own: the weights' leading digits fall
// into a few bins, and additions to one address, by lanes of a warp or by
// warps, are done one after the other. CACHED: this CTA's part fits kRun tokens
// per thread; then a thread holds their keys in registers through all passes
// (computing them again in each pass was 390 instructions per token in all), and
// shared memory the weights. Otherwise they are read again.
template <int T, int kRun, int kBlocks, bool CACHED>
__global__ void __launch_bounds__(T, kBlocks)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kWarps = T / 32;
  static_assert(T >= kBins, "a thread for every bin");
  extern __shared__ uint32_t lane_hist[];  // [kBins][32]
  // token i of this CTA's part at i + i / kRun (no bank conflicts)
  float* cache = reinterpret_cast<float*>(lane_hist + kBins * 32);
  __shared__ uint32_t hist[2][kBins];
  __shared__ uint32_t warp_sum[kWarps], cta_gt, cta_eq;
  __shared__ uint32_t s_prefix, s_need;
  griddep_wait();
  const int CS = p.cluster, rank = int(cluster_ctarank());
  const int h = int(blockIdx.x) / CS, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = p.seq_lens[b];
  int32_t* kept = p.kept + (int64_t(b) * p.Hkv + h) * p.budget;
  const float* w = p.weights + int64_t(b) * p.w_seq + int64_t(h) * p.w_head;
  float* wo = p.weights_out + int64_t(b) * p.wo_seq + int64_t(h) * p.wo_head;
  // (the whole cluster takes the same way out)
  if (!evict_len_ok(p, L)) {
    if (h == 0 && rank == 0 && tid == 0 && p.err_flags) atomicOr(p.err_flags, 2u);
    for (int j = rank * T + tid; j < p.budget; j += CS * T) kept[j] = -1;
    return;
  }
  if (L <= p.budget) {
    for (int j = rank * T + tid; j < p.budget; j += CS * T) kept[j] = j < L ? j : -1;
    if (wo != w)
      for (int j = rank * T + tid; j < max(L, p.w_clear); j += CS * T) wo[j] = j < L ? w[j] : 0.f;
    return;
  }
  const int M = L - p.sink - p.recent;                 // candidates
  const int K = p.budget - p.sink - p.recent;          // kept of them: K < M
  const int part = ((M + CS - 1) / CS + kRun - 1) / kRun * kRun;
  const int lo = min(M, rank * part), n = min(M, lo + part) - lo;  // this CTA's
  const float* c = w + p.sink + lo;
  auto sync = [&] {
    if (CS > 1) cluster_sync();
    else __syncthreads();
  };
  for (int j = rank * T + tid; j < p.sink; j += CS * T) kept[j] = j;
  for (int j = rank * T + tid; j < p.recent; j += CS * T)
    kept[p.budget - p.recent + j] = L - p.recent + j;
  // Keys of tokens [i0, i0 + kRun) of this CTA's part, of which m are there.
  uint32_t key[kRun];
  int m = 0;
  auto load_run = [&](int i0) {
    m = min(max(n - i0, 0), kRun);
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const float x = e >= m ? 0.f : CACHED ? cache[i0 + i0 / kRun + e] : c[i0 + e];
      key[e] = weight_key(x);
    }
  };
  if (CACHED) {
    for (int i0 = tid; i0 < n; i0 += T * 16) {  // sixteen loads in flight
      float x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (i0 + u * T < n) x[u] = c[i0 + u * T];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int i = i0 + u * T;
        if (i < n) cache[i + i / kRun] = x[u];
      }
    }
    __syncthreads();
    load_run(tid * kRun);
  }
  // Runs `f(i0)` with the keys of each of this thread's runs in place (a run
  // that is not there has m = 0).
  auto for_runs = [&](auto&& f) {
    if (CACHED) {
      f(tid * kRun);
    } else {
#pragma unroll 1
      for (int base = 0; base < n; base += T * kRun) {
        load_run(base + tid * kRun);
        f(base + tid * kRun);
      }
    }
  };
  uint32_t prefix = 0, need = uint32_t(K);
  if (K > 0) {
    // the K-th largest key, most significant digits first: `prefix` holds the
    // digits found, `need` how many of the keys that share them are kept
    const int bin = tid;  // of this thread, if below kBins
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < kBins * 32; i += T) lane_hist[i] = 0;
      __syncthreads();
      // (in the first pass every key matches: nothing is found yet)
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      const uint32_t want = shift == 24 ? 0u : prefix << (shift + 8);
      for_runs([&](int) {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
          if (e < m && (key[e] & mask) == want)
            atomicAdd(&lane_hist[((key[e] >> shift) & 255u) * 32 + lane], 1u);
      });
      __syncthreads();
      // (two buffers: the cluster's barrier in the next pass comes between this
      // pass's reads and the next writes of the same one)
      uint32_t* sums = hist[(shift >> 3) & 1];
      uint32_t mine = 0;
      if (bin < kBins) {
#pragma unroll 8
        for (int k = 0; k < 32; ++k) mine += lane_hist[bin * 32 + ((k + lane) & 31)];
        sums[bin] = mine;
      }
      if (CS > 1) {  // over the cluster
        cluster_sync();
        if (bin < kBins) {
          const uint32_t addr = smem_u32(&sums[bin]);
          uint32_t x[kSelCluster];  // all in flight before the first is added
#pragma unroll
          for (int r = 0; r < kSelCluster; ++r)
            x[r] = r < CS ? ld_cluster(mapa_shared(addr, r)) : 0u;
          mine = 0;
#pragma unroll
          for (int r = 0; r < kSelCluster; ++r) mine += x[r];
        }
      }
      // the digit: the largest one with at least `need` keys at or above it
      uint32_t suf = mine;  // over lanes >= this one
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_down_sync(0xffffffffu, suf, off);
        if (lane + off < 32) suf += x;
      }
      if (lane == 0) warp_sum[warp] = suf;
      __syncthreads();
      // keys in the bins above this thread's
      const uint32_t above =
          suf - mine +
          __reduce_add_sync(0xffffffffu,
                            lane < kBins / 32 && lane > warp ? warp_sum[lane] : 0u);
      if (bin < kBins && above < need && need <= above + mine) {
        s_prefix = (prefix << 8) | uint32_t(bin);
        s_need = need - above;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // `prefix` is the threshold key: every key above it is kept, and the first
  // `need` of those that equal it
  const uint32_t thr = prefix;
  uint32_t gt_before = 0, eq_before = 0;
  // Counts of the current run: above the threshold in the low half (a round of
  // the block has at most 2^14 tokens), equal to it in the high half.
  auto run_counts = [&]() -> uint32_t {
    uint32_t x = 0;
#pragma unroll
    for (int e = 0; e < kRun; ++e)
      x += e >= m ? 0u : key[e] > thr ? 1u : key[e] == thr ? 0x10000u : 0u;
    return x;
  };
  if (K > 0 && CS > 1) {  // how many this CTA has, for the CTAs after it
    if (tid == 0) cta_gt = cta_eq = 0;
    __syncthreads();
    for_runs([&](int) {
      const uint32_t x = __reduce_add_sync(0xffffffffu, run_counts());
      if (lane == 0) {
        atomicAdd(&cta_gt, x & 0xffffu);
        atomicAdd(&cta_eq, x >> 16);
      }
    });
  }
  // Also: every CTA holds its part of the weights, so that moving them in place
  // overwrites nothing that is still to be read.
  sync();
  if (K > 0) {
    if (CS > 1) {
      uint32_t g = 0, e = 0;
      if (lane < rank) {
        g = ld_cluster(mapa_shared(smem_u32(&cta_gt), lane));
        e = ld_cluster(mapa_shared(smem_u32(&cta_eq), lane));
      }
      gt_before = __reduce_add_sync(0xffffffffu, g);
      eq_before = __reduce_add_sync(0xffffffffu, e);
    }
    for_runs([&](int i0) {
      const uint32_t mine = run_counts();
      uint32_t pre = mine;  // over lanes <= this one
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, pre, off);
        if (lane >= off) pre += y;
      }
      if (lane == 31) warp_sum[warp] = pre;
      __syncthreads();
      const uint32_t ws = lane < kWarps ? warp_sum[lane] : 0u;
      pre += __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0u) - mine;  // before this run
      uint32_t gt = gt_before + (pre & 0xffffu), eq = eq_before + (pre >> 16);
      if (mine) {
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
          const bool g = e < m && key[e] > thr, q = e < m && key[e] == thr;
          if (g || (q && eq < need)) {
            const uint32_t at = p.sink + gt + min(eq, need);
            kept[at] = p.sink + lo + i0 + e;
            if (CACHED) wo[at] = cache[i0 + i0 / kRun + e];
          }
          gt += g ? 1u : 0u;
          eq += q ? 1u : 0u;
        }
      }
      if (!CACHED) {
        const uint32_t round = __reduce_add_sync(0xffffffffu, ws);
        gt_before += round & 0xffffu;
        eq_before += round >> 16;
        __syncthreads();  // warp_sum is read
      }
    });
  }
  // The other weights: the sinks stay or are copied; the recent ones move down
  // in ascending chunks, each read before it is written (their places lie
  // below every recent one that is still to be read). Where the parts do not
  // fit the caches, one CTA moves the whole row that way, by the list.
  sync();  // also: no CTA leaves while another reads its counts
  // Weights behind the new length, if they are to become 0. In place the last
  // CTA still reads from [keep_from, L): those it clears itself, at the end.
  const int keep_from = max(p.budget, wo != w ? p.w_clear : CACHED ? L - p.recent : p.budget);
  if (p.w_clear)
    for (int j = p.budget + rank * T + tid; j < keep_from; j += CS * T) wo[j] = 0.f;
  if (rank != CS - 1) return;
  if (CACHED && wo != w)
    for (int j = tid; j < p.sink; j += T) wo[j] = w[j];
  for (int j0 = CACHED ? p.budget - p.recent : 0; j0 < p.budget; j0 += T) {
    const int j = j0 + tid;
    float x = 0.f;
    if (j < p.budget) x = w[CACHED ? L - p.budget + j : __ldcg(kept + j)];
    __syncthreads();
    if (j < p.budget) wo[j] = x;
  }
  if (p.w_clear && wo == w)  // (every thread is past its reads of [keep_from, L))
    for (int j = keep_from + tid; j < L; j += T) wo[j] = 0.f;
}

template <int T, int kRun, int kBlocks, bool CACHED>
cudaError_t select_launch(const EvictParams& p, int part, int B, cudaStream_t stream) {
  constexpr size_t kMost = kHistBytes + (CACHED ? size_t(T) * (kRun + 1) * sizeof(float) : 0);
  static bool done[64] = {};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!done[device]) {
    if ((e = cudaFuncSetAttribute(evict_select_kernel<T, kRun, kBlocks, CACHED>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost))) !=
        cudaSuccess)
      return e;
    done[device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.Hkv * p.cluster), unsigned(B));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes =
      kHistBytes + (CACHED ? size_t((part + kRun - 1) / kRun) * (kRun + 1) * sizeof(float) : 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(p.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<T, kRun, kBlocks, CACHED>, p);
}

// CTAs per row: as many as hold the row, and more while the rows alone leave SMs
// idle and each CTA still has work for its threads. Small blocks for short rows
// (their barriers cost less); longer runs and two blocks per SM for long ones:
// a row takes about 23 us of passes and barriers whatever its length, so what
// counts is how many are under way (64 rows of 32k-131k tokens: 91 us with 1024
// threads of 16 tokens, one block per SM).
cudaError_t select_rows(EvictParams& p, int B, int sms, cudaStream_t stream) {
  constexpr int kSmall = 256 * 16, kLarge = 512 * 32;  // tokens a CTA holds
  p.cluster = 1;
  while (p.cluster < kSelCluster &&
         (p.w_tokens > p.cluster * kLarge ||
          (int64_t(B) * p.Hkv * p.cluster < sms && p.w_tokens > p.cluster * kSmall)))
    p.cluster *= 2;
  const int part = (p.w_tokens + p.cluster - 1) / p.cluster;
  if (part <= kSmall) return select_launch<256, 16, 4, true>(p, part, B, stream);
  if (part <= kLarge) return select_launch<512, 32, 2, true>(p, part, B, stream);
  return select_launch<512, 32, 2, false>(p, part, B, stream);
}

// --------------------------------------------------------------------- move
constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;       // chunks of 16 bytes per thread and step
constexpr int kSegment = 1024;   // rows whose places are looked up together
// Longest budget and weights rows: a pass of the move looks up kSegment rows for
// each CTA of a cluster, and a pass of the selection's loops is a token per
// thread of one, so numbers up to one pass beyond either stay in 32 bits.
constexpr int kMaxTokens = INT32_MAX - 16384;
static_assert(kSelCluster * kSegment <= 16384 && kSelCluster * 512 <= 16384, "one pass");

// Column part q of a row: chunks [c0, c0 + part) of K or V. In place the row's
// cluster of move_cluster CTAs takes the kept rows in steps, each CTA its share of
// a step; the step after is loaded before the barrier that lets this one be
// stored.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, 4)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int64_t s_src[kSegment], s_dst[kSegment];  // row starts in chunks; -1: no move
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int CS = IN_PLACE ? p.move_cluster : 1, rank = IN_PLACE ? int(blockIdx.x) % CS : 0;
  const int seg = IN_PLACE ? 0 : int(blockIdx.x) / p.parts;
  const int q = IN_PLACE ? int(blockIdx.x) / CS : int(blockIdx.x) % p.parts;
  const bool is_v = q >= p.k_parts;
  const int width = is_v ? p.pools.cv : p.pools.ck;
  const int col = (is_v ? q - p.k_parts : q) * p.part + tid % p.part;
  uint4* pool = is_v ? p.pools.v : p.pools.k;
  const int32_t* kept = p.kept + (int64_t(b) * p.Hkv + h) * p.budget;
  const int L = p.seq_lens[b];
  const bool ok = evict_len_ok(p, L);
  if (blockIdx.x == 0 && h == 0 && tid == 0) p.new_lens[b] = ok ? min(L, p.budget) : L;
  // (the whole cluster takes the same way out)
  if (!ok || (IN_PLACE && L <= p.budget)) return;
  const int step_rows = kMoveThreads / p.part * kUnroll;  // rows of a CTA in one step
  const int32_t* sbt = p.block_table + int64_t(b) * p.bt_stride;
  const int32_t* dbt = p.dst_table + int64_t(b) * p.dst_stride;
  bool bad = false;
  const int first = seg * kSegment;
  const int last = IN_PLACE ? p.budget : min(min(p.budget, L), first + kSegment);
  for (int base = first; base < last; base += CS * kSegment) {
    // the CTA's row r of this pass is row `at(r)` of the kept ones
    auto at = [&](int r) { return base + (r / step_rows * CS + rank) * step_rows + r % step_rows; };
    for (int r = tid; r < kSegment; r += kMoveThreads) {
      const int j = at(r);
      int64_t src = -1, dst = -1;
      if (j < last) {
        const int t = kept[j];
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
    __syncthreads();
    // steps of step_rows rows: load the next step before storing this one
    uint4 cur[kUnroll], nxt[kUnroll];
    auto load = [&](int r0, uint4 (&v)[kUnroll]) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * (kMoveThreads / p.part) + tid / p.part;
        if (r < kSegment && col < width && s_src[r] >= 0) v[u] = pool[s_src[r] + col];
      }
    };
    const int steps = min(kSegment / step_rows,
                          (last - base + CS * step_rows - 1) / (CS * step_rows));
    load(0, cur);
    for (int i = 0; i < steps; ++i) {
      const int r0 = i * step_rows;
      load(r0 + step_rows, nxt);
      if (IN_PLACE) {  // this step's rows are read by every thread
        if (CS > 1) cluster_sync();
        else __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * (kMoveThreads / p.part) + tid / p.part;
        if (col < width && s_src[r] >= 0) pool[s_dst[r] + col] = cur[u];
        cur[u] = nxt[u];
      }
    }
    // the next pass's rows lie above every row stored here, and its places go
    // into the same shared arrays
    __syncthreads();
  }
  if (bad && q == 0 && p.err_flags) atomicOr(p.err_flags, 1u);
}

template <bool IN_PLACE>
cudaError_t move_launch(const EvictParams& p, int B, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.parts * p.segments * p.move_cluster), unsigned(p.Hkv), unsigned(B));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(p.move_cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.move_cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<IN_PLACE>, p);
}

cudaError_t evict_launch(EvictParams& p, int B, cudaStream_t stream) {
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
    return e;
  e = select_rows(p, B, sms, stream);
  if (e != cudaSuccess) return e;
  const bool in_place = p.dst_table == p.block_table;
  p.segments = in_place ? 1 : (p.budget + kSegment - 1) / kSegment;
  // A row's 16-byte chunks in parts of 16 (256 bytes); in place with few
  // (sequence, kv head) pairs clusters of CTAs, then narrower parts, down to a
  // 32-byte sector, so that there are two blocks per SM.
  p.part = 16;
  p.move_cluster = 1;
  auto count = [&] {
    p.k_parts = (p.pools.ck + p.part - 1) / p.part;
    p.parts = p.k_parts + (p.pools.cv + p.part - 1) / p.part;
    return int64_t(p.parts) * p.Hkv * B * p.move_cluster;
  };
  // (a cluster's step is at least 64 rows a CTA: with fewer rows kept its CTAs idle)
  while (count() < 2 * sms && in_place && p.move_cluster < 8 && p.budget > 64 * p.move_cluster)
    p.move_cluster *= 2;
  while (count() < 2 * sms && in_place && p.part > 2) p.part /= 2;
  return in_place ? move_launch<true>(p, B, stream) : move_launch<false>(p, B, stream);
}

}  // namespace
}  // namespace zl

extern "C" zl_status zl_kv_evict(const zl_kv_evict_params* params, zl_stream_t stream) {
  zl_kv_evict_params given;
  if (!zl::take_params(params, offsetof(zl_kv_evict_params, weights_clear), &given))
    return ZL_ERR_INVALID_ARG;
  const zl_kv_evict_params* a = &given;
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
  if (zl::overlaps(a->new_lens, a->B, a->kept, int64_t(a->B) * a->Hkv * a->budget))
    return ZL_ERR_INVALID_ARG;
  if (!zl::rows_distinct(a->B, a->Hkv, a->weights_seq_stride, a->weights_head_stride,
                         a->weights_tokens))
    return ZL_ERR_INVALID_ARG;
  int64_t out_tokens = a->budget < a->weights_tokens ? a->budget : a->weights_tokens;
  if (a->weights_clear < 0 || (a->weights_out && a->weights_clear && a->weights_clear < out_tokens))
    return ZL_ERR_INVALID_ARG;
  if (a->weights_clear > out_tokens) out_tokens = a->weights_clear;
  if (a->weights_out && !zl::rows_distinct(a->B, a->Hkv, a->weights_out_seq_stride,
                                           a->weights_out_head_stride, out_tokens))
    return ZL_ERR_INVALID_ARG;
  if (a->budget > zl::kMaxTokens || a->weights_tokens > zl::kMaxTokens ||
      a->weights_clear > zl::kMaxTokens)
    return ZL_ERR_UNSUPPORTED;
  // (in place is NULL: the kernels that write elsewhere read without its order)
  if (a->weights_out == a->weights || a->dst_block_table == a->block_table)
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
  p.w_clear = a->weights_clear;
  const cudaError_t e = zl::evict_launch(p, a->B, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
