// GQA decode with modified scores for many query rows per kv head (a large
// drafted tree, or many heads), on tcgen05.
//
// With R = g q_len rows, the m16 tiles of gqa_kernel.cuh read every K/V tile R
// / 16 times from shared memory and L2. Here up to 256 rows share each K/V
// tile: S = Q K^T (M = 128 rows, N = 128 tokens) and O += P V (N = 128
// columns) are tcgen05.mma with S, P and O in TMEM, so a tile of 128 tokens
// (64 KB) is loaded once for all of them. Per SM and tile the load takes about
// 2800 cycles at this card's bandwidth, the products of 128 rows 1050, of 256
// rows 2100.
// Measured, 64 sequences of 512-4096 tokens with 32 heads on 8 kv heads: 16
// drafted tokens (MT = 1) 122 us, 5.2 TB/s, bound by the load and the ends of
// units; 64 (MT = 2) 167 us, 4.1 TB/s and 0.95 PFLOP/s, with a cap 212 us, bound
// by each stream's chain: 2150 cycles of softmax for 128 rows x 128 tokens, then
// 1360 from its P to the next S (PV of a half tile 256, QK 512, the rest waits
// and issue). A tile with masks takes 5000-6500.
//
// Two softmax warpgroups keep the tensor pipe fed, each with its own S and O
// ("streams"). MT = 2: stream s has rows [128 s, 128 s + 128) of the block and
// takes every tile. MT = 1 (at most 128 rows): both streams have the same rows
// and take the tiles in turn, and the epilogue joins their two results. Either
// way one stream's softmax runs under the other one's products.
//
// Work is cut as in gqa_kernel.cuh: units (sequence, kv head, row block) of
// 128-token tiles on one line, cut into equal ranges, one per CTA; cut units
// leave normalised fp32 partials for the merge kernel.
//
// TMEM (512 columns): S of stream 0, 1 (128 each; P, 64 columns of bf16 pairs,
// replaces S once it is read, in halves of 64 tokens, so that a half's PV runs
// under the other half's softmax), O of stream 0, 1 (128 each). MMAs of one CTA
// execute in the order of their issue, so QK of a stream's next tile may
// follow the PV that reads its P without a wait; the commit after a QK covers
// the PV before it, so a softmax thread that sees S of a tile may also rescale
// O.
#include "gqa_kernel.cuh"
#include "gqa_wide.h"

#include <type_traits>

namespace zl {

namespace {

constexpr int kWT = kWideTile;                 // tokens per tile
constexpr int kHalf = kWT * 128;               // 16 KB: 128 rows x 64 columns
constexpr int kBuf = 2 * kHalf;                // one K or V tile, or 128 rows of Q
constexpr int kInfo = 8;                       // tiles whose load info is kept
constexpr int kSoft = 256;                     // softmax threads
constexpr int kWideThreads = kSoft + 256;      // + K, MMA, V, Q warps and the epilogue's four
constexpr int kStage = 32 * 64;                // bytes of an epilogue warp's staging rows
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;   // + 128 * stream (S: + 64 * half tile)
constexpr int kHT = kWT / 2;                   // tokens of a half tile
constexpr int kDepthBias = kHT;                // of a position in a byte: none is below -kHT
constexpr int kFewParts = 4;                   // CTAs per unit above which the merge is FEW

template <int MT>
struct WideCfg {
  static constexpr int kRing = MT == 2 ? 4 : 5;      // K/V buffers
  static constexpr int kOffRing = MT * kBuf;
  static constexpr int kOffBar = kOffRing + kRing * kBuf;
  // (MASK, ML and EPI of piece i are barriers i & 1: the same barrier's next
  // phase then waits for those that wait for this one)
  enum : int {
    B_Q = 0, B_QFREE, B_FINAL, B_MASK0, B_ML0 = B_MASK0 + 2, B_EPI0 = B_ML0 + 2,
    B_S0 = B_EPI0 + 2, B_P0 = B_S0 + 2, B_PV0 = B_P0 + 4, B_O0 = B_PV0 + 2,
    B_OFREE0 = B_O0 + 2, B_FULL0 = B_OFREE0 + 2, B_EMPTY0 = B_FULL0 + kRing,
    B_INFO0 = B_EMPTY0 + kRing, B_COUNT = B_INFO0 + kInfo
  };
  static constexpr int kOffMisc = kOffBar + 8 * B_COUNT;   // TMEM address, abort flag
  static constexpr int kOffInfo = kOffMisc + 16;           // kInfo words
  static constexpr int kOffMl = kOffInfo + 4 * kInfo;          // [2][2][128] (m, l)
  static constexpr int kOffMask = kOffMl + 2 * 2 * 128 * 8;    // [2][512] words
  static constexpr int kOffDepth = kOffMask + 2 * 512 * 4;     // [2][256] bytes
  static constexpr int kOffStage = (kOffDepth + 2 * 256 + 127) / 128 * 128;  // [4] epilogue rows
  static constexpr int kOffPrefix = kOffStage + 4 * kStage;
  // Ring place of K and V of tile t (of n in its piece, tile_no tiles before it
  // in the CTA): the order in which the MMA warp uses them.
  static __device__ __forceinline__ uint32_t k_item(uint32_t tile_no, int t) {
    return 2 * tile_no + uint32_t(MT == 2 ? 2 * t : t == 0 ? 0 : 2 * t - 1);
  }
  static __device__ __forceinline__ uint32_t v_item(uint32_t tile_no, int t, int n) {
    return 2 * tile_no + uint32_t(MT == 2 ? 2 * t + 1 : min(2 * t + 2, 2 * n - 1));
  }
  static constexpr size_t smem_bytes(int B) { return 1024 + kOffPrefix + size_t(B + 1) * 4; }
  static constexpr size_t kSmemMax = smem_bytes(kMaxBatch);
  static_assert(kSmemMax <= 232448, "shared memory of one CTA");
};

// Wait on an mbarrier by polling, one thread; false after a timeout or an abort.
__device__ __forceinline__ bool wide_poll(uint32_t bar, uint32_t parity,
                                          const volatile int* abort_flag) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_test(bar, parity)) return true;
    if ((i & 63u) == 0 && (*abort_flag || globaltimer_ns() - t0 > kWaitTimeoutNs)) return false;
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Bits [a, b) of a 32-bit word, both clamped to 0..32.
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// Drafted bits [j0, j0 + 32) of a row's ancestor mask (words 32-bit words).
__device__ __forceinline__ uint32_t mask_word(const uint32_t* bits, int words, int j0) {
  if (j0 <= -32 || j0 >= 32 * words) return 0u;
  if (j0 < 0) return bits[0] << (-j0);
  const int w = j0 >> 5, sh = j0 & 31;
  uint32_t x = bits[w] >> sh;
  if (sh && w + 1 < words) x |= bits[w + 1] << (32 - sh);
  return x;
}

// Registers that tcgen05.ld fills are valid after tcgen05.wait::ld: nothing
// computed from them may be scheduled above it.
template <int N>
__device__ __forceinline__ void hold(uint32_t (&r)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(r[k]));
}

// The 64 scores of a half tile, two to a register pair.
__device__ __forceinline__ void load_scores(uint32_t taddr, uint64_t (&x)[kHT / 2]) {
  uint32_t v[2][32];
  tmem_ld32(taddr, v[0]);
  tmem_ld32(taddr + 32, v[1]);
  tmem_wait_ld();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    hold(v[h]);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      x[16 * h + k] =
          pack_f32x2(__uint_as_float(v[h][2 * k]), __uint_as_float(v[h][2 * k + 1]));
  }
}

// tanh(y) / y of two z = y^2 in [0, 1] (the polynomial of cap_tanh).
__device__ __forceinline__ uint64_t tanh_ratio(uint64_t z) {
  uint64_t t = fma_f32x2(z, pack_f32x2(kTanh6, kTanh6), pack_f32x2(kTanh5, kTanh5));
  t = fma_f32x2(t, z, pack_f32x2(kTanh4, kTanh4));
  t = fma_f32x2(t, z, pack_f32x2(kTanh3, kTanh3));
  t = fma_f32x2(t, z, pack_f32x2(kTanh2, kTanh2));
  t = fma_f32x2(t, z, pack_f32x2(kTanh1, kTanh1));
  return fma_f32x2(t, z, pack_f32x2(kTanh0, kTanh0));
}

// The 64 scores of a half tile, dot products v in TMEM, become out tanh(in v); near:
// this row's are all within |in v| <= 1. (Few of them at a time, in a loop: the
// tile loop has neither the registers nor the instruction cache for more.)
__device__ __forceinline__ void cap_scores(uint32_t taddr, float in, float out, bool near) {
  near = __all_sync(0xffffffffu, near);
  const uint64_t in2 = pack_f32x2(in, in), out2 = pack_f32x2(out, out);
#pragma unroll 1
  for (int c = 0; c < kHT; c += 16) {
    uint32_t v[16];
    tmem_ld16(taddr + c, v);
    tmem_wait_ld();
    hold(v);
    uint64_t y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      y[k] = mul_f32x2(pack_f32x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), in2);
    if (near) {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = mul_f32x2(tanh_ratio(mul_f32x2(y[k], y[k])), y[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t z = mul_f32x2(y[k], y[k]);
        const float2 f = unpack_f32x2(z), g = unpack_f32x2(y[k]);
        const float2 t = unpack_f32x2(mul_f32x2(tanh_ratio(z), y[k]));
        y[k] = pack_f32x2(f.x <= 1.f ? t.x : tanh_far(g.x), f.y <= 1.f ? t.y : tanh_far(g.y));
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 t = unpack_f32x2(mul_f32x2(y[k], out2));
      v[2 * k] = __float_as_uint(t.x);
      v[2 * k + 1] = __float_as_uint(t.y);
    }
    tmem_st16(taddr + c, v);
  }
  tmem_wait_st();
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 32) tmem_ld32(taddr, r);
  else tmem_ld16(taddr, r);
}

// One contiguous run of tiles of one unit, as every role walks them: from the
// newest, `last`, to the oldest. (A distance bias makes the newest scores the
// largest; oldest first, the running maximum rose and O was rescaled at nearly
// every tile: 64 drafted tokens, 64 sequences 293 us against 243.)
struct Piece {
  int b, kvh, blk, L, ntiles, last;
  bool partial;
  int slot;
  int next;
};

__device__ __forceinline__ int wide_first_tile(const WideParams& p, int L) {
  return p.window ? max(L - p.q_total - p.window + 1, 0) / kWT : 0;
}
// Places of a unit on the work line (0 for a sequence without tiles).
__device__ __forceinline__ int unit_places(const WideParams& p, int L) {
  if (!(L > 0 && int64_t(L) <= p.len_cap)) return 0;
  return (L + kWT - 1) / kWT - wide_first_tile(p, L) + kWideUnitCost;
}

// Work line: unit u of sequence b (u = kv head * nblk + row block) takes
// kWideUnitCost places for its start and end (Q, the first scores, the masked
// tiles, the epilogue), then one per tile, so that equal ranges take equal time.
// `idx` lies in a unit; the piece from it to e_c or the unit's end, whichever
// is first, has the tiles whose places it covers, and the first tiles' if it
// ends among them. (Places fit 32 bits: the host takes this kernel only when
// they do.)
__device__ __forceinline__ Piece piece_at(const WideParams& p, const int* prefix, int idx, int s_c,
                                          int e_c) {
  Piece q;
  const int U = p.Hkv * p.nblk;
  q.b = locate_seq(prefix, p.B, U, idx);
  const int first = prefix[q.b], len = prefix[q.b + 1] - first;
  const int off = idx - U * first, u = off / len;
  q.kvh = u / p.nblk;
  q.blk = u - q.kvh * p.nblk;
  const int unit0 = U * first + u * len;
  q.next = min(e_c, unit0 + len);
  const int t0 = max(idx - unit0 - kWideUnitCost, 0);
  q.ntiles = max(q.next - unit0 - kWideUnitCost, 0) - t0;
  q.partial = q.ntiles < len - kWideUnitCost;
  q.slot = idx == s_c ? 0 : 1;
  q.L = p.seq_lens[q.b];
  q.last = wide_first_tile(p, q.L) + t0 + q.ntiles - 1;
  return q;
}

// CAP: the scores are capped (instances of their own: the uncapped tile loop
// then has no registers to spare for the polynomial's constants).
template <int MT, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kWideThreads, 1)
gqa_wide_kernel(const __grid_constant__ WideParams p) {
  using Cfg = WideCfg<MT>;
  constexpr int NB = Cfg::kRing;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  auto bar = [&](int i) -> uint32_t { return sbase + Cfg::kOffBar + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 8);
  uint32_t* info = reinterpret_cast<uint32_t*>(smem + Cfg::kOffInfo);
  float2* ml = reinterpret_cast<float2*>(smem + Cfg::kOffMl);
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMask);
  uint8_t* depth_s = smem + Cfg::kOffDepth;
  int* prefix = reinterpret_cast<int*>(smem + Cfg::kOffPrefix);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.B;

  if (tid == 0) {
    mbar_init(bar(Cfg::B_Q), 1);
    mbar_init(bar(Cfg::B_QFREE), 1);
    mbar_init(bar(Cfg::B_FINAL), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Cfg::B_MASK0 + s), 32);
      mbar_init(bar(Cfg::B_ML0 + s), kSoft);
      mbar_init(bar(Cfg::B_EPI0 + s), 128);
      mbar_init(bar(Cfg::B_S0 + s), 1);
      for (int h = 0; h < 2; ++h) mbar_init(bar(Cfg::B_P0 + 2 * s + h), 128);
      mbar_init(bar(Cfg::B_PV0 + s), 1);
      mbar_init(bar(Cfg::B_O0 + s), 1);
      mbar_init(bar(Cfg::B_OFREE0 + s), 128);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(bar(Cfg::B_FULL0 + i), 1);
      mbar_init(bar(Cfg::B_EMPTY0 + i), 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(bar(Cfg::B_INFO0 + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Rows of Q past the last whole token (no copy writes them) are zeros, so that
  // their scores, which are dropped, take no slow path.
  for (int i = p.g * p.tpt * 8 + tid; i < 128 * 8; i += kWideThreads) {
#pragma unroll
    for (int k = 0; k < 2 * MT; ++k)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sbase + k * kHalf + i * 16),
                   "r"(0u)
                   : "memory");
  }
  fence_proxy_async_smem();
  // A programmatic dependent of the kernel before it on the stream: global
  // memory, and TMEM that kernel may still hold, only after it has finished.
  griddep_wait();
  if (warp == 9) {
    tmem_alloc(sbase + Cfg::kOffMisc, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
    tma_prefetch_desc(&p.tmap_q);
  }
  if (warp == 0) {  // places of a unit of each sequence, exclusive prefix sum
    const int per = (B + 31) / 32, b0 = lane * per;
    int local = 0;
    for (int i = 0; i < per; ++i) {
      if (b0 + i < B) {
        const int L = p.seq_lens[b0 + i];
        if (blockIdx.x == 0 && !(L >= 0 && int64_t(L) <= p.len_cap))
          raise_error(p.err_flags, kErrBadLen);
        local += unit_places(p, L);
      }
    }
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    int run = incl - local, longest = 0;
    for (int i = 0; i < per; ++i) {
      if (b0 + i < B) {
        const int n = unit_places(p, p.seq_lens[b0 + i]);
        prefix[b0 + i] = run;
        run += n;
        longest = max(longest, n);
      }
    }
    if (lane == 31) prefix[B] = incl;
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) info[0] = uint32_t(longest);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();  // the merge kernel waits for this whole grid
  const uint32_t tmem = *tmem_slot;
  const int c = blockIdx.x;
  const int64_t W = int64_t(p.Hkv) * p.nblk * prefix[B];
  // A piece more costs the merge about 0.4 us (two read at a time), a place 1.8
  // us: places / G * 1.8 + G / units * 0.4 is least at G = sqrt(4.5 W units).
  const int64_t units = int64_t(B) * p.Hkv * p.nblk;
  const float best = sqrtf(4.5f * float(W) * float(units));
  const TileCut cut(W, best < float(gridDim.x) ? max(int(best), 1) : int(gridDim.x));
  int s_c = c < int(cut.G) && W > 0 ? int(cut.start(c)) : 0;
  int e_c = c < int(cut.G) && W > 0 ? int(cut.start(c + 1)) : 0;
  // Few short units: one CTA each, nothing cut (a cut costs the partials' way
  // through memory and the merge's part of the call).
  const bool whole = p.whole_units == 2 ||
                     (p.whole_units == 1 && int(info[0]) <= kWideWholeTiles + kWideUnitCost);
  __syncthreads();  // info[0] is read: the K warp may use it
  if (whole && units > gridDim.x) {
    // more units than CTAs: ranges that begin and end at the nearest unit's start
    const TileCut even(W, int(gridDim.x));
    auto at_unit = [&](int64_t place) -> int {
      if (place >= W) return int(W);
      const int U = p.Hkv * p.nblk, b = locate_seq(prefix, B, U, place);
      const int len = prefix[b + 1] - prefix[b], off = int(place) - U * prefix[b];
      return U * prefix[b] + (off + len / 2) / len * len;
    };
    s_c = c < int(even.G) ? at_unit(even.start(c)) : 0;
    e_c = c < int(even.G) ? at_unit(even.start(c + 1)) : 0;
  } else if (whole) {
    s_c = e_c = 0;
    if (c < units) {
      const int U = p.Hkv * p.nblk, b = c / U, len = prefix[b + 1] - prefix[b];
      s_c = U * prefix[b] + (c - b * U) * len;
      e_c = s_c + len;
    }
  }
  if (tid == 0 && c > 0) {
    // For the merge: whether this CTA's first place is the first boundary
    // between the tiles of a unit, and if so of which one (sequence, unit),
    // the last CTA with a part of it and the slot of the first one's (c - 1).
    int4 cut_unit = make_int4(0, 0, -1, 0);
    if (e_c > s_c && !whole) {
      const int U = p.Hkv * p.nblk, b = locate_seq(prefix, B, U, s_c);
      const int first = prefix[b], len = prefix[b + 1] - first, u = (s_c - U * first) / len;
      const int unit0 = U * first + u * len, before = int(cut.start(c - 1));
      if (s_c > unit0 + kWideUnitCost && before <= unit0 + kWideUnitCost)
        cut_unit = make_int4(b, u, cut.owner(unit0 + len - 1), before >= unit0 ? 0 : 1);
    }
    p.ws_cut[c] = cut_unit;
  }

  if (warp >= 8 && warp < 12) {
    if (warp == 8 || warp == 10) {
      // --------------------------------------------------- K and V producers
      // Warp 8 loads the K, warp 10 the V of every tile into the ring places
      // of their turn. Lane i looks up the page of the tile's token block i;
      // blocks wholly past the cache end or before the oldest window, or on a
      // bad page, are not loaded. (One warp for both took 1300-1700 cycles to
      // issue the 16 copies of a tile with 16-token pages, and bounded the
      // kernel.)
      const bool is_v = warp == 10;
      const CUtensorMap* map = is_v ? &p.tmap_v : &p.tmap_k;
      const int nblocks = kWT / p.box;
      uint32_t tile_no = 0;
      bool ok = true;
      for (int idx = s_c; idx < e_c && ok;) {
        const Piece pc = piece_at(p, prefix, idx, s_c, e_c);
        if (pc.ntiles == 0) {  // only places of a unit's fixed cost
          idx = pc.next;
          continue;
        }
        const int32_t* bt = p.block_table + int64_t(pc.b) * p.bt_stride;
        const int lo = p.window ? pc.L - p.q_total - p.window + 1 : 0;
        // this lane's block of tile t: its page, -1 (nothing there), -2 (bad page)
        auto page_of = [&](int t) -> int {
          const int tok = (pc.last - t) * kWT + lane * p.box;
          if (lane >= nblocks || t >= pc.ntiles || tok >= pc.L || tok + p.box <= lo) return -1;
          const int pg = __ldg(bt + tok / p.page_size);
          return pg < 0 || pg >= p.num_pages ? -2 : pg;
        };
        int page = page_of(0);
        for (int t = 0; t < pc.ntiles && ok; ++t) {
          const int ahead = page_of(t + 1);  // in flight while this tile waits
          const uint32_t item = is_v ? Cfg::v_item(tile_no, t, pc.ntiles) : Cfg::k_item(tile_no, t);
          const uint32_t s = item % NB, ph = (item / NB) & 1;
          const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
          const uint32_t fb = bar(Cfg::B_FULL0 + s);
          const uint32_t dst = sbase + Cfg::kOffRing + s * kBuf;
          const int slot0 = (pc.last - t) * kWT % p.page_size;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(Cfg::B_EMPTY0 + s), ph ^ 1u, abort_flag));
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bytes = uint32_t(__popc(there)) * uint32_t(p.box) * 256u;
            if (bytes) mbar_arrive_expect_tx(fb, bytes);
            else mbar_arrive(fb);
          }
          __syncwarp();
          int slot = slot0;
#pragma unroll
          for (int k = 0; k < kWT / kGqaTile; ++k) {
            if (k >= nblocks) break;
            const int pg = __shfl_sync(0xffffffffu, page, k);
            if (pg >= 0 && elect_one()) {
              const uint32_t d = dst + uint32_t(k * p.box) * 128u;
              tma_load_4d(d, map, fb, 0, slot, pc.kvh, pg);
              tma_load_4d(d + kHalf, map, fb, 64, slot, pc.kvh, pg);
            }
            __syncwarp();
            slot += p.box;
            if (slot >= p.page_size) slot -= p.page_size;
          }
          if (!is_v) {
            // what the softmax threads need to know of the tile's 16-token
            // blocks: bits 0-7 on a bad page, bits 8-15 not loaded
            const int n = p.box / 16;
            const uint32_t mine = lane < nblocks ? ((1u << n) - 1u) << (lane * n) : 0u;
            const uint32_t word = __reduce_or_sync(
                0xffffffffu, (page == -2 ? mine : 0u) | (page < 0 ? mine << 8 : 0u));
            const uint32_t i = (tile_no + t) % kInfo;
            if (lane == 0) {
              info[i] = word;
              mbar_arrive(bar(Cfg::B_INFO0 + i));
            }
          }
          page = ahead;
        }
        tile_no += pc.ntiles;
        idx = pc.next;
      }
      if (!ok && lane == 0) {
        raise_error(p.err_flags, kErrTimeout);
        *abort_flag = 1;
      }
    } else if (warp == 11) {
      // ------------------------------------------------------------ Q loader
      // The piece's Q rows (two bulk copies per row tile: rows (token, head) in
      // the order of the tensor, tokens past the last one read as zeros) as
      // soon as the last QK of the piece before is done, and the tree's masks
      // and depths in a buffer of their own.
      uint32_t pieces = 0;
      bool ok = true;
      for (int idx = s_c; idx < e_c && ok;) {
        const Piece pc = piece_at(p, prefix, idx, s_c, e_c);
        if (pc.ntiles == 0) {  // only places of a unit's fixed cost
          idx = pc.next;
          continue;
        }
        if (p.tree) {
          const int words = p.q_total * p.tree_words;
          const uint32_t* src = p.tree + int64_t(pc.b) * words;
          uint32_t* dst = mask_s + (pieces & 1) * 512;
          if (pieces >= 2)  // the softmax threads are past the piece that used this buffer
            ok = __all_sync(0xffffffffu, mbar_wait(bar(Cfg::B_ML0 + (pieces & 1)),
                                                   ((pieces >> 1) - 1) & 1, abort_flag));
          if (!ok) break;
          for (int i = lane; i < words; i += 32) dst[i] = __ldg(src + i);
          __syncwarp();
          const int off = (pc.L - p.q_total) & (kHT - 1);
          for (int i = lane; i < 256; i += 32) {
            int n = 0;
            if (i < off) {
              n = i - off;
            } else if (i < off + p.q_total) {
              for (int w = 0; w < p.tree_words; ++w)
                n += __popc(dst[(i - off) * p.tree_words + w]);
              n = max(n - 1, 0);
            }
            depth_s[(pieces & 1) * 256 + i] = uint8_t(n + kDepthBias);
          }
          mbar_arrive(bar(Cfg::B_MASK0 + (pieces & 1)));
        }
        if (pieces > 0)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(bar(Cfg::B_QFREE), (pieces - 1) & 1, abort_flag));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(Cfg::B_Q), uint32_t(MT * 2 * 128 * p.g * p.tpt));
#pragma unroll
          for (int s = 0; s < MT; ++s) {
            const int tok = (pc.blk * MT + s) * p.tpt;
            tma_load_4d(sbase + s * kBuf, &p.tmap_q, bar(Cfg::B_Q), 0, pc.kvh * p.g, tok, pc.b);
            tma_load_4d(sbase + s * kBuf + kHalf, &p.tmap_q, bar(Cfg::B_Q), 64, pc.kvh * p.g,
                        tok, pc.b);
          }
        }
        __syncwarp();
        ++pieces;
        idx = pc.next;
      }
      if (!ok && lane == 0) {
        raise_error(p.err_flags, kErrTimeout);
        *abort_flag = 1;
      }
    } else {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc_qk = umma_idesc_bf16(128, kWT, false);
      const uint32_t idesc_pv = umma_idesc_bf16(128, 128, true);
      // one thread for all of it: no votes or shuffles between an arrival and its
      // MMAs (with the warp in step a wait took 160 cycles and bounded the kernel)
      if (elect_one()) {
        uint32_t item = 0, pieces = 0;
        uint32_t pn[2] = {0, 0};  // tiles whose P was taken from each stream
        bool ok = true;
        auto wait = [&](int i, uint32_t parity) -> bool {
          ok = ok && wide_poll(bar(i), parity, abort_flag);
          return ok;
        };
        auto wait_item = [&](uint32_t it) { return wait(Cfg::B_FULL0 + it % NB, (it / NB) & 1); };
        auto buf = [&](uint32_t it) -> uint32_t {
          return sbase + Cfg::kOffRing + (it % NB) * kBuf;
        };
        constexpr uint32_t kDescHi = desc_hi(1024);
        constexpr uint32_t kLboV = uint32_t(kHalf >> 4) << 16;  // V's next 64 columns
        // S_s = Q K^T, 16 dims (32 bytes of the swizzled row) per step. (All 128
        // tokens at once: with 64, each MMA still reads 4 KB of Q and takes as long.)
        auto qk = [&](int s, uint32_t it, bool release, bool last) {
          const uint32_t ad = (sbase + (MT == 2 ? s * kBuf : 0)) >> 4, bd = buf(it) >> 4;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            constexpr uint32_t kNext = kHalf >> 4;
            const uint32_t off = (k >> 2) * kNext + (k & 3) * 2;
            umma_ss(tmem + kTmemS + 128 * s, ad + off, bd + off, kDescHi, idesc_qk, k > 0);
          }
          umma_commit(bar(Cfg::B_S0 + s));
          if (release) umma_commit(bar(Cfg::B_EMPTY0 + it % NB));
          if (last) umma_commit(bar(Cfg::B_QFREE));  // Q is read for the last time
        };
        // O_s (+)= P_s[h] V_h, 16 tokens (8 TMEM columns of P) per step
        auto pv = [&](int s, int h, uint32_t it, bool first, bool release, bool last) {
          const uint32_t bd = ((buf(it) + h * (kHT * 128)) >> 4) | kLboV;
          const uint32_t d = tmem + kTmemO + 128 * s, a = tmem + kTmemS + 128 * s + kHT * h;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ts(d, a + 8 * k, bd + k * (16 * 128 / 16), kDescHi, idesc_pv, !first || k > 0);
          umma_commit(bar(Cfg::B_PV0 + s));
          if (last) umma_commit(bar(Cfg::B_O0 + s));
          if (release) umma_commit(bar(Cfg::B_EMPTY0 + it % NB));
        };
        for (int idx = s_c; idx < e_c && ok;) {
          const Piece pc = piece_at(p, prefix, idx, s_c, e_c);
          if (pc.ntiles == 0) {  // only places of a unit's fixed cost
            idx = pc.next;
            continue;
          }
          const int n = pc.ntiles;
          if (!wait(Cfg::B_Q, pieces & 1)) break;
          // the first PV of a stream overwrites the O that the epilogue reads
          auto o_free = [&](int s) -> bool {
            return pieces == 0 || wait(Cfg::B_OFREE0 + s, (pieces - 1) & 1);
          };
          if (MT == 2) {
            if (!wait_item(item)) break;
            qk(0, item, false, false);
            qk(1, item, true, n == 1);
            ++item;
            for (int t = 0; t < n && ok; ++t) {
              const uint32_t iv = item, ik = item + 1;
              const bool more = t + 1 < n;
              if (!wait_item(iv)) break;
              // stream 1 runs about half a tile behind stream 0, so this is the
              // order in which the P halves come
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                const int s = k >> 1, h = k & 1;
                if (!wait(Cfg::B_P0 + k, pn[0] & 1) || (t == 0 && h == 0 && !o_free(s))) break;
                pv(s, h, iv, t == 0 && h == 0, k == 3, h == 1 && !more);
                if (h == 1 && more) {
                  if (s == 0 && !wait_item(ik)) break;
                  qk(s, ik, s == 1, s == 1 && t + 2 == n);
                }
              }
              ++pn[0];
              item += more ? 2 : 1;
            }
          } else {
            for (int t = 0; t < 2 && t < n; ++t) {
              if (!wait_item(item)) break;
              qk(t, item++, true, t + 1 == n);
            }
            for (int t = 0; t < n && ok; ++t) {
              const int s = t & 1;
              const bool more = t + 2 < n;
              if (!wait_item(item)) break;
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                if (!wait(Cfg::B_P0 + 2 * s + h, pn[s] & 1) || (t < 2 && h == 0 && !o_free(s)))
                  break;
                pv(s, h, item, t < 2 && h == 0, h == 1, h == 1 && !more);
              }
              if (!ok) break;
              ++pn[s];
              ++item;
              if (more) {
                if (!wait_item(item)) break;
                qk(s, item++, true, t + 3 == n);
              }
            }
          }
          ++pieces;
          idx = pc.next;
        }
        if (!ok) {
          raise_error(p.err_flags, kErrTimeout);
          *abort_flag = 1;
        }
        // Every MMA done before TMEM is released.
        umma_commit(bar(Cfg::B_FINAL));
        const volatile int never = 0;
        mbar_wait(bar(Cfg::B_FINAL), 0, &never);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------- softmax
    const int s = warp >> 2;                          // stream
    const int row = 32 * (warp & 3) + lane;           // TMEM lane
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t ts = tl + kTmemS + 128 * s, to = tl + kTmemO + 128 * s;
    bool ok = true;
    auto wait_all = [&](int i, uint32_t parity) -> bool {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort_flag));
      return ok;
    };
    uint32_t tile_no = 0, pieces = 0, sn = 0;  // tiles of the CTA, pieces, tiles of this stream
    for (int idx = s_c; idx < e_c && ok;) {
      const Piece pc = piece_at(p, prefix, idx, s_c, e_c);
      if (pc.ntiles == 0) {  // only places of a unit's fixed cost
        idx = pc.next;
        continue;
      }
      const int n = pc.ntiles, L = pc.L, ctx = L - p.q_total;
      // Row `row` of this stream's row tile: token row / g of the tile's tpt,
      // head row % g (rows past the last token or past g tpt have zeros in Q:
      // they are computed and dropped).
      const int qi_all = (pc.blk * MT + (MT == 2 ? s : 0)) * p.tpt + row / p.g;
      const bool exists = row < p.g * p.tpt && qi_all < p.q_total;
      const int qi = exists ? qi_all : 0;
      const uint32_t* bits = mask_s + (pieces & 1) * 512 + qi * p.tree_words;
      // positions of the tokens from the last half-tile boundary before the
      // drafted ones on, relative to the first of these, plus kDepthBias
      const uint8_t* depth0 = depth_s + (pieces & 1) * 256;
      const int off = p.tree ? ctx & (kHT - 1) : 0;
      const uint8_t* depth = depth0 + off;
      if (p.tree && !wait_all(Cfg::B_MASK0 + (pieces & 1), (pieces >> 1) & 1)) break;
      const int pos = ctx + (p.tree ? int(depth[qi]) - kDepthBias : qi);
      const int lo_unit = p.window ? ctx - p.window + 1 : 0;  // oldest token any row sees
      const int lo_row = p.window ? max(pos - p.window + 1, 0) : 0;
      const float slope2 =
          BIAS ? __ldg(p.slopes + pc.kvh * p.g + (exists ? row % p.g : 0)) * 1.4426950408889634f
                   : 0.f;
      float m = -CUDART_INF_F, l = 0.f;
      bool bad = false;
      for (int t = MT == 2 ? 0 : s; t < n; t += MT == 2 ? 1 : 2, ++sn) {
        const uint32_t tn = tile_no + t;
        const int tok0 = (pc.last - t) * kWT;
        if (!wait_all(Cfg::B_INFO0 + tn % kInfo, (tn / kInfo) & 1)) break;
        const uint32_t tile_info = info[tn % kInfo];
        // Half tiles of 64 tokens, P in the place of S: the first half's PV runs
        // while the second half is here.
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int tok = tok0 + kHT * h;
          const uint32_t load_info = (tile_info >> (4 * h)) & 0xf0fu;  // 4 blocks of 16 tokens
          // all of it is context that every row sees
          const bool plain = load_info == 0 && tok + kHT <= ctx &&
                             (!p.window || tok >= ctx + p.q_total - p.window);
          const uint32_t tsh = ts + kHT * h;
          if (h == 0) {
            if (!wait_all(Cfg::B_S0 + s, sn & 1)) break;
            tc_fence_after();
          }
          uint64_t x[kHT / 2];  // the row's scores, two to a register pair
          load_scores(tsh, x);
          // Scores are in units of sc: base 2 once multiplied by it (sc > 0, so
          // it also takes the max).
          const float sc = CAP || BIAS ? 1.f : p.scale_log2;
          if (CAP) {
            // c tanh(s / c) in base 2 as x (f0 + f1 z + f2 z^2 + f3 z^3), z =
            // x^2, of the raw dot product x, two at a time; right up to |s| = c
            // / 2. Else the half tile takes cap_scores: the polynomial that is
            // right up to |s| = c, or where one is beyond that the full function.
            // (64 drafted tokens, 64 sequences: 212 us, 283, 405.)
            float zq[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kHT / 2; ++k) {
              const uint64_t z = mul_f32x2(x[k], x[k]);
              const float2 f = unpack_f32x2(z);
              zq[k & 1] = max3(zq[k & 1], f.x, f.y);
              uint64_t q = fma_f32x2(z, pack_f32x2(p.cap_f[3], p.cap_f[3]),
                                     pack_f32x2(p.cap_f[2], p.cap_f[2]));
              q = fma_f32x2(q, z, pack_f32x2(p.cap_f[1], p.cap_f[1]));
              q = fma_f32x2(q, z, pack_f32x2(p.cap_f[0], p.cap_f[0]));
              x[k] = mul_f32x2(q, x[k]);
            }
            const float zm = fmaxf(zq[0], zq[1]);
            if (__any_sync(0xffffffffu, !(zm <= p.cap_z))) {
              cap_scores(tsh, p.cap_in, p.cap_out, zm <= 4.f * p.cap_z);
              load_scores(tsh, x);
            }
          }
          if (BIAS) {
            const uint64_t sl2 = pack_f32x2(slope2, slope2);
            const uint64_t raw2 = pack_f32x2(p.scale_log2, p.scale_log2);
            auto add_bias = [&](uint64_t& v, uint64_t d) {
              v = CAP ? fma_f32x2(sl2, d, v) : fma_f32x2(v, raw2, mul_f32x2(sl2, d));
            };
            if (p.tree && tok + kHT > ctx) {
              // bytes to floats by way of 2^23 + byte, which is exact
              const uint32_t* rel =
                  reinterpret_cast<const uint32_t*>(depth0 + min(tok - ctx + off, 256 - kHT));
              const float back = -(8388608.f + float(kDepthBias + pos - ctx));
              const uint64_t back2 = pack_f32x2(back, back);
#pragma unroll
              for (int k = 0; k < kHT / 4; ++k) {
                const uint32_t w = rel[k];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint64_t d = add_f32x2(
                      pack_f32x2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + 2 * e)),
                                 __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441 + 2 * e))),
                      back2);
                  add_bias(x[2 * k + e], d);
                }
              }
            } else {
              // distances of two tokens by adding, which is exact; two chains
              const float d0 = float(tok - pos);
              uint64_t d[2] = {pack_f32x2(d0, d0 + 1.f), pack_f32x2(d0 + 2.f, d0 + 3.f)};
              const uint64_t four = pack_f32x2(4.f, 4.f);
#pragma unroll
              for (int k = 0; k < kHT / 2; ++k) {
                add_bias(x[k], d[k & 1]);
                d[k & 1] = add_f32x2(d[k & 1], four);
              }
            }
          }
          if (!plain) {
#pragma unroll
            for (int w = 0; w < kHT / 32; ++w) {
              const int base = tok + 32 * w;
              uint32_t vis;
              if (p.tree) {
                vis = bit_range(lo_row - base, min(ctx, L) - base);
                if (base + 32 > ctx) {
                  uint32_t dr =
                      mask_word(bits, p.tree_words, base - ctx) & bit_range(-base, L - base);
                  if (p.window && p.window < p.q_total)  // only then can it hide a drafted token
                    for (uint32_t todo = dr; todo; todo &= todo - 1) {
                      const int k = __ffs(todo) - 1;
                      if (pos - ctx - int(depth[base + k - ctx]) + kDepthBias >= p.window)
                        dr &= ~(1u << k);
                    }
                  vis |= dr;
                }
              } else {
                vis = bit_range(lo_row - base, min(pos + 1, L) - base);
              }
              const uint32_t two = load_info >> (2 * w);
              bad |= (vis & ((two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u))) != 0;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 f = unpack_f32x2(x[16 * w + k]);
                x[16 * w + k] = pack_f32x2((vis >> (2 * k)) & 1u ? f.x : -CUDART_INF_F,
                                           (vis >> (2 * k + 1)) & 1u ? f.y : -CUDART_INF_F);
              }
            }
          }
          float mq[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int k = 0; k < kHT / 2; ++k) {
            const float2 f = unpack_f32x2(x[k]);
            mq[k & 1] = max3(mq[k & 1], f.x, f.y);
          }
          const float mx = fmaxf(mq[0], mq[1]) * sc;
          // The base moves only past 2^8 (P stays at most 256); one vote per
          // warp, since the TMEM accesses are warp-wide.
          if (__any_sync(0xffffffffu, mx > m + kLazyLog2)) {
            const float mn = fmaxf(m, mx);
            const float alpha = m == -CUDART_INF_F ? 0.f : ex2_approx(m - mn);
            m = mn;
            l *= alpha;
            const bool first = h == 0 && t < (MT == 2 ? 1 : 2);
            if (!first) {  // O holds earlier half tiles: all of them, once their PV is done
              const uint32_t done = 2 * sn + h - 1;  // PVs of this stream before this one's
              if (!wait_all(Cfg::B_PV0 + s, done & 1)) break;
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < 8; ++cc) {
                uint32_t o[16];
                tmem_ld16(to + 16 * cc, o);
                tmem_wait_ld();
                hold(o);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st16(to + 16 * cc, o);
              }
            }
          }
          const float base = m == -CUDART_INF_F ? 0.f : m;
          const uint64_t sc2 = pack_f32x2(sc, sc), nb2 = pack_f32x2(-base, -base);
          uint64_t ls[2] = {0ull, 0ull};  // sums of the even and the odd tokens' P, twice
          uint32_t pk[kHT / 2];
#pragma unroll
          for (int k = 0; k < kHT / 2; ++k) {
            const float2 f = unpack_f32x2(fma_f32x2(x[k], sc2, nb2));
            const float a = ex2_approx(f.x), e = ex2_approx(f.y);
            pk[k] = pack_bf16x2(a, e);
            ls[k & 1] = add_f32x2(ls[k & 1], pack_f32x2(a, e));
          }
          tmem_st32(tsh, pk);
          {
            const float2 a = unpack_f32x2(add_f32x2(ls[0], ls[1]));
            l += a.x + a.y;
          }
          tmem_wait_st();
          // V rows that were not loaded, lie past the end or before the oldest
          // window are zeroed (P is 0 there, but 0 * NaN is not)
          if (!plain && (MT == 1 || s == 0) &&
              ((load_info >> 8) != 0 || tok + kHT > L || tok < lo_unit)) {
            const uint32_t iv = Cfg::v_item(tile_no, t, n);
            if (!wait_all(Cfg::B_FULL0 + iv % NB, (iv / NB) & 1)) break;
            // one 128-byte half row per thread
            const int vr = row & 63, at = tok + vr;
            if (((load_info >> (8 + (vr >> 4))) & 1u) || at >= L || at < lo_unit) {
              const uint32_t dst = sbase + Cfg::kOffRing + (iv % NB) * kBuf + (row >> 6) * kHalf +
                                   (kHT * h + vr) * 128;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + k * 16),
                             "r"(0u)
                             : "memory");
            }
            fence_proxy_async_smem();
          }
          tc_fence_before();
          mbar_arrive(bar(Cfg::B_P0 + 2 * s + h));
        }
        if (!ok) break;
      }
      if (!ok) break;
      // the row's base and sum for the epilogue (once it has read the ones that
      // were here; base NaN, which no score makes it: the row saw a bad page)
      const uint32_t par = pieces & 1;
      if (pieces >= 2 && !wait_all(Cfg::B_EPI0 + par, ((pieces >> 1) - 1) & 1)) break;
      ml[par * 256 + s * 128 + row] = make_float2(bad ? CUDART_NAN_F : m, l);
      mbar_arrive(bar(Cfg::B_ML0 + par));
      tile_no += n;
      ++pieces;
      idx = pc.next;
    }
    if (!ok) {
      raise_error(p.err_flags, kErrTimeout);
      *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // O / l of the finished piece, while the softmax warpgroups are at the
    // next one; for MT = 1 joined over the streams. Thread `row` holds row
    // `row`; the values pass through 2 KB of shared memory per warp so that a
    // store instruction covers 8 rows x 64 bytes (one row per thread would
    // touch 32 lines with 16 bytes each).
    const int row = 32 * (warp & 3) + lane;
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t stage = sbase + Cfg::kOffStage + (warp & 3) * kStage;
    bool ok = true;
    auto wait_all = [&](int i, uint32_t parity) -> bool {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort_flag));
      return ok;
    };
    // this lane's 16-byte chunks of the 64-byte staging rows (chunk c of row r
    // at c ^ (r / 2 % 4): free of bank conflicts both ways)
    const uint32_t put = stage + lane * 64, sw = (lane >> 1) & 3;
    auto flush = [&](char* mine, int64_t off) {  // mine: where this lane's row goes, or nullptr
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        uint4 u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4))
                     : "memory");
        const uint64_t to_row = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), r);
        if (to_row)
          *reinterpret_cast<uint4*>(reinterpret_cast<char*>(to_row) + off + (lane & 3) * 16) = u;
      }
      __syncwarp();
    };
    auto stash = [&](int c, uint32_t a, uint32_t b, uint32_t d, uint32_t e) {
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                       put + ((uint32_t(c) ^ sw) << 4)),
                   "r"(a), "r"(b), "r"(d), "r"(e)
                   : "memory");
    };
    uint32_t pieces = 0, on1 = 0;  // pieces, and those with an O of stream 1 (MT = 1)
    for (int idx = s_c; idx < e_c && ok;) {
      const Piece pc = piece_at(p, prefix, idx, s_c, e_c);
      if (pc.ntiles == 0) {  // only places of a unit's fixed cost
        idx = pc.next;
        continue;
      }
      const bool both = MT == 1 && pc.ntiles > 1;  // stream 1 had a tile
      const uint32_t par = pieces & 1;
      if (!wait_all(Cfg::B_ML0 + par, (pieces >> 1) & 1)) break;
      float2 r[2];
      r[0] = ml[par * 256 + row];
      r[1] = ml[par * 256 + 128 + row];
      mbar_arrive(bar(Cfg::B_EPI0 + par));
#pragma unroll 1
      for (int s = 0; s < MT && ok; ++s) {
        const int qi = (pc.blk * MT + s) * p.tpt + row / p.g;
        const bool exists = row < p.g * p.tpt && qi < p.q_total;
        const int64_t orow =
            (int64_t(pc.b) * p.q_total + qi) * p.Hq + pc.kvh * p.g + row % p.g;
        const int64_t wrow = (int64_t(c) * 2 + pc.slot) * (MT * 128) + s * 128 + row;
        // m, l and the weights w0, w1 of the streams' O
        float m = s ? r[1].x : r[0].x, l = s ? r[1].y : r[0].y, w0 = 1.f, w1 = 0.f;
        if (MT == 1) {
          m = fmaxf(r[0].x, r[1].x);
          w0 = r[0].x == -CUDART_INF_F ? 0.f : ex2_approx(r[0].x - m);
          w1 = r[1].x == -CUDART_INF_F ? 0.f : ex2_approx(r[1].x - m);
          l = r[0].y * w0 + r[1].y * w1;
        }
        const bool row_bad =
            MT == 1 ? isnan(r[0].x) || isnan(r[1].x) : isnan(s ? r[1].x : r[0].x);
        const bool none = row_bad || no_weight<kModeMod>(l);
        const float inv = none ? 0.f : 1.f / l;
        const float lse2 = none ? -CUDART_INF_F : m + log2f(l);
        w0 *= inv;
        w1 *= inv;
        if (__any_sync(0xffffffffu, row_bad && exists) && lane == 0)
          raise_error(p.err_flags, kErrBadPage);
        char* mine = !exists ? nullptr
                     : pc.partial ? reinterpret_cast<char*>(p.ws_o + wrow * kGqaHeadDim)
                                  : reinterpret_cast<char*>(p.out + orow * kGqaHeadDim);
        if (!wait_all(Cfg::B_O0 + s, pieces & 1)) break;
        if (both && !wait_all(Cfg::B_O0 + 1, on1 & 1)) break;
        tc_fence_after();
        // kStep columns of the row's result, w0 O_0 + w1 O_1, read at once (a
        // read takes about 300 cycles under the softmax threads' own,
        // whatever its width; for MT = 1 two O's have to fit the registers)
        constexpr int kStep = MT == 2 ? 32 : 16;
        auto columns = [&](int cc, float (&f)[kStep]) {
          uint32_t a[kStep], d[kStep];
          tmem_ld<kStep>(tl + kTmemO + 128 * s + kStep * cc, a);
          if (both) tmem_ld<kStep>(tl + kTmemO + 128 + kStep * cc, d);
          tmem_wait_ld();
          hold(a);
#pragma unroll
          for (int k = 0; k < kStep; ++k) f[k] = none ? 0.f : __uint_as_float(a[k]) * w0;
          if (both) {
            hold(d);
            if (!none) {
#pragma unroll
              for (int k = 0; k < kStep; ++k) f[k] = fmaf(__uint_as_float(d[k]), w1, f[k]);
            }
          }
        };
        // O is read in full: the next piece may overwrite it (stream 1 first:
        // the MMA warp does not wait for it in every piece)
        auto hand_back = [&] {
          tc_fence_before();
          if (MT == 1) mbar_arrive(bar(Cfg::B_OFREE0 + 1));
          mbar_arrive(bar(Cfg::B_OFREE0 + s));
        };
        if (pc.partial) {
#pragma unroll 1
          for (int cc = 0; cc < 128 / kStep; ++cc) {
            float f[kStep];
            columns(cc, f);
            if (cc == 128 / kStep - 1) hand_back();
#pragma unroll
            for (int h = 0; h < kStep / 16; ++h) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                stash(q, __float_as_uint(f[16 * h + 4 * q]),
                      __float_as_uint(f[16 * h + 4 * q + 1]),
                      __float_as_uint(f[16 * h + 4 * q + 2]),
                      __float_as_uint(f[16 * h + 4 * q + 3]));
              flush(mine, int64_t(kStep / 16 * cc + h) * 64);
            }
          }
        } else {  // 32 columns at a time (all 128 packed first took registers for which
                  // MT = 1 spilled 448 bytes: 16 drafted tokens 125 us against 122)
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 32 / kStep; ++h) {
              float f[kStep];
              columns(32 / kStep * cc + h, f);
#pragma unroll
              for (int k = 0; k < kStep / 2; ++k)
                w[kStep / 2 * h + k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
            }
            if (cc == 3) hand_back();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              stash(q, w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            flush(mine, int64_t(cc) * 64);
          }
        }
        if (exists) {
          // (of a partial: NaN a bad page, +inf a sum that is no number)
          if (pc.partial)
            p.ws_lse[wrow] = row_bad ? CUDART_NAN_F : isnan(l) ? CUDART_INF_F : lse2;
          else if (p.lse) p.lse[orow] = lse2 * 0.69314718055994531f;
        }
      }
      on1 += both ? 1 : 0;
      ++pieces;
      idx = pc.next;
    }
    if (!ok) {
      raise_error(p.err_flags, kErrTimeout);
      *abort_flag = 1;
    }
    // Sequences without tiles: zeros, lse = -inf.
    for (int b = c; b < B; b += gridDim.x) {
      if (prefix[b + 1] != prefix[b]) continue;
      const int64_t rows = int64_t(p.q_total) * p.Hq, row0 = int64_t(b) * rows;
      uint4* dst = reinterpret_cast<uint4*>(p.out + row0 * kGqaHeadDim);
      for (int64_t i = row; i < rows * kGqaHeadDim / 8; i += 128)
        dst[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (int64_t i = row; i < rows; i += 128) p.lse[row0 + i] = -CUDART_INF_F;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    // a role gave up: copies may still be on their way into this CTA's shared
    // memory (otherwise the MMA warp has waited for every one)
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000) {
    }
  }
  if (warp == 9) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partials of the units cut between CTAs, kRows rows per warp. Block
// (c - 1, y) takes rows 8 kRows y .. of the unit whose first cut is CTA c's
// first place, if there is one (the attention kernel wrote that down), and
// adds its parts in the order of the CTAs. FEW (few units, in many parts each):
// block (unit, y) looks for its unit's first cut among the G CTAs', and a warp
// takes one row, eight parts at a time (16 drafted tokens after 60000, 32 heads
// on one kv head: 55.0 -> 47.4 us; 43 drafted after 3000, 4 units: 26.7 -> 23.5).
template <int MT, bool FEW>
__global__ void __launch_bounds__(256)
gqa_wide_merge(const __grid_constant__ WideParams p, int G) {
  constexpr int kRows = FEW ? 1 : kMergeRows;
  // parts whose loads are in flight together (most units have two)
  constexpr int kBatch = FEW ? 8 : 2;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int c = blockIdx.x + 1;
  if (FEW) {
    __shared__ int s_c;
    if (threadIdx.x == 0) s_c = 0;
    __syncthreads();
    for (int i = 1 + threadIdx.x; i < G; i += 256) {
      const int4 e = __ldcg(p.ws_cut + i);
      if (e.z >= 0 && int64_t(e.x) * p.Hkv * p.nblk + e.y == blockIdx.x) s_c = i;
    }
    __syncthreads();
    c = s_c;
    if (c == 0) return;
  }
  const int4 u = __ldcg(p.ws_cut + c);
  if (u.z < 0) return;
  const int b = u.x, kvh = u.y / p.nblk, blk = u.y - kvh * p.nblk;
  const int row0 = blockIdx.y * (8 * kRows) + warp * kRows;
  int64_t orow[kRows];
  bool live[kRows], any = false;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int row = row0 + k, r = row & 127, qi = (blk * MT + row / 128) * p.tpt + r / p.g;
    live[k] = r < p.g * p.tpt && qi < p.q_total;
    any |= live[k];
    orow[k] = (int64_t(b) * p.q_total + qi) * p.Hq + kvh * p.g + r % p.g;
  }
  if (!any) return;
  MergeAcc<kRows> acc;
  acc.init();
  for (int c0 = c - 1; c0 <= u.z; c0 += kBatch) {
    float l[kBatch][kRows];
    float4 o[kBatch][kRows];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int cc = c0 + q;
      const int64_t wrow = (int64_t(cc) * 2 + (cc == c - 1 ? u.w : 0)) * (MT * 128) + row0;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (cc <= u.z && live[k]) {
          l[q][k] = __ldcg(p.ws_lse + wrow + k);
          o[q][k] =
              __ldcg(reinterpret_cast<const float4*>(p.ws_o + (wrow + k) * kGqaHeadDim) + lane);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q)
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (c0 + q <= u.z && live[k]) acc.add(k, l[q][k], o[q][k]);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (!live[k]) continue;
    const bool none = ((acc.bad >> k) & 1u) || no_weight<kModeMod>(acc.den[k]);
    const float inv = none ? 0.f : 1.f / acc.den[k];
    uint2 o = make_uint2(0u, 0u);
    if (!none)
      o = make_uint2(pack_bf16x2(acc.acc[k].x * inv, acc.acc[k].y * inv),
                     pack_bf16x2(acc.acc[k].z * inv, acc.acc[k].w * inv));
    reinterpret_cast<uint2*>(p.out + orow[k] * kGqaHeadDim)[lane] = o;
    if (p.lse && lane == 0)
      p.lse[orow[k]] = none ? -CUDART_INF_F
                            : (acc.mx[k] + log2f(acc.den[k])) * 0.69314718055994531f;
  }
}

template <int MT, bool CAP, bool BIAS>
cudaError_t launch(const WideParams& p, int grid, bool no_merge, cudaStream_t stream,
                   cudaEvent_t attn_begin, cudaEvent_t attn_end) {
  static bool done[kMaxDevices] = {};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!done[device]) {
    if ((e = cudaFuncSetAttribute(gqa_wide_kernel<MT, CAP, BIAS>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  int(WideCfg<MT>::kSmemMax))) != cudaSuccess)
      return e;
    done[device] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (attn_begin && (e = cudaEventRecord(attn_begin, stream)) != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = WideCfg<MT>::smem_bytes(p.B);
  if ((e = cudaLaunchKernelEx(&cfg, gqa_wide_kernel<MT, CAP, BIAS>, p)) != cudaSuccess) return e;
  if (attn_end && (e = cudaEventRecord(attn_end, stream)) != cudaSuccess) return e;
  if (grid < 2 || no_merge) return cudaSuccess;  // nothing is cut
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  const int64_t units = int64_t(p.B) * p.Hkv * p.nblk;
  if (units * kFewParts <= grid) {
    cfg.gridDim = dim3(unsigned(units), unsigned(MT * 128 / 8));
    return cudaLaunchKernelEx(&cfg, gqa_wide_merge<MT, true>, p, grid);
  }
  cfg.gridDim = dim3(unsigned(grid - 1), unsigned(MT * 128 / (8 * kMergeRows)));
  return cudaLaunchKernelEx(&cfg, gqa_wide_merge<MT, false>, p, grid);
}

}  // namespace

cudaError_t gqa_wide_launch(const WideParams& p, int grid, bool no_merge, cudaStream_t stream,
                            cudaEvent_t attn_begin, cudaEvent_t attn_end) {
  auto pick = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    auto* f = p.cap_in > 0.f ? (p.slopes ? launch<MT, true, true> : launch<MT, true, false>)
                             : (p.slopes ? launch<MT, false, true> : launch<MT, false, false>);
    return f(p, grid, no_merge, stream, attn_begin, attn_end);
  };
  return p.mt == 2 ? pick(std::integral_constant<int, 2>())
                   : pick(std::integral_constant<int, 1>());
}

}  // namespace zl
