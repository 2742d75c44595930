// Decode attention over a cache held in 4 bits (zl_decode_attn_q4; the row is
// described in include/zl_decode_attn.h).
//
// 144 bytes per token and kv head instead of 512: the same arithmetic has to pass
// in less than a third of the time, so what bounds the kernel besides HBM is what
// an SM issues per token: conversions, products by scales, matrix instructions. So:
//
// - Transposed products, S^T = K Q^T and O^T = V^T P^T, by mma.m16n8k16: the cache
//   is the 16-row operand and query rows are columns, 8 to an instruction (NT = 1
//   or 2 of them), so a token costs 8 + 8 instructions per 16, where queries as the
//   16-row operand would take 16 + 16.
// - Codes become fp16 pairs by one conversion each and take an eighth of their scale
//   (kUnit) in one fp16 product, exact: 6 significant bits, from 2^-21 to 46080. (The
//   whole scale would leave fp16 where its byte is 0xE3 or more, which zl_kv_append_q4
//   does not write, but others may.) fp16 rather than bf16: there is a conversion to
//   it, and P keeps 11 bits. A query row is scaled by a power of two
//   so that its largest element is in [2^14, 2^15): what falls below fp16's range is
//   2^-39 of it, and the factor goes into the softmax scale.
// - Which element, token or column sits where in a fragment is free as long as both
//   operands agree: a lane reads 16 bytes of a K row (32 consecutive elements) and
//   8 bytes of each of four V rows (one scale block). V's pairs run along tokens:
//   two tokens' words are interleaved nibble by nibble before the conversion.
// - P^T in the layout of the second product comes out of the first one by a
//   transposition of 8 x 8 fragments (movmatrix).
//
// Every warp streams the tiles (32 tokens of one kv head) of its own ring through
// TMA, one stage a tile, and is its own producer: no barrier between warps, but for
// the merge of slices below. A CTA has HB x S warps: HB kv heads side by side (a
// "bundle": with heads next to each other in memory their rows share sectors), S
// slices of the tiles of each. The tiles of all (sequence, bundle, row group) units
// are laid end to end and cut into equal ranges, one per CTA; slice s takes every
// S-th tile. Slices are merged in shared memory at the end of each unit, units that
// are cut between CTAs by a second, programmatically dependent launch, in CTA order. Short
// calls, as max_seq_len tells, have no cut and no second launch: a unit to a CTA, or to a
// cluster of them that merges it out of its CTAs' shared memory.
//
// What an SM issues decides: an mma.sync holds the issue port for 8 cycles, every other
// instruction for one, and nothing overlaps that (in registers alone, 16 conversions,
// 16 products and 4 mma take the sum of it). A ring per CTA with copies for all its
// heads at once, its warps taking turns at issuing them, needs fewer instructions and
// was slower all the same: the warps then wait for one another. Queries and page ids
// brought into L2 ahead of their use cost more in registers and instructions than they
// save (8 sequences of 32k-131k tokens: 126 us with them, 123 without).
//
// Measured, 32 query heads on 8 kv heads, from a graph: 8 sequences of 32k-131k tokens
// 123 us, 5.9 TB/s of 6.8 that a copy reaches (HBM); 64 of 512-4096 tokens 42 us (7 until
// the first tile is there, 28 of streaming, 7 of ends and merge), verifying 4 drafted
// tokens each 58 us (matrix instructions: 64 a tile, from 8 warps), 16 tokens 194 us, 64 719:
// every 16 rows of a kv head read, convert and scale its tiles again; 32 sequences of
// 1000-8000 tokens with 32 heads on one kv head 23 us.
#include "q4.cuh"
#include "q4_host.h"
#include "ptx.cuh"

#include <math_constants.h>

#include <atomic>
#include <cmath>
#include <type_traits>

namespace zl {
namespace {

constexpr int kHalf = 16;  // tokens of one copy, within a page (page sizes are multiples)
constexpr int kTile = 32;  // tokens of a ring stage: two such halves, on pages of their own
constexpr int kHalfBytes = kHalf * kQ4Row;
constexpr int kTileBytes = kTile * kQ4Row;
constexpr int kMaxBundle = 8;
constexpr int kMaxWarps = 8;  // of a CTA
// Two CTAs to an SM, of 128 registers; with 16 columns, whose outputs and queries alone
// take 96, one of 245. (64 sequences verifying 4 tokens each: with 12 warps of 168
// registers, which spill, 70 us where this took 63, and 73 with the queries in shared
// memory.)
constexpr int ctas_per_sm(int nt) { return nt == 1 ? 2 : 1; }
// What a unit costs beside its tiles (queries, the masked tile, the epilogue: some 4 us of
// a warp that shares its scheduler with three, where a tile takes 1.7), in tiles of each
// slice: places of the line that hold none. (64 sequences of 512-4096 tokens: with 2 44.1
// us, with 4 44.9; verifying 4 tokens each, so 16 columns: 65.5 and 62.6; 32 heads on one
// kv head: 27.2 and 25.2, without 36.)
constexpr int unit_cost(int nt) { return nt == 1 ? 2 : 4; }
// Short units get a CTA each where there are CTAs enough: cut, each would take n tiles of
// every slice times units / CTAs, and a merge, which costs as much as some 4 tiles. n is
// the longest's, so 8 at most. (32 units of 8 tiles for 304 CTAs: 12.0 us cut, 14.6 whole; 128
// of 5 13.1 and 12.3; with 16 columns 88 of 6 for 152 CTAs 18.1 and 15.2.)
__host__ __device__ constexpr bool whole_units(int64_t units, int64_t ctas, int64_t n) {
  return units <= ctas && n <= 8 && n * (ctas - units) <= 4 * ctas;
}
constexpr int kMaxDevices = 64;
constexpr uint64_t kTestStallNs = 50ull * 1000 * 1000;  // bound of the test hook's wait
constexpr double kLog2e = 1.4426950408889634;
// What an element counts in the products: 1 / kUnit of its value, put right in the
// softmax factor and at the end of a piece.
constexpr int kLogUnit = 3;
constexpr float kUnit = 8.f;
constexpr uint32_t kUnitF16x2 = 0x30003000u;  // 1 / kUnit twice, as fp16
// A row's softmax base moves when a score exceeds it by more than kMove, to kSlack
// below the largest: P stays below 2^15 (fp16), and starts at 2^7 so that only what
// is 2^-21 of the largest leaves fp16's normal numbers.
constexpr float kMove = 15.f;
constexpr float kSlack = 7.f;
// The base before there is one: the largest finite number, so that a score of -inf (below
// 32 bits' range) weighs nothing with it, as with any other base, and every other score
// moves it, but for those that are its own negative, whose P is 1. (With an infinity -inf
// was NaN where a slice began with such scores, and weighed nothing elsewhere.)
constexpr float kNoBase = 3.402823466e38f;

struct Q4Params {
  CUtensorMap tmap;  // 4-D bytes {144, page_size, Hkv, num_pages}, box {144, 16 or 32, 1, 1}
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  // workspace: partials of cut units, slots [CTA][2][HB][rr]: normalised outputs,
  // base-2 lse (NaN: bad, +inf: no number)
  float* ws_lse;
  float* ws_o;
  uint32_t* err_flags;
  int B, q_len, Hq, Hkv, g, page_size, num_pages;
  int HB, S, log_s;      // heads of a bundle, slices (a power of two) and their exponent
  int stages;            // of a ring
  int units_per_seq;     // bundles x row groups
  int rgroups, rr, rows; // row groups of rr rows, rows = g * q_len of a kv head
  int ctas;              // CTAs of the attention kernel
  int cost;              // places of a unit that hold no tile, a multiple of S
  int box32;             // 1: pages of a multiple of 32 tokens, copied 32 at a time
  int test_stall;        // ZL_DECODE_TEST_STALL
  int whole;             // 1: no merge: CTA c takes unit c (max_seq_len is short), or
  int log_c;             // 2^log_c CTAs, a cluster, share unit c >> log_c and merge it themselves
  Divisor page;          // by page_size
  float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t* f, uint32_t bits) {
  if (f) atomicOr(f, bits);
}

__device__ __forceinline__ int tiles_of(const Q4Params& p, int L) {
  if (L < 0 || int64_t(L) > p.bt_stride * p.page_size) return 0;
  return int((uint32_t(L) + kTile - 1) / kTile);  // (lengths go up to 2^31 - 1)
}

// How the line of W tiles is cut: G ranges, or (short units) one unit per CTA.
struct Cut {
  int64_t W;
  uint32_t G, Wr;
  int64_t Wq;  // W = Wq G + Wr
  bool whole;  // CTA c takes unit c
  __device__ __forceinline__ Cut(const Q4Params& p, int64_t tiles, int longest) {
    W = tiles * p.units_per_seq;
    const int64_t units = int64_t(p.B) * p.units_per_seq;
    whole = p.whole || whole_units(units, p.ctas, (longest + p.S - 1) >> p.log_s);
    if (W < (INT64_C(1) << 31)) {  // (nearly always: 64-bit divisions are slow)
      const uint32_t w = uint32_t(W);
      G = min(uint32_t(p.ctas), max(w >> p.log_s, 1u));
      Wq = w / G;
      Wr = w - uint32_t(Wq) * G;
    } else {
      G = uint32_t(p.ctas);
      Wq = W / G;
      Wr = uint32_t(W - Wq * G);
    }
  }
  // floor(c W / G) (c Wr < G^2 < 2^32)
  __device__ __forceinline__ int64_t start(int c) const {
    return int64_t(c) * Wq + (uint32_t(c) * Wr) / G;
  }
  // The CTA whose range holds tile x: the largest c with start(c) <= x, from an
  // estimate that is off by one at most.
  __device__ __forceinline__ int owner(int64_t x) const {
    int c = min(int(float(x) * (float(G) / float(W))), int(G) - 1);
    while (start(c) > x) --c;
    while (c + 1 < int(G) && start(c + 1) <= x) ++c;
    return c;
  }
};

// Largest b below B with m * prefix[b] <= idx < m * prefix[B] (sequences without tiles are
// skipped: the next prefix equals theirs), by a warp, 32 places a step.
__device__ __forceinline__ int locate(const int32_t* prefix, int B, int m, int64_t idx) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // among lo .. lo + n - 1, lo the least
  while (n > 1) {
    const int step = (n + 31) >> 5, at = min(lane * step, n - 1);
    const uint32_t below =
        __ballot_sync(0xffffffffu, lane == 0 || int64_t(m) * prefix[lo + at] <= idx);
    const int last = 31 - __clz(int(below));
    const int next = min(last * step, n - 1);
    lo += next;
    n = min(step, n - next);
  }
  return lo;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing added to.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// a where m is set, b elsewhere, in one instruction.
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(d) : "r"(a), "r"(b), "r"(m));
  return d;
}

// 8 x 8 fragment of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Fragment row r of the 16 tokens of a half is token half_token(r): even rows of
// each half take tokens 0, 2, 4, 6 (second half: 1, 3, 5, 7), odd ones 12, 14, 8, 10
// (13, 15, 9, 11). Rows of 36 words: with neighbouring rows 4 mod 8 tokens apart the
// K reads, and with a lane's four V tokens 2 mod 8 apart the V reads, touch every
// bank once.
__device__ __forceinline__ int half_token(int r) {
  const int k = r & 7;
  return ((k & 1) ? ((k + 3) & 7) + 8 : k) + (r >> 3);
}

// To 1 ulp, and to 2^-22 (the outputs are rounded to 2^-9 and lse is compared in 2^-20).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// From the shared memory of a CTA of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Merges n partials of a row, four columns per lane, in order.
struct RowMerge {
  float m, den;
  float4 o;
  bool bad;
  __device__ __forceinline__ void init() {
    m = -CUDART_INF_F;
    den = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    bad = false;
  }
  // A part of base-2 lse l with normalised outputs v.
  __device__ __forceinline__ void add(float l, float4 v) {
    bad |= isnan(l);
    const float mn = fmaxf(m, l);
    if (mn == -CUDART_INF_F || isnan(l)) return;
    const float a = ex2_approx(m - mn), w = ex2_approx(l - mn);
    den = fmaf(den, a, w);
    o.x = fmaf(w, v.x, o.x * a);
    o.y = fmaf(w, v.y, o.y * a);
    o.z = fmaf(w, v.z, o.z * a);
    o.w = fmaf(w, v.w, o.w * a);
    m = mn;
  }
};

// Index of row r (of a kv head's g * q_len) among the [B, q_len, Hq] query rows.
__device__ __forceinline__ int64_t query_row(const Q4Params& p, int b, int h, int r) {
  const int i = r / p.g;
  return (int64_t(b) * p.q_len + i) * p.Hq + h * p.g + (r - i * p.g);
}

// The line: each sequence with tiles takes that many places and those of the unit's cost,
// for every of its units. Places before each sequence for one unit, prefix[0 .. B] in
// shared memory, behind them where HALVES a bit for each sequence whose last tile has a
// token in its second half, and the most tiles that one has; by the whole block.
template <bool HALVES>
__device__ __forceinline__ void scan_tiles(const Q4Params& p, int32_t* prefix, int* longest) {
  __shared__ int part_sum[32], part_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int per = (p.B + 32 * warps - 1) / (32 * warps) * 32;  // a warp's run of sequences
  const int b0 = warp * per;
  int carry = 0, most = 0;
  for (int i = 0; i < per && b0 + i < p.B; i += 32) {
    const int b = b0 + i + lane;
    const int L = b < p.B ? __ldcg(p.seq_lens + b) : 0;
    const int n = tiles_of(p, L);
    if (HALVES) {
      const uint32_t both = __ballot_sync(0xffffffffu, n > 0 && (L - 1) % kTile >= kHalf);
      if (lane == 0) prefix[p.B + 1 + (b0 + i) / 32] = int32_t(both);
    }
    int incl = n > 0 ? n + p.cost : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    most = max(most, n);
    if (b < p.B) prefix[b + 1] = carry + incl;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  if (lane == 0) {
    part_sum[warp] = carry;
    part_max[warp] = most;
  }
  __syncthreads();
  int before = 0, top = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += part_sum[w];
    top = max(top, part_max[w]);
  }
  for (int i = lane; i < per && b0 + i < p.B; i += 32) prefix[b0 + i + 1] += before;
  if (threadIdx.x == 0) prefix[0] = 0;
  *longest = top;
  __syncthreads();
}

// CLUSTER: p.log_c > 0 (an instance of its own: the code that it adds costs short calls
// 0.3 us).
template <int NT, bool CLUSTER>
__global__ void __launch_bounds__(32 * kMaxWarps, ctas_per_sm(NT))
q4_decode_kernel(const __grid_constant__ Q4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HB = p.HB, S = p.S, log_s = p.log_s, W = HB * S;  // W warps
  const int NS = p.stages;
  uint8_t* ring = smem + warp * NS * kTileBytes;
  // slices' results at the end of a unit: base-2 lse [warp][8 NT], outputs [warp][8 NT][128]
  constexpr int kRows = 8 * NT;
  float* merge_l = reinterpret_cast<float*>(smem + W * NS * kTileBytes);
  float* merge_o = merge_l + (S > 1 ? W * kRows : 0);
  uint64_t* bars = reinterpret_cast<uint64_t*>(merge_o + (S > 1 ? W * kRows * 128 : 0));
  const uint32_t full = smem_u32(bars + warp * NS);
  int32_t* prefix = reinterpret_cast<int32_t*>(bars + W * NS);  // [B + 1], and B bits
  __shared__ int abort_flag;

  if (tid == 0) abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(full + 8 * s, 1);
    fence_mbar_init();
    if (warp == 0) tma_prefetch_desc(&p.tmap);
  }
  // nothing before this reads or writes global memory
  griddep_wait();
  int longest;
  scan_tiles<true>(p, prefix, &longest);
  const int32_t* both = prefix + p.B + 1;

  const int M = p.units_per_seq;
  const int c = blockIdx.x;
  // This CTA's part: len places of the line, from place r_c of sequence b_c's on (its units
  // end to end). Both below 2^31 (host).
  int b_c = 0, r_c = 0, len = 0;
  {
    const Cut cut(p, prefix[p.B], longest);
    if (cut.whole) {
      const int unit = CLUSTER ? c >> p.log_c : c;
      if (unit < int64_t(p.B) * M) {
        b_c = unit / M;
        len = prefix[b_c + 1] - prefix[b_c];
        r_c = (unit - b_c * M) * len;
        if (CLUSTER && len > 0) {  // this CTA's share of each slice
          const int n = len - p.cost, m = (n + S - 1) >> log_s;
          const int k = c & ((1 << p.log_c) - 1);
          const int j0 = (k * m >> p.log_c) << log_s;
          len = min(((k + 1) * m >> p.log_c) << log_s, n) - j0;
          r_c += j0;
        }
      }
    } else if (c < int(cut.G) && cut.W > 0) {
      const int64_t s_c = cut.start(c);
      len = int(cut.start(c + 1) - s_c);
      b_c = locate(prefix, p.B, M, s_c);
      r_c = int(s_c - int64_t(M) * prefix[b_c]);
    }
  }
  // places of all units of sequence b
  auto seq_tiles = [&](int b) { return (prefix[b + 1] - prefix[b]) * M; };

  const int sl = warp / HB, hb = warp - sl * HB;
  // This warp's tiles: of the range's places sl, sl + S, .. those that hold one.
  int count = 0;
  {
    int b = b_c, r = r_c;
    for (int at = 0; at < len;) {
      while (r >= seq_tiles(b)) r -= seq_tiles(b++);
      const int places = prefix[b + 1] - prefix[b], n = places - p.cost;
      const int j = M > 1 ? r % places : r;
      const int piece = min(len - at, places - j), real = max(min(piece, n - j), 0);
      const int skip = (sl - at) & (S - 1);
      if (skip < real) count += ((real - 1 - skip) >> log_s) + 1;
      at += piece;
      r += piece;
    }
  }
  // Moves (b, r) to the first place from r on, in steps of S, that holds a tile; returns how
  // many of the unit's tiles lie from there on in such steps, and the tile's own number.
  auto to_tile = [&](int& b, int& r, int& unit, int& j) -> int {
    for (;;) {
      while (r >= seq_tiles(b)) r -= seq_tiles(b++);
      const int places = prefix[b + 1] - prefix[b], n = places - p.cost;
      unit = M > 1 ? r / places : 0;
      j = r - unit * places;
      if (j < n) return (n - j + S - 1) >> log_s;
      r += (places - j + S - 1) & -S;
    }
  };
  // The i-th of this warp's tiles behind the one at (b, r).
  auto tile_behind = [&](int i, int& b, int& r, int& unit, int& j) {
    for (;;) {
      const int here = to_tile(b, r, unit, j);
      if (i < here) {
        r += i * S;
        j += i * S;
        return;
      }
      i -= here;
      r += here * S;
    }
  };

  // ---- the warp as its own producer: lanes 2 i and 2 i + 1 hold page and place of
  // the halves of its tile 16 j + i (place -1: no token there, or a bad page)
  int page = 0, coord = -1;
  int b_next = b_c, r_next = r_c + sl;  // where the next batch begins
  bool any_bad = false;  // a half on a bad page so far (the same in every lane)
  auto resolve = [&](int k0) {
    page = 0;
    coord = -1;
    int unit, j;
    if (k0 + (lane >> 1) < count) {
      int b = b_next, r = r_next;
      tile_behind(lane >> 1, b, r, unit, j);
      const int t = j * kTile + (lane & 1) * kHalf, pg = int(p.page.quotient(uint32_t(t)));
      // (a half behind the last token has no page; the table's row is not read there)
      if (!(lane & 1) || j + 1 + p.cost < prefix[b + 1] - prefix[b] ||
          (both[b / 32] >> (b % 32) & 1)) {
        page = p.block_table[b * p.bt_stride + pg];
        coord = (t - pg * p.page_size) |
                (((p.rgroups > 1 ? unit / p.rgroups : unit) * HB + hb) << 10);
      }
    }
    if (k0 + 16 < count) tile_behind(16, b_next, r_next, unit, j);
    const bool bad = page < 0 || page >= p.num_pages;
    any_bad |= __any_sync(0xffffffffu, bad);
    if (bad) {
      flag(p.err_flags, ZL_DEVERR_BAD_PAGE);
      coord = -1;
    }
  };
  // Tile k into the stage at `to`; the same values in every lane, one lane issues (a
  // copy per lane would be issued lane by lane).
  auto issue = [&](int k, uint32_t to, uint32_t bar) {
    const int src = 2 * (k & 15);
    if (src == 0) resolve(k);
    const int c0 = __shfl_sync(0xffffffffu, coord, src), p0 = __shfl_sync(0xffffffffu, page, src);
    if (p.box32) {  // both halves lie on one page
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, c0 >= 0 ? kTileBytes : 0);
        if (c0 >= 0) tma_load_4d(to, &p.tmap, bar, 0, c0 & 1023, c0 >> 10, p0);
      }
    } else {
      const int c1 = __shfl_sync(0xffffffffu, coord, src + 1);
      const int p1 = __shfl_sync(0xffffffffu, page, src + 1);
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, (c0 >= 0 ? kHalfBytes : 0) + (c1 >= 0 ? kHalfBytes : 0));
        if (c0 >= 0) tma_load_4d(to, &p.tmap, bar, 0, c0 & 1023, c0 >> 10, p0);
        if (c1 >= 0) tma_load_4d(to + kHalfBytes, &p.tmap, bar, 0, c1 & 1023, c1 >> 10, p1);
      }
    }
  };
  const uint32_t ring_u32 = smem_u32(ring);
  __syncwarp();
  for (int k = 0; k < NS && k < count; ++k) issue(k, ring_u32 + k * kTileBytes, full + 8 * k);

  // Sequences without tiles: zeros.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    const int L = p.seq_lens[b];
    if (tid == 0 && L != 0) flag(p.err_flags, ZL_DEVERR_BAD_SEQ_LEN);
    const int64_t r0 = int64_t(b) * p.q_len * p.Hq;
    uint4* o = reinterpret_cast<uint4*>(p.out + r0 * 128);
    for (int64_t e = tid; e < int64_t(p.q_len) * p.Hq * 16; e += blockDim.x)
      o[e] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int64_t e = tid; e < int64_t(p.q_len) * p.Hq; e += blockDim.x)
        p.lse[r0 + e] = -CUDART_INF_F;
  }

  const int gid = lane >> 2, t4 = lane & 3;
  const int tok_k = half_token(gid);   // K: this lane's first row (the other is one on)
  const int tok_a = half_token(2 * t4), tok_b = half_token(2 * t4 + 1);  // V: and one on each
  const uint8_t* tile_at = ring;  // the stage to be read next
  uint32_t bar_at = full, phase = 0;
  int left = count - NS;  // tiles not issued yet
  bool dead = false;      // a wait gave up: nothing is waited for or issued any more
  int left_dead = 0;
  auto wait = [&] {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar_at, phase))) return;
    if (__all_sync(0xffffffffu, mbar_wait(bar_at, phase, &abort_flag))) return;
    if (lane == 0) {
      flag(p.err_flags, ZL_DEVERR_TIMEOUT);
      *const_cast<volatile int*>(&abort_flag) = 1;
    }
    dead = true;
    left_dead = left;
  };
  // Hands the stage back, to the tile NS further on.
  auto next = [&] {
    __syncwarp();  // every lane has read the stage
    if (left > 0 && !dead) issue(count - left, smem_u32(tile_at), bar_at);
    --left;
    tile_at += kTileBytes;
    bar_at += 8;
    if (bar_at == full + 8 * NS) {
      tile_at = ring;
      bar_at = full;
      phase ^= 1u;
    }
  };
  bool merged_before = false;
  if (p.test_stall && warp == 0) {  // as where a wait of its first tile gives up
    __shared__ int never_set;
    if (lane == 0) {
      never_set = 0;
      if (!flag_wait(&never_set, kTestStallNs)) {
        flag(p.err_flags, ZL_DEVERR_TIMEOUT);
        *const_cast<volatile int*>(&abort_flag) = 1;
      }
    }
    __syncwarp();
    dead = true;
    left_dead = left;
  }

  int pos = 0;  // in this CTA's range
  while (pos < len) {
    while (r_c >= seq_tiles(b_c)) r_c -= seq_tiles(b_c++);
    const int b = b_c;
    const int places = prefix[b + 1] - prefix[b], n = places - p.cost;
    const int unit = M > 1 ? r_c / places : 0, j0 = r_c - unit * places;
    const int piece_end = min(len, pos - j0 + places);
    const bool cut_unit = j0 > 0 || piece_end - pos < n;
    const int slot = j0 > 0 || pos == 0 ? 0 : 1;  // (1: the unit begins behind the range's start)
    const int h = unit / p.rgroups * HB + hb;
    const int row0 = unit % p.rgroups * p.rr;
    const int R = min(p.rr, p.rows - row0);
    const int L = p.seq_lens[b];

    // Q^T fragments: column gid is query row row0 + 8 nt + gid; this lane's 32
    // elements from 32 t4 on, as fp16 times a power of two.
    uint32_t qf[NT][16];
    uint64_t fac2[NT];  // softmax scales of columns 2 t4 and 2 t4 + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + gid;
      uint4 w[4] = {};
      if (r < R) {
        const uint4* src =
            reinterpret_cast<const uint4*>(p.q + query_row(p, b, h, row0 + r) * 128) + 4 * t4;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = src[i];
      }
      const uint32_t* x = reinterpret_cast<const uint32_t*>(w);
      // the largest magnitude, by its bits (NaN above infinity)
      uint32_t m2 = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m2 = __vmaxu2(m2, x[i] & 0x7FFF7FFFu);
      uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // times 2^(14 - e), e the exponent of the largest (at least -100); a row that holds
      // a NaN or an infinity becomes NaN
      const int e = max(int(amax >> 7) - 127, -100);
      const float up =
          amax < 0x7F80u ? __uint_as_float(uint32_t(127 + 14 - e) << 23) : CUDART_NAN_F;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 v = unpack_bf16x2(x[i]);
        qf[nt][i] = pack_f16x2(v.x * up, v.y * up);
      }
      const float down = p.scale_log2 * __uint_as_float(uint32_t(127 - 14 + kLogUnit + e) << 23);
      fac2[nt] = pack_f32x2(__shfl_sync(0xffffffffu, down, 8 * t4),
                            __shfl_sync(0xffffffffu, down, 8 * t4 + 4));
    }
    // tokens that column 2 t4 + u of 8-column tile nt sees
    auto limit = [&](int nt, int u) {
      return L - p.q_len + 1 + (row0 + 8 * nt + 2 * t4 + u) / p.g;
    };
    const int all_see = L - p.q_len + 1 + row0 / p.g;  // tokens that every row sees

    float o[NT][8][4];
    float base[NT][2], l[NT][2];  // base: it is added to a score (kNoBase: none yet)
    bool bad_row[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        base[nt][u] = kNoBase;
        l[nt][u] = 0.f;
        bad_row[nt][u] = false;
      }
    }

    // One tile: tokens tok0 .. tok0 + 31 of the sequence; MASKED: some row does not see
    // all of them. valid: how many there are.
    auto run_tile = [&](auto masked_t, int tok0, int valid) {
      constexpr bool MASKED = decltype(masked_t)::value;
      const uint8_t* tile = tile_at;
      // S^T: of each half, rows tok_k and tok_k + 1 of K, 32 elements of each
      float s[2][NT][4];
      {
        uint4 ca[2], cb[2];
        uint32_t fa[2][2], fb[2][2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* row = tile + hf * kHalfBytes + tok_k * kQ4Row;
          ca[hf] = *reinterpret_cast<const uint4*>(row + 16 * t4);
          cb[hf] = *reinterpret_cast<const uint4*>(row + kQ4Row + 16 * t4);
          const uint8_t* sc = row + kQ4KScales + 2 * t4;
          fa[hf][0] = mul_f16x2(sc[0] * 0x00800080u, kUnitF16x2);
          fa[hf][1] = mul_f16x2(sc[1] * 0x00800080u, kUnitF16x2);
          fb[hf][0] = mul_f16x2(sc[kQ4Row] * 0x00800080u, kUnitF16x2);
          fb[hf][1] = mul_f16x2(sc[kQ4Row + 1] * 0x00800080u, kUnitF16x2);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t xa[4], xb[4];
            q4_pairs(w == 0 ? ca[hf].x : w == 1 ? ca[hf].y : w == 2 ? ca[hf].z : ca[hf].w, xa);
            q4_pairs(w == 0 ? cb[hf].x : w == 1 ? cb[hf].y : w == 2 ? cb[hf].z : cb[hf].w, xb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              xa[i] = mul_f16x2(xa[i], fa[hf][w >> 1]);
              xb[i] = mul_f16x2(xb[i], fb[hf][w >> 1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (w == 0)
                mma_f16_first(s[hf][nt], xa[0], xb[0], xa[1], xb[1], qf[nt][4 * w], qf[nt][4 * w + 1]);
              else
                mma_f16(s[hf][nt], xa[0], xb[0], xa[1], xb[1], qf[nt][4 * w], qf[nt][4 * w + 1]);
              mma_f16(s[hf][nt], xa[2], xb[2], xa[3], xb[3], qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
            }
          }
        }
      }

      // Softmax. This lane: of each half tokens tok_k, tok_k + 1 of columns 2 t4, 2 t4 + 1.
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        auto hidden = [&](int hf, int i) {
          return MASKED && tok0 + 16 * hf + tok_k + (i >> 1) >= limit(nt, i & 1);
        };
        float y[2][4];
        auto scores = [&] {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (not fused: the largest score less itself is 0 at any size)
              if ((i & 1) == 0) {
                const float2 v = unpack_f32x2(add_f32x2(
                    mul_f32x2(pack_f32x2(s[hf][nt][i], s[hf][nt][i + 1]), fac2[nt]),
                    pack_f32x2(base[nt][0], base[nt][1])));
                y[hf][i] = v.x;
                y[hf][i + 1] = v.y;
              }
            }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (hidden(hf, i)) y[hf][i] = -CUDART_INF_F;
        };
        scores();
        const float top = fmaxf(fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3])),
                                fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
        if (__any_sync(0xffffffffu, top > kMove)) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float mx = -CUDART_INF_F;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int i = u; i < 4; i += 2)
                if (!hidden(hf, i)) mx = fmaxf(mx, __fmul_rn(s[hf][nt][i], u ? unpack_f32x2(fac2[nt]).y : unpack_f32x2(fac2[nt]).x));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            // moves to kSlack below the largest where that is upwards
            const float nb = kSlack - mx;
            if (mx != -CUDART_INF_F && nb < base[nt][u]) {
              const float alpha = ex2_approx(nb - base[nt][u]);  // (0 from kNoBase)
              base[nt][u] = nb;
              l[nt][u] *= alpha;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                o[nt][mt][u] *= alpha;
                o[nt][mt][u + 2] *= alpha;
              }
            }
          }
          scores();
        }
        uint64_t sum = pack_f32x2(l[nt][0], l[nt][1]);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[hf][i] = ex2_approx(y[hf][i]);
          sum = add_f32x2(sum, add_f32x2(pack_f32x2(y[hf][0], y[hf][1]),
                                         pack_f32x2(y[hf][2], y[hf][3])));
          pf[hf][nt][0] = transpose_8x8(pack_f16x2(y[hf][0], y[hf][1]));
          pf[hf][nt][1] = transpose_8x8(pack_f16x2(y[hf][2], y[hf][3]));
        }
        const float2 sums = unpack_f32x2(sum);
        l[nt][0] = sums.x;
        l[nt][1] = sums.y;
      }

      // O^T: elements 16 gid .. 16 gid + 15 of V rows a, b (first 8 fragment rows of a
      // half's 16 tokens), a + 1, b + 1 (the others)
      uint32_t nan_at = 0;  // tokens whose block of this lane's elements is NaN
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint8_t* ra = tile + hf * kHalfBytes + tok_a * kQ4Row + kQ4VCodes + 8 * gid;
        const uint8_t* rb = tile + hf * kHalfBytes + tok_b * kQ4Row + kQ4VCodes + 8 * gid;
        const uint2 a0 = *reinterpret_cast<const uint2*>(ra);
        const uint2 a1 = *reinterpret_cast<const uint2*>(ra + kQ4Row);
        const uint2 b0 = *reinterpret_cast<const uint2*>(rb);
        const uint2 b1 = *reinterpret_cast<const uint2*>(rb + kQ4Row);
        const uint8_t* sa = tile + hf * kHalfBytes + tok_a * kQ4Row + kQ4VScales + gid;
        const uint8_t* sb = tile + hf * kHalfBytes + tok_b * kQ4Row + kQ4VScales + gid;
        uint32_t s0 = sa[0], s1 = sa[kQ4Row], s2 = sb[0], s3 = sb[kQ4Row];
        if (MASKED) {  // what lies behind the sequence may hold anything
          s0 = 16 * hf + tok_a < valid ? s0 : 0u;
          s1 = 16 * hf + tok_a + 1 < valid ? s1 : 0u;
          s2 = 16 * hf + tok_b < valid ? s2 : 0u;
          s3 = 16 * hf + tok_b + 1 < valid ? s3 : 0u;
          // a NaN would reach rows that do not see its token (0 times it): kept apart
          auto keep_apart = [&](uint32_t& sv, int tok) {
            if (sv >= 0xF8u) {
              nan_at |= 1u << (16 * hf + tok);
              sv = 0u;
            }
          };
          keep_apart(s0, tok_a);
          keep_apart(s1, tok_a + 1);
          keep_apart(s2, tok_b);
          keep_apart(s3, tok_b + 1);
        }
        const uint32_t f0 = mul_f16x2(s0 * 0x80u + s2 * 0x800000u, kUnitF16x2);
        const uint32_t f1 = mul_f16x2(s1 * 0x80u + s3 * 0x800000u, kUnitF16x2);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t wa0 = w ? a0.y : a0.x, wb0 = w ? b0.y : b0.x;
          const uint32_t wa1 = w ? a1.y : a1.x, wb1 = w ? b1.y : b1.x;
          uint32_t x0[4], y0[4], x1[4], y1[4];  // even and odd elements
          q4_pairs(select_bits(wa0, wb0 << 4, 0x0F0F0F0Fu), x0);
          q4_pairs(select_bits(wa0 >> 4, wb0, 0x0F0F0F0Fu), y0);
          q4_pairs(select_bits(wa1, wb1 << 4, 0x0F0F0F0Fu), x1);
          q4_pairs(select_bits(wa1 >> 4, wb1, 0x0F0F0F0Fu), y1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t m0 = mul_f16x2(x0[i], f0), m1 = mul_f16x2(y0[i], f0);
            const uint32_t m2 = mul_f16x2(x1[i], f1), m3 = mul_f16x2(y1[i], f1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[nt][4 * w + i], m0, m1, m2, m3, pf[hf][nt][0], pf[hf][nt][1]);
          }
        }
      }
      if (MASKED && __any_sync(0xffffffffu, nan_at != 0)) {
        nan_at |= __shfl_xor_sync(0xffffffffu, nan_at, 1);
        nan_at |= __shfl_xor_sync(0xffffffffu, nan_at, 2);
        if (nan_at) {
          const int first = tok0 + __ffs(int(nan_at)) - 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (first < limit(nt, u))
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) o[nt][mt][u] = o[nt][mt][u + 2] = CUDART_NAN_F;
        }
      }
    };

    // this slice's tiles of the piece: todo of them from token tok0 on, the first `plain`
    // of which every row sees whole
    const int t0 = pos + ((sl - pos) & (S - 1));
    const int real_end = min(piece_end, pos - j0 + n);  // (behind it: places without a tile)
    int todo = t0 < real_end ? ((real_end - 1 - t0) >> log_s) + 1 : 0;
    int tok0 = (j0 + t0 - pos) * kTile;
    const int stride = S * kTile;  // tokens from one to the next
    while (todo > 0) {
      int plain =
          all_see - kTile >= tok0 ? min(todo, ((all_see - kTile - tok0) >> (log_s + 5)) + 1) : 0;
      for (; plain > 0 && !dead; --plain) {
        wait();
        if (dead || any_bad) break;
        run_tile(std::false_type{}, tok0, kTile);
        next();
        --todo;
        tok0 += stride;
      }
      if (todo == 0) break;
      // one of the others: the newest, or any where a page was bad
      if (plain == 0 && !dead) wait();
      if (!dead) {
        int whole = kTile;  // tokens before a bad half
        if (any_bad) {
          const int at = tok0 + (lane & 1) * kHalf;
          int pg = 0;
          if (at < L) pg = p.block_table[b * p.bt_stride + p.page.quotient(uint32_t(at))];
          const uint32_t bad = __ballot_sync(0xffffffffu, pg < 0 || pg >= p.num_pages) & 3u;
          whole = bad & 1u ? 0 : bad ? kHalf : kTile;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) bad_row[nt][u] |= bad && tok0 + whole < limit(nt, u);
        }
        // (a row that does not see the bad half still needs the good one)
        if (whole > 0) run_tile(std::true_type{}, tok0, min(L - tok0, whole));
      } else {  // never read: its rows end as those that see a bad page
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 2; ++u) bad_row[nt][u] |= tok0 < limit(nt, u);
      }
      next();
      --todo;
      tok0 += stride;
    }

    r_c += piece_end - pos;
    const bool any_tile = j0 < n;
    pos = piece_end;
    // The merge may be placed on this SM from here on: earlier it would take the room of
    // CTAs that have not begun.
    if (pos == len) griddep_launch_dependents();
    if (!any_tile) continue;  // (only places without tiles)

    // ---- end of the piece: sums over the 8 lanes of a column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], 4);
        l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], 8);
        l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], 16);
      }
    const int64_t part0 = ((int64_t(c) * 2 + slot) * HB + hb) * p.rr;
    if (S == 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 8 * nt + 2 * t4 + u;
          if (r >= R) continue;
          const bool none = bad_row[nt][u] || l[nt][u] == 0.f;
          const float inv = none ? 0.f : kUnit * rcp_approx(l[nt][u]);
          const float lse2 = none ? -CUDART_INF_F : lg2_approx(l[nt][u]) - base[nt][u];
          float v[16];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            v[2 * mt] = none ? 0.f : o[nt][mt][u] * inv;
            v[2 * mt + 1] = none ? 0.f : o[nt][mt][u + 2] * inv;
          }
          if (cut_unit) {
            float4* to = reinterpret_cast<float4*>(p.ws_o + (part0 + r) * 128 + 16 * gid);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (gid == 0)
              p.ws_lse[part0 + r] = bad_row[nt][u] ? CUDART_NAN_F
                                    : isnan(lse2)  ? CUDART_INF_F
                                                   : lse2;
          } else {
            const int64_t row = query_row(p, b, h, row0 + r);
            uint4* to = reinterpret_cast<uint4*>(p.out + row * 128 + 16 * gid);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              to[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]),
                                 pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                 pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                                 pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
            if (p.lse && gid == 0) p.lse[row] = lse2 * 0.69314718055994531f;
          }
        }
    } else {
      // Slices: each leaves its rows, then takes every S-th over all of them.
      if (merged_before) named_barrier(1 + hb, S * 32);
      merged_before = true;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 8 * nt + 2 * t4 + u;
          if (r >= R) continue;
          const bool none = bad_row[nt][u] || l[nt][u] == 0.f;
          const float inv = none ? 0.f : kUnit * rcp_approx(l[nt][u]);
          const float lse2 = none ? -CUDART_INF_F : lg2_approx(l[nt][u]) - base[nt][u];
          float* to = merge_o + (warp * kRows + r) * 128 + 16 * gid;
#pragma unroll
          for (int mt = 0; mt < 8; mt += 2)
            *reinterpret_cast<float4*>(to + 2 * mt) =
                make_float4(none ? 0.f : o[nt][mt][u] * inv, none ? 0.f : o[nt][mt][u + 2] * inv,
                            none ? 0.f : o[nt][mt + 1][u] * inv,
                            none ? 0.f : o[nt][mt + 1][u + 2] * inv);
          if (gid == 0)
            merge_l[warp * kRows + r] = bad_row[nt][u] ? CUDART_NAN_F
                                        : isnan(lse2)  ? CUDART_INF_F
                                                       : lse2;
        }
      named_barrier(1 + hb, S * 32);
      const int first = hb;  // warp of slice 0
      for (int r = sl; r < R; r += S) {
        // (the largest first: then nothing waits for the slice before)
        float top = -CUDART_INF_F, den = 0.f;
        bool bad = false;
        for (int s = 0; s < S; ++s) {
          const float ls = merge_l[(first + s * HB) * kRows + r];
          bad |= isnan(ls);
          top = fmaxf(top, ls);
        }
        const bool none = bad || top == -CUDART_INF_F;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!none) {
#pragma unroll 4
          for (int s = 0; s < S; ++s) {
            const int at = (first + s * HB) * kRows + r;
            const float wgt = ex2_approx(merge_l[at] - top);
            const float4 os = reinterpret_cast<const float4*>(merge_o + at * 128)[lane];
            den += wgt;
            v.x = fmaf(wgt, os.x, v.x);
            v.y = fmaf(wgt, os.y, v.y);
            v.z = fmaf(wgt, os.z, v.z);
            v.w = fmaf(wgt, os.w, v.w);
          }
          const float inv = rcp_approx(den);
          v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        }
        const float lse2 = none ? -CUDART_INF_F : top + lg2_approx(den);
        if (CLUSTER) {  // (this warp alone reads or writes row r by now)
          __syncwarp();
          reinterpret_cast<float4*>(merge_o + (first * kRows + r) * 128)[lane] = v;
          if (lane == 0)
            merge_l[first * kRows + r] = bad ? CUDART_NAN_F : isnan(lse2) ? CUDART_INF_F : lse2;
        } else if (cut_unit) {
          const int64_t at = part0 + r;
          reinterpret_cast<float4*>(p.ws_o + at * 128)[lane] = v;
          if (lane == 0) p.ws_lse[at] = bad ? CUDART_NAN_F : isnan(lse2) ? CUDART_INF_F : lse2;
        } else {
          const int64_t row = query_row(p, b, h, row0 + r);
          reinterpret_cast<uint2*>(p.out + row * 128)[lane] =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          if (p.lse && lane == 0) p.lse[row] = lse2 * 0.69314718055994531f;
        }
      }
    }
  }
  // A warp that stopped leaves no copy in flight (but for one that never ends).
  if (dead) {
    const volatile int never = 0;
    const int k_dead = count - NS - left_dead;
    for (int k = k_dead; k < min(count, k_dead + NS); ++k)
      mbar_wait(full + 8 * (k % NS), uint32_t(k / NS) & 1u, &never);
  }
  if constexpr (!CLUSTER) return;

  // ---- a cluster's unit: the rows of all its heads, spread over all its warps
  if (len == 0)
    for (int e = tid; e < HB * kRows; e += blockDim.x) merge_l[e] = -CUDART_INF_F;
  __syncwarp();
  cluster_sync();
  const int unit = c >> p.log_c, b = unit / M;
  if (b < p.B && prefix[b + 1] > prefix[b]) {
    const int C = 1 << p.log_c, v = unit - b * M;
    const int row0 = v % p.rgroups * p.rr, R = min(p.rr, p.rows - row0);
    for (int id = (c & (C - 1)) * W + warp; id < HB * R; id += C * W) {
      const int hh = id / R, r = id - hh * R;
      const uint32_t l_at = smem_u32(merge_l + hh * kRows + r);
      const uint32_t o_at = smem_u32(merge_o + (hh * kRows + r) * 128 + 4 * lane);
      RowMerge m;
      m.init();
#pragma unroll 4
      for (int k = 0; k < C; ++k) {
        const float part = ld_cluster(mapa_shared(l_at, k));
        float4 o4 = ld_cluster_v4(mapa_shared(o_at, k));
        if (part != -CUDART_INF_F) m.add(part, o4);  // (nothing was written for none)
      }
      const bool none = m.bad || m.den == 0.f;
      const float inv = none ? 0.f : rcp_approx(m.den);
      const int64_t row = query_row(p, b, v / p.rgroups * HB + hh, row0 + r);
      uint2 w = make_uint2(0u, 0u);
      if (!none)
        w = make_uint2(pack_bf16x2(m.o.x * inv, m.o.y * inv), pack_bf16x2(m.o.z * inv, m.o.w * inv));
      reinterpret_cast<uint2*>(p.out + row * 128)[lane] = w;
      if (p.lse && lane == 0)
        p.lse[row] = none ? -CUDART_INF_F : (m.m + lg2_approx(m.den)) * 0.69314718055994531f;
    }
  }
  __syncwarp();
  cluster_sync();  // (until then the others may read this CTA's rows)
}

// Rows of units that were cut: the parts in CTA order, PW warps to a row (each takes
// every PW-th part), 8 / PW rows to a block.
template <int PW>
__global__ void __launch_bounds__(256) q4_merge_kernel(const __grid_constant__ Q4Params p) {
  griddep_launch_dependents();
  extern __shared__ int32_t prefix[];  // [B + 1]
  constexpr int kRows = 8 / PW;
  __shared__ float2 part_ml[kRows][PW];  // maximum (NaN: bad) and sum
  __shared__ float4 part_o[kRows][PW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % PW, local = warp / PW;
  // (The lengths may be read before the attention is done: what came before it in the
  // stream was, when the attention let this launch begin.)
  int longest;
  scan_tiles<false>(p, prefix, &longest);
  const int b = blockIdx.y;
  const int n = prefix[b + 1] - prefix[b] - p.cost;  // tiles (below 1: none)
  const Cut cut(p, prefix[p.B], longest);
  // The CTAs that hold a unit's tiles, and 1 in .z where the first of them began before the
  // unit; of the sequence's first units ahead of the wait.
  auto span_of = [&](int unit) {
    const int64_t U0 =
        int64_t(p.units_per_seq) * prefix[b] + int64_t(unit) * (prefix[b + 1] - prefix[b]);
    const int lo = cut.owner(U0);
    return make_int3(lo, cut.owner(U0 + n - 1), U0 > cut.start(lo) ? 1 : 0);
  };
  constexpr int kSpans = 64;
  __shared__ int3 spans[kSpans];
  if (n > 0 && !cut.whole)
    for (int i = threadIdx.x; i < min(p.units_per_seq, kSpans); i += blockDim.x)
      spans[i] = span_of(i);
  __syncthreads();
  griddep_wait();
  if (n < 1 || cut.whole) return;
  const int64_t per_slot = int64_t(p.HB) * p.rr;
  const int rows = p.Hkv * p.rows;  // of the sequence: (head, its row)
  for (int id0 = blockIdx.x * kRows; id0 < rows; id0 += gridDim.x * kRows) {
    const int id = id0 + local;
    const int h = id / p.rows, r = id - h * p.rows;
    RowMerge m;
    m.init();
    int lo = 0, hi = 0;
    if (id < rows) {
      const int bundle = h / p.HB, rg = p.rgroups > 1 ? r / p.rr : 0;
      const int unit = bundle * p.rgroups + rg;
      const int3 span = unit < kSpans ? spans[unit] : span_of(unit);
      lo = span.x, hi = span.y;
      const int first_slot = span.z;
      const int64_t at0 = (h - bundle * p.HB) * p.rr + (r - rg * p.rr);
      for (int c0 = lo < hi ? lo + w : hi + 1; c0 <= hi; c0 += 4 * PW) {
        float l[4];
        float4 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + i * PW;
          if (c <= hi) {
            const int64_t at = (int64_t(c) * 2 + (c == lo ? first_slot : 0)) * per_slot + at0;
            l[i] = __ldcg(p.ws_lse + at);
            o[i] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + at * 128) + lane);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + i * PW <= hi) m.add(l[i], o[i]);
      }
    }
    if constexpr (PW > 1) {
      if (id0 != blockIdx.x * kRows) __syncthreads();  // (the last round has been read)
      if (lane == 0) part_ml[local][w] = make_float2(m.bad ? CUDART_NAN_F : m.m, m.den);
      part_o[local][w][lane] = m.o;
      __syncthreads();
      if (w > 0) continue;
#pragma unroll
      for (int i = 1; i < PW; ++i) {
        const float2 ml = part_ml[local][i];
        const float4 v = part_o[local][i][lane];
        m.bad |= isnan(ml.x);
        const float mn = fmaxf(m.m, ml.x);
        if (mn == -CUDART_INF_F || isnan(ml.x)) continue;
        const float a = ex2_approx(m.m - mn), c = ex2_approx(ml.x - mn);
        m.den = fmaf(m.den, a, ml.y * c);
        m.o.x = fmaf(v.x, c, m.o.x * a);
        m.o.y = fmaf(v.y, c, m.o.y * a);
        m.o.z = fmaf(v.z, c, m.o.z * a);
        m.o.w = fmaf(v.w, c, m.o.w * a);
        m.m = mn;
      }
    }
    if (lo == hi) continue;  // not cut
    const bool none = m.bad || m.den == 0.f;
    const float inv = none ? 0.f : rcp_approx(m.den);
    const int64_t row = query_row(p, b, h, r);
    uint2 v = make_uint2(0u, 0u);
    if (!none)
      v = make_uint2(pack_bf16x2(m.o.x * inv, m.o.y * inv), pack_bf16x2(m.o.z * inv, m.o.w * inv));
    reinterpret_cast<uint2*>(p.out + row * 128)[lane] = v;
    if (p.lse && lane == 0)
      p.lse[row] = none ? -CUDART_INF_F : (m.m + lg2_approx(m.den)) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------------- host
struct Plan {
  int nt, g, rows, rgroups, rr, HB, S, stages, units_per_seq, ctas, merge_warps;
  int sms;
  bool whole;  // known from max_seq_len: a CTA for every unit, or
  int log_c;   // a cluster of 2^log_c
  size_t smem, off_o, bytes;
};

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

size_t smem_bytes(const Plan& pl, int B) {
  const size_t W = size_t(pl.HB) * pl.S;
  size_t n = W * pl.stages * (kTileBytes + 8) + (size_t(B) + 1 + (size_t(B) + 31) / 32) * 4;
  if (pl.S > 1) n += W * 8 * pl.nt * (4 + 128 * 4);
  return n;
}

zl_status validate(const zl_decode_attn_q4_params* a) {
  if (!a || a->struct_size != sizeof(*a)) return ZL_ERR_INVALID_ARG;
  if (a->B < 1 || a->Hq < 1 || a->Hkv < 1 || a->q_len < 1 || a->page_size < 1 ||
      a->num_pages < 1 || a->block_table_stride < 1 || a->num_ctas < 0 || a->max_seq_len < 0)
    return ZL_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0 || a->flags & ~ZL_DECODE_TEST_STALL) return ZL_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return ZL_ERR_INVALID_ARG;
  if (a->Hq / a->Hkv > 128 || a->q_len > 128 || a->B > kMaxBatch || a->Hkv > 65535 ||
      a->num_ctas > 65535)
    return ZL_ERR_UNSUPPORTED;
  if (a->page_size % kHalf || a->page_size > 1024) return ZL_ERR_UNSUPPORTED;
  // (tile sums in 32 bits; the line of tiles times the CTAs in 64)
  if (a->block_table_stride >= (INT64_C(1) << 31)) return ZL_ERR_UNSUPPORTED;
  const int64_t tiles = a->block_table_stride * (a->page_size / kHalf) * a->B;
  if (tiles >= (INT64_C(1) << 31) || tiles * a->Hkv >= (INT64_C(1) << 40))
    return ZL_ERR_UNSUPPORTED;
  return ZL_OK;
}

template <int NT>
zl_status occupancy(size_t smem, int threads, int* n) {
  // asked once per device and form (the sizes are few: threads and, in 1 KB steps, the
  // shared memory)
  static std::atomic<int> known[kMaxDevices][16][256] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ZL_ERR_CUDA;
  std::atomic<int>& k = known[dev][threads / 32][smem / 1024];
  if ((*n = k.load(std::memory_order_relaxed)) > 0) return ZL_OK;
  for (auto kernel : {q4_decode_kernel<NT, false>, q4_decode_kernel<NT, true>})
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) !=
        cudaSuccess)
      return ZL_ERR_CUDA;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, q4_decode_kernel<NT, false>, threads,
                                                    smem) != cudaSuccess ||
      *n < 1)
    return ZL_ERR_CUDA;
  k.store(*n, std::memory_order_relaxed);
  return ZL_OK;
}

zl_status make_plan(const zl_decode_attn_q4_params* a, Plan* pl) {
  zl_status st = validate(a);
  if (st != ZL_OK) return st;
  int sms;
  if ((st = sm_count(&sms)) != ZL_OK) return st;
  pl->sms = sms;
  pl->g = a->Hq / a->Hkv;
  pl->rows = pl->g * a->q_len;
  pl->rgroups = (pl->rows + 15) / 16;
  pl->rr = (pl->rows + pl->rgroups - 1) / pl->rgroups;
  pl->rgroups = (pl->rows + pl->rr - 1) / pl->rr;
  pl->nt = pl->rr > 8 ? 2 : 1;
  // Bundle: of the divisors of Hkv up to 8 the one that leaves the fewest warps of a CTA
  // idle, the largest of those. In small calls, where slices cut the time of a unit, the
  // least with which every CTA has one unit at most: each takes some 3 us beside its tiles.
  // (51 sequences of 8-32 tokens, 5 query tokens, 32 heads on 8: 38 us with one head to a
  // CTA, 8.7 so; 64 of 64-256 tokens 18 and 11.)
  pl->HB = 1;
  const int64_t len = a->max_seq_len > 0 ? a->max_seq_len : 4096;
  const int64_t single = int64_t(a->B) * a->Hkv * pl->rgroups;  // units of one head
  const bool large = single * ((len + kTile - 1) / kTile) >= int64_t(sms) * 32;
  for (int d = 2; d <= kMaxBundle; ++d)
    if (a->Hkv % d == 0 && kMaxWarps / d * d >= kMaxWarps / pl->HB * pl->HB &&
        (large || single > int64_t(ctas_per_sm(pl->nt)) * sms * pl->HB))
      pl->HB = d;
  pl->S = 1;  // a power of two
  while (2 * pl->S * pl->HB <= kMaxWarps) pl->S *= 2;
  pl->units_per_seq = a->Hkv / pl->HB * pl->rgroups;
  // Two stages to a warp, 147 KB on an SM: more only make the requests of all SMs wait
  // for one another (with three 64 sequences of 512-4096 tokens took 49 us, not 45, and
  // 8 of 32k-131k 130, not 125).
  pl->stages = 2;
  pl->smem = round_up(smem_bytes(*pl, a->B), 1024);
  int per_sm = 0;
  const int threads = pl->HB * pl->S * 32;
  st = pl->nt == 1 ? occupancy<1>(pl->smem, threads, &per_sm)
                   : occupancy<2>(pl->smem, threads, &per_sm);
  if (st != ZL_OK) return st;
  pl->ctas = a->num_ctas > 0 ? a->num_ctas : per_sm * sms;
  if (a->num_ctas == 0 && a->max_seq_len > 0) {
    const int64_t most =
        int64_t(a->B) * pl->units_per_seq * ((len + kTile - 1) / kTile + unit_cost(pl->nt) * pl->S);
    pl->ctas = int(std::max<int64_t>(1, std::min<int64_t>(pl->ctas, most)));
  }
  const int64_t units = int64_t(a->B) * pl->units_per_seq;
  const int64_t most = ((len + kTile - 1) / kTile + pl->S - 1) / pl->S;  // tiles of a slice
  // Where they are short, one unit to a CTA, or a cluster of 2, 4 or 8 CTAs to a unit, which
  // costs 2 tiles' time more (of 8: 4), where cut units and their merge cost 5 (with 16
  // columns, whose tiles take longer, 4). (A cluster lies in one part of the device, where a
  // few SMs may be left over: of 4 or 8, three quarters of the CTAs at most. 4 sequences of
  // 1000-2000 tokens, 32 heads on 8: 11.9 us cut, 9.7 so; 3 of 807-1012, 5 query tokens, 12
  // heads on 6, 12.2 whole and 10.4.)
  pl->log_c = 0;
  pl->whole = a->max_seq_len > 0 && whole_units(units, pl->ctas, most);
  if (a->max_seq_len > 0 && a->num_ctas == 0 && pl->S > 1) {
    int64_t least = pl->whole ? most * pl->ctas
                              : most * units + (pl->nt == 1 ? 5 : 4) * int64_t(pl->ctas);
    for (int k = 1; k <= 3; ++k) {
      const int64_t n = (most + (1 << k) - 1) >> k, cost = (n + (k < 3 ? 2 : 4)) * pl->ctas;
      if ((units << k) * (k > 1 ? 4 : 3) > int64_t(pl->ctas) * 3 || n > 8 || 1 << k > most ||
          cost >= least)
        continue;
      least = cost;
      pl->log_c = k;
      pl->whole = true;
    }
  }
  if (pl->whole) pl->ctas = int(units << pl->log_c);
  // a warp of the merge reads four parts at a time; more warps to a row where a unit
  // is cut into more
  const int64_t parts = pl->ctas / units + 2;
  pl->merge_warps = parts > 24 ? 8 : parts > 12 ? 4 : parts > 6 ? 2 : 1;
  // (a CTA counts its tiles, and those of a sequence's units, in 32 bits)
  const int64_t line =
      (a->block_table_stride * a->page_size / kTile + 1 + unit_cost(pl->nt) * pl->S) * pl->units_per_seq;
  if (line * a->B / pl->ctas >= (INT64_C(1) << 29) || line >= (INT64_C(1) << 29))
    return ZL_ERR_UNSUPPORTED;
  const size_t slots = size_t(pl->ctas) * 2 * pl->HB * pl->rr;
  pl->off_o = round_up(slots * 4, 256);
  pl->bytes = pl->whole ? 0 : pl->off_o + slots * 128 * 4;
  return ZL_OK;
}

zl_status encode_pool(const zl_decode_attn_q4_params* a, CUtensorMap* map) {
  const cuuint64_t dims[4] = {kQ4Row, cuuint64_t(a->page_size), cuuint64_t(a->Hkv),
                              cuuint64_t(a->num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(a->token_stride), cuuint64_t(a->head_stride),
                                 cuuint64_t(a->page_stride)};
  const cuuint32_t box[4] = {kQ4Row, cuuint32_t(a->page_size % kTile ? kHalf : kTile), 1, 1};
  const CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                                  const_cast<void*>(a->pool), dims, strides, box);
  if (r == CUDA_ERROR_NOT_INITIALIZED) return ZL_ERR_CUDA;
  return r == CUDA_SUCCESS ? ZL_OK : ZL_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace zl

extern "C" zl_status zl_decode_attn_q4_workspace_size(const zl_decode_attn_q4_params* a,
                                                      size_t* bytes) {
  if (!bytes) return ZL_ERR_INVALID_ARG;
  zl::Plan pl;
  const zl_status st = zl::make_plan(a, &pl);
  if (st == ZL_OK) *bytes = pl.bytes;
  return st;
}

extern "C" zl_status zl_decode_attn_q4(const zl_decode_attn_q4_params* a, zl_stream_t stream) {
  using namespace zl;
  zl_status st = validate(a);
  if (st != ZL_OK) return st;
  if ((st = q4_check_pool(a)) != ZL_OK) return st;
  if (!a->q || !a->out || !aligned_to(a->q, 16) || !aligned_to(a->out, 16) ||
      !aligned_to(a->lse, 4))
    return ZL_ERR_INVALID_ARG;
  Plan pl;
  if ((st = make_plan(a, &pl)) != ZL_OK) return st;
  if (pl.bytes > 0 &&
      (!a->workspace || !aligned_to(a->workspace, 256) || a->workspace_bytes < pl.bytes))
    return ZL_ERR_WORKSPACE;
  Q4Params p;
  std::memset(&p, 0, sizeof(p));
  if ((st = encode_pool(a, &p.tmap)) != ZL_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.seq_lens = a->seq_lens;
  char* ws = static_cast<char*>(a->workspace);
  p.ws_lse = reinterpret_cast<float*>(ws);
  p.ws_o = reinterpret_cast<float*>(ws + pl.off_o);
  p.err_flags = a->err_flags;
  p.B = a->B;
  p.q_len = a->q_len;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = pl.g;
  p.page_size = a->page_size;
  p.num_pages = a->num_pages;
  p.HB = pl.HB;
  p.S = pl.S;
  while (1 << p.log_s < pl.S) ++p.log_s;
  p.stages = pl.stages;
  p.units_per_seq = pl.units_per_seq;
  p.rgroups = pl.rgroups;
  p.rr = pl.rr;
  p.rows = pl.rows;
  p.ctas = pl.ctas;
  p.cost = unit_cost(pl.nt) * pl.S;
  p.box32 = a->page_size % kTile == 0;
  p.test_stall = a->flags & ZL_DECODE_TEST_STALL ? 1 : 0;
  p.whole = pl.whole;
  p.log_c = pl.log_c;
  p.page = Divisor(uint32_t(a->page_size));
  p.scale_log2 = float(double(a->scale) * kLog2e);

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(pl.ctas));
  cfg.blockDim = dim3(unsigned(pl.HB * pl.S) * 32);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << pl.log_c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pl.log_c > 0 ? 2 : 1;
  cudaError_t e;
  if (pl.log_c > 0)
    e = pl.nt == 1 ? cudaLaunchKernelEx(&cfg, q4_decode_kernel<1, true>, p)
                   : cudaLaunchKernelEx(&cfg, q4_decode_kernel<2, true>, p);
  else
    e = pl.nt == 1 ? cudaLaunchKernelEx(&cfg, q4_decode_kernel<1, false>, p)
                   : cudaLaunchKernelEx(&cfg, q4_decode_kernel<2, false>, p);
  if (e != cudaSuccess) return ZL_ERR_CUDA;
  if (pl.whole) return ZL_OK;  // no unit is cut
  const int64_t rows = int64_t(a->Hkv) * pl.rows;  // of a sequence
  const int64_t blocks = (rows * pl.merge_warps + 7) / 8;  // four to an SM at most
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(blocks, std::max(1, 4 * pl.sms / a->B))),
                     unsigned(a->B));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = (size_t(a->B) + 1) * 4;
  switch (pl.merge_warps) {
    case 8: e = cudaLaunchKernelEx(&cfg, q4_merge_kernel<8>, p); break;
    case 4: e = cudaLaunchKernelEx(&cfg, q4_merge_kernel<4>, p); break;
    case 2: e = cudaLaunchKernelEx(&cfg, q4_merge_kernel<2>, p); break;
    default: e = cudaLaunchKernelEx(&cfg, q4_merge_kernel<1>, p);
  }
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
