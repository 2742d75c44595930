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
// - Codes become fp16 pairs by one conversion each and take their scale in one
//   fp16 product, exact (6 significant bits). fp16 rather than bf16: there is a
//   conversion to it, and P keeps 11 bits. A query row is scaled by a power of two
//   so that its largest element is in [2^14, 2^15): what falls below fp16's range is
//   2^-39 of it, and the factor goes into the softmax scale.
// - Which element, token or column sits where in a fragment is free as long as both
//   operands agree: a lane reads 16 bytes of a K row (32 consecutive elements) and
//   8 bytes of each of four V rows (one scale block). V's pairs run along tokens:
//   two tokens' words are interleaved nibble by nibble before the conversion.
// - P^T in the layout of the second product comes out of the first one by a
//   transposition of 8 x 8 fragments (movmatrix).
//
// Every warp streams the tiles (16 tokens of one kv head) of its own ring through
// TMA, one stage a tile, and is its own producer: no barrier between warps, but for
// the merge of slices below. A CTA has HB x S warps: HB kv heads side by side (a
// "bundle": with heads next to each other in memory their rows share sectors), S
// slices of the tiles of each. The tiles of all (sequence, bundle, row group) units
// are laid end to end and cut into equal ranges, one per CTA; slice s takes every
// S-th tile. Slices are merged in shared memory at the end of each unit, units that
// are cut between CTAs by a second, programmatically dependent launch, in CTA order.
#include "q4.cuh"
#include "q4_host.h"
#include "ptx.cuh"

#include <math_constants.h>

#include <cmath>

namespace zl {
namespace {

constexpr int kTile = 16;
constexpr int kTileBytes = kTile * kQ4Row;
constexpr int kMaxWarps = 8;
constexpr int kMaxDevices = 64;
constexpr double kLog2e = 1.4426950408889634;
// A row's softmax base moves when a score exceeds it by more than kMove, to kSlack
// below the largest: P stays below 2^15 (fp16), and starts at 2^7 so that only what
// is 2^-21 of the largest leaves fp16's normal numbers.
constexpr float kMove = 15.f;
constexpr float kSlack = 7.f;

struct Q4Params {
  CUtensorMap tmap;  // 4-D bytes {144, page_size, Hkv, num_pages}, box {144, 16, 1, 1}
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  // workspace: tile prefix sums [B + 1] and the longest unit; partials of cut units,
  // slots [CTA][2][HB][rr]: normalised outputs, base-2 lse (NaN: bad, +inf: no number)
  int32_t* ws_prefix;
  float* ws_lse;
  float* ws_o;
  uint32_t* err_flags;
  int B, q_len, Hq, Hkv, g, page_size, num_pages;
  int HB, S, stages;     // heads of a bundle, slices, ring stages per warp
  int units_per_seq;     // bundles x row groups
  int rgroups, rr, rows; // row groups of rr rows, rows = g * q_len of a kv head
  int ctas;              // CTAs of the attention kernel
  float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t* f, uint32_t bits) {
  if (f) atomicOr(f, bits);
}

__device__ __forceinline__ int tiles_of(const Q4Params& p, int L) {
  if (L < 0 || int64_t(L) > p.bt_stride * p.page_size) return 0;
  return (L + kTile - 1) / kTile;
}

// How the line of W tiles is cut: G ranges, or (short units) one unit per CTA.
struct Cut {
  int64_t W;
  int G;
  bool whole;  // CTA c takes unit c
  __device__ __forceinline__ Cut(const Q4Params& p, int64_t tiles, int longest) {
    W = tiles * p.units_per_seq;
    const int64_t units = int64_t(p.B) * p.units_per_seq;
    whole = units <= p.ctas && longest <= 4 * p.S;
    G = int(min(int64_t(p.ctas), max(W / (2 * p.S), int64_t(1))));
  }
  __device__ __forceinline__ int64_t start(int c) const { return W * c / G; }
  // The CTA whose range holds tile x: the largest c with start(c) <= x.
  __device__ __forceinline__ int owner(int64_t x) const { return int(((x + 1) * G - 1) / W); }
};

// Largest b with units_per_seq * prefix[b] <= idx (sequences without tiles are
// skipped: the next prefix equals theirs).
__device__ __forceinline__ int locate(const int32_t* prefix, int B, int m, int64_t idx) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (int64_t(m) * prefix[mid] <= idx) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Fragment row r of the 16 tokens of a tile is token tile_token(r): even rows of
// each half take tokens 0, 2, 4, 6 (second half: 1, 3, 5, 7), odd ones 12, 14, 8, 10
// (13, 15, 9, 11). Rows of 36 words: with neighbouring rows 4 mod 8 tokens apart the
// K reads, and with a lane's four V tokens 2 mod 8 apart the V reads, touch every
// bank once.
__device__ __forceinline__ int tile_token(int r) {
  const int k = r & 7;
  return ((k & 1) ? ((k + 3) & 7) + 8 : k) + (r >> 3);
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

template <int NT>
__global__ void __launch_bounds__(kMaxWarps * 32, NT == 1 ? 2 : 1)
q4_decode_kernel(const __grid_constant__ Q4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = p.HB * p.S;  // warps
  const int NS = p.stages;
  uint8_t* ring = smem + warp * NS * kTileBytes;
  // slices' results at the end of a unit: base-2 lse [warp][NT * 8], outputs [..][128]
  float* merge_l = reinterpret_cast<float*>(smem + W * NS * kTileBytes);
  float* merge_o = merge_l + (p.S > 1 ? W * NT * 8 : 0);
  uint64_t* full_bars = reinterpret_cast<uint64_t*>(merge_o + (p.S > 1 ? W * NT * 8 * 128 : 0));
  const uint32_t full = smem_u32(full_bars + warp * NS);
  int32_t* prefix = reinterpret_cast<int32_t*>(full_bars + W * NS);  // [B + 1]
  __shared__ int abort_flag, longest;

  if (tid == 0) abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(full + 8 * s, 1);
    fence_mbar_init();
    if (warp == 0) tma_prefetch_desc(&p.tmap);
  }
  // nothing before this reads or writes global memory
  griddep_wait();

  if (warp == 0) {
    const int per = (p.B + 31) / 32;
    int local = 0, nmax = 0;
    for (int i = 0; i < per; ++i) {
      const int b = lane * per + i;
      if (b < p.B) {
        const int n = tiles_of(p, __ldg(p.seq_lens + b));
        local += n;
        nmax = max(nmax, n);
      }
    }
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
      nmax = max(nmax, __shfl_xor_sync(0xffffffffu, nmax, off));
    }
    int run = incl - local;
    for (int i = 0; i < per; ++i) {
      const int b = lane * per + i;
      if (b < p.B) {
        prefix[b] = run;
        run += tiles_of(p, __ldg(p.seq_lens + b));
      }
    }
    if (lane == 31) prefix[p.B] = incl;
    if (lane == 0) longest = nmax;
  }
  __syncthreads();
  griddep_launch_dependents();
  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.B; b += blockDim.x) p.ws_prefix[b] = prefix[b];
    if (tid == 0) p.ws_prefix[p.B + 1] = longest;
  }

  // Sequences without tiles: zeros.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    const int L = __ldg(p.seq_lens + b);
    if (tid == 0 && L != 0) flag(p.err_flags, ZL_DEVERR_BAD_SEQ_LEN);
    const int64_t r0 = int64_t(b) * p.q_len * p.Hq;
    uint4* o = reinterpret_cast<uint4*>(p.out + r0 * 128);
    for (int64_t e = tid; e < int64_t(p.q_len) * p.Hq * 16; e += blockDim.x)
      o[e] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int64_t e = tid; e < int64_t(p.q_len) * p.Hq; e += blockDim.x)
        p.lse[r0 + e] = -CUDART_INF_F;
  }

  const int M = p.units_per_seq, S = p.S;
  const Cut cut(p, prefix[p.B], longest);
  int64_t s_c = 0, e_c = 0;
  const int c = blockIdx.x;
  if (cut.whole) {
    if (c < int64_t(p.B) * M) {
      const int b = c / M, n = prefix[b + 1] - prefix[b];
      s_c = int64_t(M) * prefix[b] + int64_t(c - b * M) * n;
      e_c = s_c + n;
    }
  } else if (c < cut.G && cut.W > 0) {
    s_c = cut.start(c);
    e_c = cut.start(c + 1);
  }

  const int hb = warp % p.HB, sl = warp / p.HB;
  const int64_t first = s_c + sl;  // this warp's tiles: first, first + S, ..
  const int64_t count = first < e_c ? (e_c - 1 - first) / S + 1 : 0;

  // ---- the warp as its own producer: lane i holds page and place of tile 32 j + i
  int page = 0, coord = 0, next_page = 0, next_coord = 0;
  uint32_t bad_tiles = 0;   // of the batch being issued
  uint32_t bad_stages = 0;  // stages that hold a tile on a bad page
  auto resolve = [&](int64_t k0) {
    const int64_t k = k0 + lane;
    next_page = 0;
    if (k < count) {
      const int64_t idx = first + k * S;
      const int b = locate(prefix, p.B, M, idx);
      const int n = prefix[b + 1] - prefix[b];
      const int64_t r = idx - int64_t(M) * prefix[b];
      const int unit = int(r / n), t = int(r - int64_t(unit) * n) * kTile;
      const int h = unit / p.rgroups * p.HB + hb;
      next_page = __ldg(p.block_table + b * p.bt_stride + t / p.page_size);
      next_coord = (t % p.page_size) | (h << 10);
    }
  };
  auto issue = [&](int64_t k, int stage) {
    const int src = int(k) & 31;
    if (src == 0) {
      page = next_page;
      coord = next_coord;
      const bool bad = page < 0 || page >= p.num_pages;
      bad_tiles = __ballot_sync(0xffffffffu, bad);
      if (bad) flag(p.err_flags, ZL_DEVERR_BAD_PAGE);
      resolve(k + 32);
    }
    const bool bad = (bad_tiles >> src) & 1u;
    bad_stages = (bad_stages & ~(1u << stage)) | (uint32_t(bad) << stage);
    if (lane == src && !bad) {
      mbar_arrive_expect_tx(full + 8 * stage, kTileBytes);
      tma_load_4d(smem_u32(ring + stage * kTileBytes), &p.tmap, full + 8 * stage, 0, coord & 1023,
                  coord >> 10, page);
    } else if (lane == src) {
      mbar_arrive(full + 8 * stage);
    }
  };
  __syncwarp();
  if (count > 0) {
    resolve(0);
    for (int k = 0; k < NS && k < count; ++k) issue(k, k);
  }

  const int gid = lane >> 2, t4 = lane & 3;
  const int tok_k = tile_token(gid);   // K: this lane's first row (the other is one on)
  const int tok_a = tile_token(2 * t4), tok_b = tile_token(2 * t4 + 1);  // V: and one on each
  int64_t k_done = 0;  // tiles of this warp consumed
  int stage = 0;
  uint32_t phase = 0;
  bool dead = false, merged_before = false;
  int64_t k_dead = 0;

  int64_t idx = s_c;
  while (idx < e_c) {
    const int b = locate(prefix, p.B, M, idx);
    const int n = prefix[b + 1] - prefix[b];
    const int64_t r0 = idx - int64_t(M) * prefix[b];
    const int unit = int(r0 / n), j0 = int(r0 - int64_t(unit) * n);
    const int64_t piece_end = min(e_c, idx - j0 + n);
    const bool cut_unit = j0 > 0 || piece_end < idx - j0 + n;
    const int slot = idx == s_c ? 0 : 1;
    const int h = unit / p.rgroups * p.HB + hb;
    const int row0 = unit % p.rgroups * p.rr;
    const int R = min(p.rr, p.rows - row0);
    const int L = __ldg(p.seq_lens + b);

    // Q^T fragments: column gid is query row row0 + 8 nt + gid; this lane's 32
    // elements from 32 t4 on, as fp16 times a power of two.
    uint32_t qf[NT][16];
    float fac[NT][2];  // softmax scale of columns 2 t4 and 2 t4 + 1
    int lim[NT][2];    // tokens they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + gid;
      uint4 w[4] = {};
      if (r < R) {
        const uint4* src =
            reinterpret_cast<const uint4*>(p.q + query_row(p, b, h, row0 + r) * 128) + 4 * t4;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(src + i);
      }
      const uint32_t* x = reinterpret_cast<const uint32_t*>(w);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 v = unpack_bf16x2(x[i]);
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^(14 - e), e the exponent of the largest (at least -100)
      const int e = max(int(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = __uint_as_float(uint32_t(127 + 14 - e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 v = unpack_bf16x2(x[i]);
        // (x * 0 is NaN for an infinity: the row is NaN then, whatever it meets)
        qf[nt][i] = pack_f16x2(fmaf(v.x, 0.f, v.x * up), fmaf(v.y, 0.f, v.y * up));
      }
      const float down = p.scale_log2 * __uint_as_float(uint32_t(127 - 14 + e) << 23);
      fac[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t4);
      fac[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
#pragma unroll
      for (int u = 0; u < 2; ++u) lim[nt][u] = L - p.q_len + 1 + (row0 + 8 * nt + 2 * t4 + u) / p.g;
    }
    const int all_see = L - p.q_len + 1 + row0 / p.g;  // tokens that every row sees

    float o[NT][8][4];
    float base[NT][2], l[NT][2];  // base: minus it is added to a score (+inf: none yet)
    bool bad_row[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        base[nt][u] = CUDART_INF_F;
        l[nt][u] = 0.f;
        bad_row[nt][u] = false;
      }
    }

    // this slice's first tile of the piece
    const int64_t behind = (idx - s_c) % S;
    int64_t t = idx + (sl >= behind ? sl - behind : sl + S - behind);
    for (; t < piece_end; t += S) {
      const int tok0 = (j0 + int(t - idx)) * kTile;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(full + 8 * stage, phase, &abort_flag))) {
        if (lane == 0) {
          flag(p.err_flags, ZL_DEVERR_TIMEOUT);
          *const_cast<volatile int*>(&abort_flag) = 1;
        }
        dead = true;
        k_dead = k_done;
      }
      if (!dead && ((bad_stages >> stage) & 1u)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 2; ++u) bad_row[nt][u] |= tok0 < lim[nt][u];
      } else if (!dead) {
        const uint8_t* tile = ring + stage * kTileBytes;
        const bool masked = tok0 + kTile > all_see;

        // S^T: rows tok_k and tok_k + 1 of K, 32 elements of each
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        {
          const uint8_t* row = tile + tok_k * kQ4Row;
          const uint4 ca = *reinterpret_cast<const uint4*>(row + 16 * t4);
          const uint4 cb = *reinterpret_cast<const uint4*>(row + kQ4Row + 16 * t4);
          const uint32_t sa = *reinterpret_cast<const uint16_t*>(row + kQ4KScales + 2 * t4);
          const uint32_t sb = *reinterpret_cast<const uint16_t*>(row + kQ4Row + kQ4KScales + 2 * t4);
          const uint32_t fa[2] = {(sa & 255u) * 0x00800080u, (sa >> 8) * 0x00800080u};
          const uint32_t fb[2] = {(sb & 255u) * 0x00800080u, (sb >> 8) * 0x00800080u};
          const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t xa[4], xb[4];
            q4_pairs(wa[w], xa);
            q4_pairs(wb[w], xb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              xa[i] = mul_f16x2(xa[i], fa[w >> 1]);
              xb[i] = mul_f16x2(xb[i], fb[w >> 1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(s[nt], xa[0], xb[0], xa[1], xb[1], qf[nt][4 * w], qf[nt][4 * w + 1]);
              mma_f16(s[nt], xa[2], xb[2], xa[3], xb[3], qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
            }
          }
        }

        // Softmax. This lane: tokens tok_k, tok_k + 1 of columns 2 t4, 2 t4 + 1.
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y[4];
          auto scores = [&] {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (not fused: the largest score less itself is 0 at any size)
              y[i] = __fadd_rn(__fmul_rn(s[nt][i], fac[nt][i & 1]), base[nt][i & 1]);
              if (masked && tok0 + tok_k + (i >> 1) >= lim[nt][i & 1]) y[i] = -CUDART_INF_F;
            }
          };
          scores();
          if (__any_sync(0xffffffffu, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) > kMove)) {
            float mx[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float x0 = __fmul_rn(s[nt][u], fac[nt][u]), x1 = __fmul_rn(s[nt][u + 2], fac[nt][u]);
              if (masked && tok0 + tok_k >= lim[nt][u]) x0 = -CUDART_INF_F;
              if (masked && tok0 + tok_k + 1 >= lim[nt][u]) x1 = -CUDART_INF_F;
              mx[u] = fmaxf(x0, x1);
              mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 4));
              mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 8));
              mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 16));
              // moves to kSlack below the largest where that is upwards
              const float nb = kSlack - mx[u];
              if (mx[u] != -CUDART_INF_F && nb < base[nt][u]) {
                const float alpha =
                    base[nt][u] == CUDART_INF_F ? 0.f : ex2_approx(nb - base[nt][u]);
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
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = ex2_approx(y[i]);
          l[nt][0] += y[0] + y[2];
          l[nt][1] += y[1] + y[3];
          pf[nt][0] = transpose_8x8(pack_f16x2(y[0], y[1]));
          pf[nt][1] = transpose_8x8(pack_f16x2(y[2], y[3]));
        }

        // O^T: elements 16 gid .. 16 gid + 15 of V rows a, b (first half of the 16
        // tokens), a + 1, b + 1 (second half)
        {
          const uint8_t* ra = tile + tok_a * kQ4Row + kQ4VCodes + 8 * gid;
          const uint8_t* rb = tile + tok_b * kQ4Row + kQ4VCodes + 8 * gid;
          const uint2 a0 = *reinterpret_cast<const uint2*>(ra);
          const uint2 a1 = *reinterpret_cast<const uint2*>(ra + kQ4Row);
          const uint2 b0 = *reinterpret_cast<const uint2*>(rb);
          const uint2 b1 = *reinterpret_cast<const uint2*>(rb + kQ4Row);
          const int at = kQ4VScales + gid;
          uint32_t s0 = tile[tok_a * kQ4Row + at], s1 = tile[(tok_a + 1) * kQ4Row + at];
          uint32_t s2 = tile[tok_b * kQ4Row + at], s3 = tile[(tok_b + 1) * kQ4Row + at];
          if (masked) {  // what lies behind the sequence may hold anything
            const int valid = L - tok0;
            s0 = tok_a < valid ? s0 : 0u;
            s1 = tok_a + 1 < valid ? s1 : 0u;
            s2 = tok_b < valid ? s2 : 0u;
            s3 = tok_b + 1 < valid ? s3 : 0u;
          }
          const uint32_t f0 = s0 * 0x80u + s2 * 0x800000u, f1 = s1 * 0x80u + s3 * 0x800000u;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t wa0 = w ? a0.y : a0.x, wb0 = w ? b0.y : b0.x;
            const uint32_t wa1 = w ? a1.y : a1.x, wb1 = w ? b1.y : b1.x;
            uint32_t x0[4], y0[4], x1[4], y1[4];  // even and odd elements of both halves
            q4_pairs((wa0 & 0x0F0F0F0Fu) | ((wb0 << 4) & 0xF0F0F0F0u), x0);
            q4_pairs(((wa0 >> 4) & 0x0F0F0F0Fu) | (wb0 & 0xF0F0F0F0u), y0);
            q4_pairs((wa1 & 0x0F0F0F0Fu) | ((wb1 << 4) & 0xF0F0F0F0u), x1);
            q4_pairs(((wa1 >> 4) & 0x0F0F0F0Fu) | (wb1 & 0xF0F0F0F0u), y1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t m0 = mul_f16x2(x0[i], f0), m1 = mul_f16x2(y0[i], f0);
              const uint32_t m2 = mul_f16x2(x1[i], f1), m3 = mul_f16x2(y1[i], f1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][4 * w + i], m0, m1, m2, m3, pf[nt][0], pf[nt][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (!dead && k_done + NS < count) issue(k_done + NS, stage);
      ++k_done;
      if (++stage == NS) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // ---- end of the piece: sums over the 8 lanes of a column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], 4);
        l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], 8);
        l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], 16);
      }
    const int64_t part0 = ((int64_t(c) * 2 + slot) * p.HB + hb) * p.rr;
    if (S == 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 8 * nt + 2 * t4 + u;
          if (r >= R) continue;
          const bool none = bad_row[nt][u] || l[nt][u] == 0.f;
          const float inv = none ? 0.f : __frcp_rn(l[nt][u]);
          const float lse2 = none ? -CUDART_INF_F : log2f(l[nt][u]) - base[nt][u];
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
      // Slices: each leaves its rows, then takes every S-th row over all of them.
      if (merged_before) named_barrier(1 + hb, S * 32);
      merged_before = true;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 8 * nt + 2 * t4 + u;
          if (r >= R) continue;
          const bool none = bad_row[nt][u] || l[nt][u] == 0.f;
          const float inv = none ? 0.f : __frcp_rn(l[nt][u]);
          const float lse2 = none ? -CUDART_INF_F : log2f(l[nt][u]) - base[nt][u];
          float* to = merge_o + (warp * NT * 8 + r) * 128 + 16 * gid;
#pragma unroll
          for (int mt = 0; mt < 8; mt += 2)
            *reinterpret_cast<float4*>(to + 2 * mt) =
                make_float4(none ? 0.f : o[nt][mt][u] * inv, none ? 0.f : o[nt][mt][u + 2] * inv,
                            none ? 0.f : o[nt][mt + 1][u] * inv,
                            none ? 0.f : o[nt][mt + 1][u + 2] * inv);
          if (gid == 0)
            merge_l[warp * NT * 8 + r] = bad_row[nt][u] ? CUDART_NAN_F
                                            : isnan(lse2)  ? CUDART_INF_F
                                                           : lse2;
        }
      named_barrier(1 + hb, S * 32);
      for (int r = sl; r < R; r += S) {
        RowMerge m;
        m.init();
        for (int s = 0; s < S; ++s) {
          const int at = (s * p.HB + hb) * NT * 8 + r;
          m.add(merge_l[at], reinterpret_cast<const float4*>(merge_o + at * 128)[lane]);
        }
        const bool none = m.bad || m.den == 0.f;
        const float inv = none ? 0.f : __frcp_rn(m.den);
        const float lse2 = none ? -CUDART_INF_F : m.m + log2f(m.den);
        const float4 v = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(m.o.x * inv, m.o.y * inv, m.o.z * inv, m.o.w * inv);
        if (cut_unit) {
          reinterpret_cast<float4*>(p.ws_o + (part0 + r) * 128)[lane] = v;
          if (lane == 0)
            p.ws_lse[part0 + r] = m.bad ? CUDART_NAN_F : isnan(lse2) ? CUDART_INF_F : lse2;
        } else {
          const int64_t row = query_row(p, b, h, row0 + r);
          reinterpret_cast<uint2*>(p.out + row * 128)[lane] =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          if (p.lse && lane == 0) p.lse[row] = lse2 * 0.69314718055994531f;
        }
      }
    }
    idx = piece_end;
  }
  // A warp that stopped leaves no copy in flight (but for one that never ends).
  if (dead) {
    const volatile int never = 0;
    for (int64_t k = k_dead; k < min(count, k_dead + NS); ++k)
      mbar_wait(full + 8 * int(k % NS), uint32_t(k / NS) & 1u, &never);
  }
}

// Rows of units that were cut, one warp each: the parts in CTA order.
__global__ void __launch_bounds__(256) q4_merge_kernel(const __grid_constant__ Q4Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = int64_t(p.B) * p.Hkv * p.rows;
  const int64_t w = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= rows) return;
  const int r = int(w % p.rows);
  const int64_t bh = w / p.rows;
  const int h = int(bh % p.Hkv), b = int(bh / p.Hkv);
  const int32_t n0 = __ldcg(p.ws_prefix + b), n = __ldcg(p.ws_prefix + b + 1) - n0;
  if (n == 0) return;
  const Cut cut(p, __ldcg(p.ws_prefix + p.B), __ldcg(p.ws_prefix + p.B + 1));
  if (cut.whole) return;
  const int bundle = h / p.HB, rg = r / p.rr;
  const int64_t U0 =
      int64_t(p.units_per_seq) * n0 + int64_t(bundle * p.rgroups + rg) * n;
  const int lo = cut.owner(U0), hi = cut.owner(U0 + n - 1);
  if (lo == hi) return;
  RowMerge m;
  m.init();
  const int first_slot = U0 > cut.start(lo) ? 1 : 0;
  for (int c0 = lo; c0 <= hi; c0 += 4) {
    float l[4];
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i;
      if (c <= hi) {
        const int64_t at =
            ((int64_t(c) * 2 + (c == lo ? first_slot : 0)) * p.HB + (h - bundle * p.HB)) * p.rr +
            (r - rg * p.rr);
        l[i] = __ldcg(p.ws_lse + at);
        o[i] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + at * 128) + lane);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c0 + i <= hi) m.add(l[i], o[i]);
  }
  const bool none = m.bad || m.den == 0.f;
  const float inv = none ? 0.f : __frcp_rn(m.den);
  const int64_t row = query_row(p, b, h, r);
  uint2 v = make_uint2(0u, 0u);
  if (!none)
    v = make_uint2(pack_bf16x2(m.o.x * inv, m.o.y * inv), pack_bf16x2(m.o.z * inv, m.o.w * inv));
  reinterpret_cast<uint2*>(p.out + row * 128)[lane] = v;
  if (p.lse && lane == 0)
    p.lse[row] = none ? -CUDART_INF_F : (m.m + log2f(m.den)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------------- host
struct Plan {
  int nt, g, rows, rgroups, rr, HB, S, stages, units_per_seq, ctas;
  size_t smem, off_lse, off_o, bytes;
};

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

size_t smem_bytes(const Plan& pl, int B) {
  const size_t W = size_t(pl.HB) * pl.S;
  size_t n = W * pl.stages * (kTileBytes + 8) + (size_t(B) + 1) * 4;
  if (pl.S > 1) n += W * pl.nt * 8 * (4 + 128 * 4);
  return n;
}

zl_status validate(const zl_decode_attn_q4_params* a) {
  if (!a || a->struct_size != sizeof(*a)) return ZL_ERR_INVALID_ARG;
  if (a->B < 1 || a->Hq < 1 || a->Hkv < 1 || a->q_len < 1 || a->page_size < 1 ||
      a->num_pages < 1 || a->block_table_stride < 1 || a->num_ctas < 0 || a->max_seq_len < 0)
    return ZL_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0) return ZL_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return ZL_ERR_INVALID_ARG;
  if (a->Hq / a->Hkv > 128 || a->q_len > 128 || a->B > kMaxBatch || a->Hkv > 65535 ||
      a->num_ctas > 65535)
    return ZL_ERR_UNSUPPORTED;
  if (a->page_size % kTile || a->page_size > 1024) return ZL_ERR_UNSUPPORTED;
  // (tile sums in 32 bits; the line of tiles times the CTAs in 64)
  if (a->block_table_stride >= (INT64_C(1) << 31)) return ZL_ERR_UNSUPPORTED;
  const int64_t tiles = a->block_table_stride * (a->page_size / kTile) * a->B;
  if (tiles >= (INT64_C(1) << 31) || tiles * a->Hkv >= (INT64_C(1) << 40))
    return ZL_ERR_UNSUPPORTED;
  return ZL_OK;
}

template <int NT>
zl_status occupancy(size_t smem, int threads, int* n) {
  static bool done[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ZL_ERR_CUDA;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(q4_decode_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             226 * 1024) != cudaSuccess)
      return ZL_ERR_CUDA;
    done[dev] = true;
  }
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, q4_decode_kernel<NT>, threads, smem) !=
      cudaSuccess)
    return ZL_ERR_CUDA;
  return *n > 0 ? ZL_OK : ZL_ERR_CUDA;
}

zl_status make_plan(const zl_decode_attn_q4_params* a, Plan* pl) {
  zl_status st = validate(a);
  if (st != ZL_OK) return st;
  int sms;
  if ((st = sm_count(&sms)) != ZL_OK) return st;
  pl->g = a->Hq / a->Hkv;
  pl->rows = pl->g * a->q_len;
  pl->rgroups = (pl->rows + 15) / 16;
  pl->rr = (pl->rows + pl->rgroups - 1) / pl->rgroups;
  pl->rgroups = (pl->rows + pl->rr - 1) / pl->rr;
  pl->nt = pl->rr > 8 ? 2 : 1;
  // heads of a bundle: the most, up to 8, that divide Hkv; one in small calls
  pl->HB = 1;
  const int64_t len = a->max_seq_len > 0 ? a->max_seq_len : 4096;
  const int64_t tiles = int64_t(a->B) * a->Hkv * pl->rgroups * ((len + kTile - 1) / kTile);
  if (tiles >= int64_t(sms) * 64)
    for (int d = 2; d <= 8; ++d)
      if (a->Hkv % d == 0) pl->HB = d;
  pl->S = kMaxWarps / pl->HB;
  pl->units_per_seq = a->Hkv / pl->HB * pl->rgroups;
  // ring: what two CTAs (NT = 2: one) leave an SM, at most 8 stages
  const size_t room = (pl->nt == 1 ? 112 : 200) * 1024;
  pl->stages = 8;
  while (pl->stages > 3 && smem_bytes(*pl, a->B) > room) --pl->stages;
  pl->smem = smem_bytes(*pl, a->B);
  int per_sm = 0;
  const int threads = pl->HB * pl->S * 32;
  st = pl->nt == 1 ? occupancy<1>(pl->smem, threads, &per_sm)
                   : occupancy<2>(pl->smem, threads, &per_sm);
  if (st != ZL_OK) return st;
  pl->ctas = a->num_ctas > 0 ? a->num_ctas : per_sm * sms;
  if (a->num_ctas == 0 && a->max_seq_len > 0) {
    const int64_t most = int64_t(a->B) * pl->units_per_seq * ((len + kTile - 1) / kTile);
    pl->ctas = int(std::max<int64_t>(1, std::min<int64_t>(pl->ctas, most)));
  }
  const size_t slots = size_t(pl->ctas) * 2 * pl->HB * pl->rr;
  pl->off_lse = round_up((size_t(a->B) + 2) * 4, 256);
  pl->off_o = pl->off_lse + round_up(slots * 4, 256);
  pl->bytes = pl->off_o + slots * 128 * 4;
  return ZL_OK;
}

// Maps this thread encoded recently (a decode loop keeps its pool).
struct MapKey {
  const void* pool;
  int64_t page_stride, token_stride, head_stride;
  int32_t page_size, Hkv, num_pages;
  bool operator==(const MapKey& o) const {
    return pool == o.pool && page_stride == o.page_stride && token_stride == o.token_stride &&
           head_stride == o.head_stride && page_size == o.page_size && Hkv == o.Hkv &&
           num_pages == o.num_pages;
  }
};
constexpr int kMapCache = 4;
thread_local MapKey t_keys[kMapCache];
thread_local CUtensorMap t_maps[kMapCache];
thread_local int t_used = 0, t_next = 0;

zl_status encode_pool(const zl_decode_attn_q4_params* a, CUtensorMap* map) {
  const MapKey key{a->pool, a->page_stride, a->token_stride, a->head_stride,
                   a->page_size, a->Hkv, a->num_pages};
  for (int i = 0; i < t_used; ++i)
    if (t_keys[i] == key) {
      *map = t_maps[i];
      return ZL_OK;
    }
  const cuuint64_t dims[4] = {kQ4Row, cuuint64_t(a->page_size), cuuint64_t(a->Hkv),
                              cuuint64_t(a->num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(a->token_stride), cuuint64_t(a->head_stride),
                                 cuuint64_t(a->page_stride)};
  const cuuint32_t box[4] = {kQ4Row, kTile, 1, 1};
  const CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                                  const_cast<void*>(a->pool), dims, strides, box);
  if (r == CUDA_ERROR_NOT_INITIALIZED) return ZL_ERR_CUDA;
  if (r != CUDA_SUCCESS) return ZL_ERR_UNSUPPORTED;
  t_keys[t_next] = key;
  t_maps[t_next] = *map;
  t_next = (t_next + 1) % kMapCache;
  if (t_used < kMapCache) ++t_used;
  return ZL_OK;
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
  if (!a->workspace || !aligned_to(a->workspace, 256) || a->workspace_bytes < pl.bytes)
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
  p.ws_prefix = reinterpret_cast<int32_t*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + pl.off_lse);
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
  p.stages = pl.stages;
  p.units_per_seq = pl.units_per_seq;
  p.rgroups = pl.rgroups;
  p.rr = pl.rr;
  p.rows = pl.rows;
  p.ctas = pl.ctas;
  p.scale_log2 = float(double(a->scale) * kLog2e);

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(pl.ctas));
  cfg.blockDim = dim3(unsigned(pl.HB * pl.S * 32));
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = pl.nt == 1 ? cudaLaunchKernelEx(&cfg, q4_decode_kernel<1>, p)
                             : cudaLaunchKernelEx(&cfg, q4_decode_kernel<2>, p);
  if (e != cudaSuccess) return ZL_ERR_CUDA;
  const int64_t rows = int64_t(a->B) * a->Hkv * pl.rows;
  cfg.gridDim = dim3(unsigned((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, q4_merge_kernel, p);
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
