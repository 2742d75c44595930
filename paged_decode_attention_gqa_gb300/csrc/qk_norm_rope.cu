// Norm and rotation of queries and keys per head, with the store in the cache
// (zl_qk_norm_rope; formulas in include/zl_decode_attn.h).
//
// Memory-bound: 256 bytes in and 256 (or, into a 4-bit cache, 72) out per head and
// token. 8 lanes take a head: 16 elements each, as two chunks of 8 chosen so that
// both elements of every rotated pair are the lane's own (half-split pairs: chunk l
// and chunk l + n_freq / 8; interleaved or not rotated: chunks 2 l and 2 l + 1), so
// only the sum of squares crosses lanes. A warp takes a token (a part of its heads where
// tokens are few), four heads at a time, queries, then keys, then values: the lane's
// sines and cosines stay in registers, and rows are loaded two rounds ahead, across
// tokens, as the positions are. (16384 tokens of 40 heads: with blocks of 8 tokens that read
// the angles from shared memory for every head, and with rows one round ahead, 66 us; ahead
// within a token only, 61; so 60, 5.6 TB/s. Where a token has 6 heads, 62372 tokens, 79 and
// 50.) Pairs of elements go through packed 32-bit operations. Into a 4-bit pool the rounding
// to codes bounds it: 16384 tokens of 32 + 8 + 8 heads 82 us, 4.3 TB/s, an SM issuing in 71 %
// of all cycles; into bf16 pools 79 us, 5.1 TB/s.
//
// The angle: positions times turns. freq_turns is a frequency in turns, 64 bits
// behind the point, so the product's low 64 bits are the angle without its whole
// turns, right to 2^-33 of a turn at any position below 2^31, where 32-bit radians
// lose every digit. The top 32 bits go to sine and cosine of half-turns.
#include "q4.cuh"
#include "q4_host.h"
#include "ptx.cuh"

#include <cmath>
#include <initializer_list>

namespace zl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxFreq = 64;

struct NormRope {
  const uint4* x[3];    // q, k, v
  uint4* out[2];        // q_out, k_out (k_out may be null)
  int64_t stride[3], out_stride[2];  // per token, in chunks of 8 elements
  const float* weight[2];
  float eps, rope_scale;
  const int32_t* positions;
  int64_t axis_stride;
  uint8_t* pool[2];     // K (or the 4-bit rows), V
  int64_t page_stride, token_stride, head_stride;  // bytes
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  uint32_t* err_flags;
  int64_t tokens;       // B * q_len
  int q_len, Hq, Hkv, page_size, num_pages;
  int n_freq;
  int heads;            // Hq + Hkv (+ Hkv of v)
  int parts, part;      // parts of a token's heads, heads in each (a multiple of 4)
  uint64_t turns[kMaxFreq];
  uint8_t axes[kMaxFreq];
};

// Two bf16 of a word as two 32-bit floats, low half first.
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return pack_f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool INTERLEAVED, int CACHE>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kernel(
    const __grid_constant__ NormRope p) {
  // (no griddep_launch_dependents: blocks that wait beside these cost more than they save,
  // 64 us a prompt of 16384 tokens where this took 61.5, call after call)
  griddep_wait();
  __shared__ __align__(16) float cosine[kWarps][kMaxFreq], sine[kWarps][kMaxFreq];
  // elements 8 c + 4 j .. + 3 at [j][c]: a quarter-warp's reads touch every bank once
  __shared__ __align__(16) float weight[2][2][16][4];
  // (lanes read different ones, which the parameters' memory hands out one by one)
  __shared__ uint64_t turns[kMaxFreq];
  __shared__ int64_t axis_at[kMaxFreq];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 7;
  const int pair_lanes = INTERLEAVED ? 0 : p.n_freq >> 3;  // lanes with half-split pairs
  const bool turned = 8 * l < p.n_freq;
  // chunks of a lane in a row of q or k (one of v: 2 l and 2 l + 1)
  const int qa = l < pair_lanes ? l : 2 * l, qb = l < pair_lanes ? l + pair_lanes : 2 * l + 1;
  const int units = int(p.tokens * p.parts), step = gridDim.x * kWarps;
  // What unit u is: token, heads begin .. end - 1 of it.
  auto unit_at = [&](int u, int& tok, int& begin, int& end) {
    tok = p.parts > 1 ? u / p.parts : u;
    begin = (u - tok * p.parts) * p.part;
    end = min(begin + p.part, p.heads);
  };
  // Row r of a token: a head of q, then of k, then of v.
  auto head_of = [&](int r, int& h) {
    h = r;
    if (h < p.Hq) return 0;
    h -= p.Hq;
    if (CACHE == ZL_CACHE_NONE || h < p.Hkv) return 1;
    h -= p.Hkv;
    return 2;
  };
  // The position that frequency f goes by.
  auto position = [&](int tok, int f) {
    if (f >= p.n_freq) return 0;
    if (p.positions) return p.positions[axis_at[f] + tok];
    const int seq = tok / p.q_len;
    return p.seq_lens[seq] - p.q_len + (tok - seq * p.q_len);
  };
  // Rows are loaded two rounds ahead, those of the next unit too: the round to be loaded is
  // row r_a (of this lane) of unit u_a.
  int u_a = blockIdx.x * kWarps + warp, tok_a = 0, r_a = 0, end_a = 0;
  if (u_a < units) {
    unit_at(u_a, tok_a, r_a, end_a);
    r_a += lane >> 3;
  }
  uint4 a[2], b[2];  // of this round and the next
  auto load = [&](uint4& x, uint4& y) {
    if (u_a >= units) return;
    if (r_a < end_a) {
      int h;
      const int kind = head_of(r_a, h);
      const uint4* src = p.x[kind] + tok_a * p.stride[kind] + h * 16;
      x = src[CACHE != ZL_CACHE_NONE && kind == 2 ? 2 * l : qa];
      y = src[CACHE != ZL_CACHE_NONE && kind == 2 ? 2 * l + 1 : qb];
    }
    r_a += 4;
    if (r_a - (lane >> 3) < end_a) return;
    u_a += step;
    unit_at(u_a, tok_a, r_a, end_a);
    r_a += lane >> 3;
  };
  const int first = tok_a;
  load(a[0], b[0]);
  load(a[1], b[1]);
  for (int e = threadIdx.x; e < 256; e += kThreads) {
    const float* w = p.weight[e >> 7];
    const int d = e & 127;
    weight[e >> 7][(d >> 2) & 1][d >> 3][d & 3] = w ? w[d] : 1.f;
  }
  for (int f = threadIdx.x; f < p.n_freq; f += kThreads) {
    turns[f] = p.turns[f];
    axis_at[f] = p.axes[f] * p.axis_stride;
  }
  __syncthreads();
  int pos[2] = {};  // of this lane's two frequencies, for the unit to come
  if (blockIdx.x * kWarps + warp < units) {
    pos[0] = position(first, lane);
    pos[1] = position(first, lane + 32);
  }

  for (int u = blockIdx.x * kWarps + warp; u < units; u += step) {
    int tok, begin, end;
    unit_at(u, tok, begin, end);
    int r = begin + (lane >> 3);

    // Angles: a lane computes those of two frequencies, and takes its own eight.
    __syncwarp();  // (the last token's have been read)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int f = lane + 32 * e;
      if (f >= p.n_freq) break;
      const uint64_t turn = uint64_t(int64_t(pos[e])) * turns[f] + 0x80000000ull;
      float sn, cs;
      sincospif(float(int32_t(turn >> 32)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
      cosine[warp][f] = cs * p.rope_scale;
      sine[warp][f] = sn * p.rope_scale;
    }
    if (u + step < units) {
      const int next = p.parts > 1 ? (u + step) / p.parts : u + step;
      pos[0] = position(next, lane);
      pos[1] = position(next, lane + 32);
    }
    __syncwarp();
    ulonglong2 co[2] = {}, si[2] = {};
    if (turned) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        co[c] = *reinterpret_cast<const ulonglong2*>(&cosine[warp][8 * l + 4 * c]);
        si[c] = *reinterpret_cast<const ulonglong2*>(&sine[warp][8 * l + 4 * c]);
      }
    }
    int64_t place = -1;  // of the token in the pool, -1: not stored
    if constexpr (CACHE != ZL_CACHE_NONE) {
      const int seq = tok / p.q_len, i = tok - seq * p.q_len;
      const int L = p.seq_lens[seq];
      uint32_t err = 0;
      if (L < p.q_len || int64_t(L) > p.bt_stride * p.page_size) {
        err = ZL_DEVERR_BAD_SEQ_LEN;
      } else {
        const int t = L - p.q_len + i;
        const int page = p.block_table[seq * p.bt_stride + t / p.page_size];
        if (page < 0 || page >= p.num_pages)
          err = ZL_DEVERR_BAD_PAGE;
        else
          place = int64_t(page) * p.page_stride + int64_t(t % p.page_size) * p.token_stride;
      }
      if (err && lane == 0 && begin == 0 && p.err_flags) atomicOr(p.err_flags, err);
    }

    for (; r - (lane >> 3) < end; r += 4) {
      const bool live = r < end;  // (every lane stays for the shuffles)
      int h;
      const int kind = head_of(live ? r : begin, h);
      const bool of_v = CACHE != ZL_CACHE_NONE && kind == 2;
      const bool split = !of_v && l < pair_lanes;
      const int ca = of_v ? 2 * l : qa, cb = of_v ? 2 * l + 1 : qb;
      uint32_t y[2][4] = {{a[0].x, a[0].y, a[0].z, a[0].w}, {b[0].x, b[0].y, b[0].z, b[0].w}};
      a[0] = a[1];
      b[0] = b[1];
      load(a[1], b[1]);
      uint64_t x[2][4], sums = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[c][e] = widen(y[c][e]);
          sums = fma_f32x2(x[c][e], x[c][e], sums);
        }
      const float2 two = unpack_f32x2(sums);
      float ss = two.x + two.y;
      ss += __shfl_xor_sync(0xffffffffu, ss, 1);
      ss += __shfl_xor_sync(0xffffffffu, ss, 2);
      ss += __shfl_xor_sync(0xffffffffu, ss, 4);
      if (!of_v) {  // (a row of v goes as it is)
        if (p.weight[kind]) {
          const float inv = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
          const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const ulonglong2 w =
                  *reinterpret_cast<const ulonglong2*>(weight[kind][j][c ? cb : ca]);
              x[c][2 * j] = mul_f32x2(mul_f32x2(x[c][2 * j], inv2), w.x);
              x[c][2 * j + 1] = mul_f32x2(mul_f32x2(x[c][2 * j + 1], inv2), w.y);
            }
        }
        if (turned) {
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint64_t c2 = e & 2 ? co[e >> 2].y : co[e >> 2].x;
              const uint64_t s2 = e & 2 ? si[e >> 2].y : si[e >> 2].x;
              const float c = e & 1 ? unpack_f32x2(c2).y : unpack_f32x2(c2).x;
              const float s = e & 1 ? unpack_f32x2(s2).y : unpack_f32x2(s2).x;
              const float2 v = unpack_f32x2(x[e >> 2][e & 3]);
              x[e >> 2][e & 3] = pack_f32x2(v.x * c - v.y * s, v.y * c + v.x * s);
            }
          } else {
            const uint64_t minus = pack_f32x2(-1.f, -1.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t c = e & 1 ? co[e >> 1].y : co[e >> 1].x;
              const uint64_t s = e & 1 ? si[e >> 1].y : si[e >> 1].x;
              const uint64_t m = x[0][e], v = x[1][e];
              x[0][e] = fma_f32x2(mul_f32x2(v, s), minus, mul_f32x2(m, c));
              x[1][e] = fma_f32x2(m, s, mul_f32x2(v, c));
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack_f32x2(x[c][e]);
            y[c][e] = pack_bf16x2(v.x, v.y);
          }
        uint4* to = p.out[kind];
        if (live && (CACHE == ZL_CACHE_NONE || to)) {
          to += tok * p.out_stride[kind] + h * 16;
          to[ca] = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
          to[cb] = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
        }
      }
      if constexpr (CACHE != ZL_CACHE_NONE) {
        const bool store = live && kind > 0 && place >= 0;
        const int64_t row = place + int64_t(h) * p.head_stride;
        if constexpr (CACHE == ZL_CACHE_BF16) {
          if (store) {
            uint4* to = reinterpret_cast<uint4*>(p.pool[kind - 1] + row);
            to[ca] = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
            to[cb] = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
          }
        } else {
          // A scale's 16 elements are chunks 2 m and 2 m + 1: the lane's own two, or
          // (half-split pairs; an even number of such lanes) one of its own and one of
          // the next lane's.
          uint32_t ma = q4_amax8(y[0]), mb = q4_amax8(y[1]);
          const uint32_t oa = __shfl_xor_sync(0xffffffffu, ma, 1);
          const uint32_t ob = __shfl_xor_sync(0xffffffffu, mb, 1);
          ma = max(ma, split ? oa : mb);
          mb = split ? max(mb, ob) : ma;
          if (store) {
            const Q4Scale sa = q4_scale(ma), sb = q4_scale(mb);
            uint8_t* to = p.pool[0] + row;
            const int kv = kind - 1;
            uint32_t* codes = reinterpret_cast<uint32_t*>(to + kv * kQ4VCodes);
            codes[ca] = q4_codes(y[0], sa);
            codes[cb] = q4_codes(y[1], sb);
            if (!(ca & 1)) {
              to[kQ4KScales + 8 * kv + (ca >> 1)] = uint8_t(sa.byte);
              if (split) to[kQ4KScales + 8 * kv + (cb >> 1)] = uint8_t(sb.byte);
            }
          }
        }
      }
    }
  }
}

// Rows of `width` bytes every `stride` bytes, T of them.
struct RowSet {
  const void* base;
  int64_t stride, width;
};

// Whether a row of a and a row of b share a byte. Sets of different strides count
// as apart only where their whole ranges are.
bool rows_meet(const RowSet& a, const RowSet& b, int64_t T) {
  const intptr_t x = reinterpret_cast<intptr_t>(a.base), y = reinterpret_cast<intptr_t>(b.base);
  const int64_t span_a = (T - 1) * a.stride + a.width, span_b = (T - 1) * b.stride + b.width;
  if (x + span_a <= y || y + span_b <= x) return false;
  if (T == 1 || a.stride != b.stride) return true;
  int64_t d = (y - x) % a.stride;  // where a row of b begins behind one of a
  if (d < 0) d += a.stride;
  return d < a.width || a.stride - d < b.width;
}

zl_status validate(const zl_qk_norm_rope_params* a) {
  if (!a || a->struct_size != sizeof(*a)) return ZL_ERR_INVALID_ARG;
  if (a->B < 1 || a->q_len < 1 || a->Hq < 1 || a->Hkv < 1) return ZL_ERR_INVALID_ARG;
  if (a->cache < ZL_CACHE_NONE || a->cache > ZL_CACHE_Q4) return ZL_ERR_INVALID_ARG;
  const bool cached = a->cache != ZL_CACHE_NONE;
  if (!a->q || !a->k || !a->q_out || (!cached && !a->k_out)) return ZL_ERR_INVALID_ARG;
  for (const void* x : {a->q, a->k, a->v, static_cast<const void*>(a->q_out),
                        static_cast<const void*>(a->k_out),
                        static_cast<const void*>(a->q_weight),
                        static_cast<const void*>(a->k_weight)})
    if (!aligned_to(x, 16)) return ZL_ERR_INVALID_ARG;
  if (!aligned_to(a->positions, 4) || !aligned_to(a->err_flags, 4) ||
      !aligned_to(a->block_table, 4) || !aligned_to(a->seq_lens, 4))
    return ZL_ERR_INVALID_ARG;
  const int64_t wq = int64_t(a->Hq) * 128, wk = int64_t(a->Hkv) * 128;
  if (a->q_stride % 8 || a->k_stride % 8 || a->q_out_stride % 8 || a->q_stride < wq ||
      a->k_stride < wk || a->q_out_stride < wq)
    return ZL_ERR_INVALID_ARG;
  if (a->k_out && (a->k_out_stride % 8 || a->k_out_stride < wk)) return ZL_ERR_INVALID_ARG;
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps) || !std::isfinite(a->rope_scale))
    return ZL_ERR_INVALID_ARG;
  if (a->n_freq < 0 || a->n_axes < 1 || (a->n_freq > 0 && !a->freq_turns))
    return ZL_ERR_INVALID_ARG;
  if (a->n_freq % 16 || a->n_freq > kMaxFreq || a->n_axes > 4 || a->Hq > 65535 || a->Hkv > 65535)
    return ZL_ERR_UNSUPPORTED;
  if (a->axes)
    for (int i = 0; i < a->n_freq; ++i)
      if (a->axes[i] >= a->n_axes) return ZL_ERR_INVALID_ARG;
  const int64_t T = int64_t(a->B) * a->q_len;
  if (T > (1 << 30)) return ZL_ERR_UNSUPPORTED;  // (a terabyte of queries is more than fits)
  if (a->positions ? (a->n_axes > 1 && a->axis_stride < T) : !a->seq_lens && a->n_freq > 0)
    return ZL_ERR_INVALID_ARG;
  if (cached) {
    if (!a->v || a->v_stride % 8 || a->v_stride < wk) return ZL_ERR_INVALID_ARG;
    if (!a->k_pool || !a->block_table || !a->seq_lens || a->page_size < 1 || a->num_pages < 1 ||
        a->block_table_stride < 1)
      return ZL_ERR_INVALID_ARG;
    if ((a->cache == ZL_CACHE_BF16) != (a->v_pool != nullptr)) return ZL_ERR_INVALID_ARG;
    if (!aligned_to(a->k_pool, 16) || !aligned_to(a->v_pool, 16)) return ZL_ERR_INVALID_ARG;
    const int64_t unit = a->cache == ZL_CACHE_Q4 ? 16 : 8;
    if (a->page_stride <= 0 || a->token_stride <= 0 || a->head_stride <= 0 ||
        a->page_stride % unit || a->token_stride % unit || a->head_stride % unit)
      return ZL_ERR_INVALID_ARG;
  }
  // What is written meets nothing that is read, but for a row written over itself.
  const RowSet q{a->q, a->q_stride * 2, wq * 2}, k{a->k, a->k_stride * 2, wk * 2},
      qo{a->q_out, a->q_out_stride * 2, wq * 2}, ko{a->k_out, a->k_out_stride * 2, wk * 2},
      v{a->v, a->v_stride * 2, wk * 2};
  const bool q_in_place = a->q_out == a->q && a->q_out_stride == a->q_stride;
  const bool k_in_place = a->k_out == a->k && a->k_out_stride == a->k_stride;
  if ((!q_in_place && rows_meet(qo, q, T)) || rows_meet(qo, k, T) ||
      (cached && rows_meet(qo, v, T)))
    return ZL_ERR_INVALID_ARG;
  if (a->k_out && ((!k_in_place && rows_meet(ko, k, T)) || rows_meet(ko, q, T) ||
                   rows_meet(ko, qo, T) || (cached && rows_meet(ko, v, T))))
    return ZL_ERR_INVALID_ARG;
  return ZL_OK;
}

}  // namespace
}  // namespace zl

extern "C" zl_status zl_qk_norm_rope(const zl_qk_norm_rope_params* a, zl_stream_t stream) {
  using namespace zl;
  zl_status st = validate(a);
  if (st != ZL_OK) return st;
  int sms;
  if ((st = sm_count(&sms)) != ZL_OK) return st;
  const bool cached = a->cache != ZL_CACHE_NONE;
  NormRope p;
  std::memset(&p, 0, sizeof(p));
  p.x[0] = static_cast<const uint4*>(a->q);
  p.x[1] = static_cast<const uint4*>(a->k);
  p.x[2] = cached ? static_cast<const uint4*>(a->v) : nullptr;
  p.out[0] = static_cast<uint4*>(a->q_out);
  p.out[1] = static_cast<uint4*>(a->k_out);
  p.stride[0] = a->q_stride / 8;
  p.stride[1] = a->k_stride / 8;
  p.stride[2] = a->v_stride / 8;
  p.out_stride[0] = a->q_out_stride / 8;
  p.out_stride[1] = a->k_out_stride / 8;
  p.weight[0] = a->q_weight;
  p.weight[1] = a->k_weight;
  p.eps = a->eps;
  p.rope_scale = a->rope_scale;
  p.positions = a->positions;
  p.axis_stride = a->axis_stride;
  if (cached) {
    const int64_t bytes = a->cache == ZL_CACHE_Q4 ? 1 : 2;
    p.pool[0] = static_cast<uint8_t*>(a->k_pool);
    p.pool[1] = static_cast<uint8_t*>(a->v_pool);
    p.page_stride = a->page_stride * bytes;
    p.token_stride = a->token_stride * bytes;
    p.head_stride = a->head_stride * bytes;
    p.block_table = a->block_table;
    p.bt_stride = a->block_table_stride;
    p.page_size = a->page_size;
    p.num_pages = a->num_pages;
  }
  p.seq_lens = a->seq_lens;
  p.err_flags = a->err_flags;
  p.tokens = int64_t(a->B) * a->q_len;
  p.q_len = a->q_len;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.n_freq = a->n_freq;
  for (int i = 0; i < a->n_freq; ++i) {
    p.turns[i] = a->freq_turns[i];
    p.axes[i] = a->axes ? a->axes[i] : 0;
  }
  p.heads = a->Hq + a->Hkv + (cached ? a->Hkv : 0);
  // A warp to a token, or to a part of its heads (a multiple of 4) where that leaves SMs
  // with fewer than 8 warps.
  const int fours = (p.heads + 3) / 4;
  p.parts = int(std::max<int64_t>(1, std::min<int64_t>(fours, 8 * sms / p.tokens)));
  p.part = (fours + p.parts - 1) / p.parts * 4;
  p.parts = (p.heads + p.part - 1) / p.part;
  // three blocks are resident on an SM; with more units than warps these take several
  const int64_t blocks = (p.tokens * p.parts + kWarps - 1) / kWarps;
  const unsigned grid = unsigned(std::min<int64_t>(blocks, 3 * sms));
  auto launch = [&](auto kernel) { return launch_after(kernel, dim3(grid), kThreads, stream, p); };
  switch (a->cache * 2 + (a->interleaved ? 1 : 0)) {
    case 0: return launch(qk_norm_rope_kernel<false, ZL_CACHE_NONE>);
    case 1: return launch(qk_norm_rope_kernel<true, ZL_CACHE_NONE>);
    case 2: return launch(qk_norm_rope_kernel<false, ZL_CACHE_BF16>);
    case 3: return launch(qk_norm_rope_kernel<true, ZL_CACHE_BF16>);
    case 4: return launch(qk_norm_rope_kernel<false, ZL_CACHE_Q4>);
    default: return launch(qk_norm_rope_kernel<true, ZL_CACHE_Q4>);
  }
}
