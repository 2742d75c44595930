// Norm and rotation of queries and keys per head, with the store in the cache
// (zl_qk_norm_rope; formulas in include/zl_decode_attn.h).
//
// Memory-bound: 256 bytes in and 256 (or, into a 4-bit cache, 72) out per head and
// token. 8 lanes take a head: 16 elements each, as two chunks of 8 chosen so that
// both elements of every rotated pair are the lane's own (half-split pairs: chunk l
// and chunk l + n_freq / 8; interleaved or not rotated: chunks 2 l and 2 l + 1), so
// only the sum of squares crosses lanes. A block takes a few tokens; the sines and
// cosines of each are computed once for all its heads.
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

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 8;  // heads a block works on at once
constexpr int kMaxTokens = 8;        // tokens of a block
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
  int cache, n_freq, interleaved;
  int tokens_per_block, heads, heads_per_block;  // heads: Hq + Hkv (+ Hkv of v)
  uint64_t turns[kMaxFreq];
  uint8_t axes[kMaxFreq];
};

__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(
    const __grid_constant__ NormRope p) {
  griddep_launch_dependents();
  __shared__ __align__(16) float cosine[kMaxTokens][kMaxFreq], sine[kMaxTokens][kMaxFreq];
  __shared__ __align__(16) float weight[2][128];
  __shared__ int64_t place[kMaxTokens];  // of the token's row in the pool, -1: not stored
  const int64_t tok0 = int64_t(blockIdx.x) * p.tokens_per_block;
  const int ntok = int(min(int64_t(p.tokens_per_block), p.tokens - tok0));

  for (int e = threadIdx.x; e < ntok * p.n_freq; e += kThreads) {
    const int tt = e / p.n_freq, f = e - tt * p.n_freq;
    const int64_t tok = tok0 + tt;
    int pos;
    if (p.positions) {
      pos = __ldg(p.positions + p.axes[f] * p.axis_stride + tok);
    } else {
      const int64_t b = tok / p.q_len;
      pos = __ldg(p.seq_lens + b) - p.q_len + int(tok - b * p.q_len);
    }
    const uint64_t turn = uint64_t(int64_t(pos)) * p.turns[f] + 0x80000000ull;
    float s, c;
    sincospif(float(int32_t(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cosine[tt][f] = c * p.rope_scale;
    sine[tt][f] = s * p.rope_scale;
  }
  for (int e = threadIdx.x; e < 256; e += kThreads) {
    const float* w = p.weight[e >> 7];
    weight[e >> 7][e & 127] = w ? __ldg(w + (e & 127)) : 1.f;
  }
  if (p.cache != ZL_CACHE_NONE && int(threadIdx.x) < ntok) {
    const int64_t tok = tok0 + threadIdx.x, b = tok / p.q_len;
    const int i = int(tok - b * p.q_len), L = __ldg(p.seq_lens + b);
    int64_t at = -1;
    uint32_t err = 0;
    if (L < p.q_len || int64_t(L) > p.bt_stride * p.page_size) {
      err = ZL_DEVERR_BAD_SEQ_LEN;
    } else {
      const int t = L - p.q_len + i;
      const int page = __ldg(p.block_table + b * p.bt_stride + t / p.page_size);
      if (page < 0 || page >= p.num_pages)
        err = ZL_DEVERR_BAD_PAGE;
      else
        at = int64_t(page) * p.page_stride + int64_t(t % p.page_size) * p.token_stride;
    }
    if (err && blockIdx.y == 0 && p.err_flags) atomicOr(p.err_flags, err);
    place[threadIdx.x] = at;
  }
  __syncthreads();

  const int l = threadIdx.x & 7;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int nh = min(p.heads_per_block, p.heads - h0);
  const int total = ntok * nh;
  const int pair_lanes = p.interleaved ? 0 : p.n_freq >> 3;  // lanes with half-split pairs
  for (int r0 = 0; r0 < total; r0 += kRows) {
    const int r = r0 + int(threadIdx.x >> 3);
    const bool live = r < total;  // (every lane stays for the shuffles)
    const int tt = live ? r / nh : 0;
    int h = live ? h0 + r - tt * nh : 0;
    const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
    h -= kind == 0 ? 0 : kind == 1 ? p.Hq : p.Hq + p.Hkv;
    const int64_t tok = tok0 + tt;
    const bool split = kind < 2 && l < pair_lanes;
    const int ca = split ? l : 2 * l, cb = split ? l + pair_lanes : 2 * l + 1;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (live) {
      const uint4* src = p.x[kind] + tok * p.stride[kind] + int64_t(h) * 16;
      a = src[ca];
      b = src[cb];
    }
    uint32_t y[2][4] = {{a.x, a.y, a.z, a.w}, {b.x, b.y, b.z, b.w}};
    float x[2][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_bf16x2(y[c][i]);
        x[c][2 * i] = v.x;
        x[c][2 * i + 1] = v.y;
        ss = fmaf(v.x, v.x, ss);
        ss = fmaf(v.y, v.y, ss);
      }
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    ss += __shfl_xor_sync(0xffffffffu, ss, 4);
    if (kind < 2) {  // (a row of v goes as it is)
      if (p.weight[kind]) {
        const float inv = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
        const float* wa = &weight[kind][8 * ca];
        const float* wb = &weight[kind][8 * cb];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[0][i] = x[0][i] * inv * wa[i];
          x[1][i] = x[1][i] * inv * wb[i];
        }
      }
      if (8 * l < p.n_freq) {
        const float* co = &cosine[tt][8 * l];
        const float* si = &sine[tt][8 * l];
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& u = x[i >> 2][2 * (i & 3)];
            float& v = x[i >> 2][2 * (i & 3) + 1];
            const float u0 = u, v0 = v;
            u = u0 * co[i] - v0 * si[i];
            v = v0 * co[i] + u0 * si[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float u = x[0][i], v = x[1][i];
            x[0][i] = u * co[i] - v * si[i];
            x[1][i] = v * co[i] + u * si[i];
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[c][i] = pack_bf16x2(x[c][2 * i], x[c][2 * i + 1]);
      uint4* to = p.out[kind];
      if (live && to) {
        to += tok * p.out_stride[kind] + int64_t(h) * 16;
        to[ca] = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
        to[cb] = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
      }
    }
    if (p.cache == ZL_CACHE_NONE) continue;
    const int64_t at = place[tt];
    const bool store = live && kind > 0 && at >= 0;
    const int64_t row = at + int64_t(h) * p.head_stride;
    if (p.cache == ZL_CACHE_BF16) {
      if (store) {
        uint4* to = reinterpret_cast<uint4*>(p.pool[kind - 1] + row);
        to[ca] = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
        to[cb] = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
      }
      continue;
    }
    // A scale's 16 elements are chunks 2 m and 2 m + 1: the lane's own two, or
    // (half-split pairs; an even number of such lanes) one of its own and one of
    // the next lane's.
    uint32_t ma = q4_amax8(y[0]), mb = q4_amax8(y[1]);
    const uint32_t oa = __shfl_xor_sync(0xffffffffu, ma, 1), ob = __shfl_xor_sync(0xffffffffu, mb, 1);
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
  p.cache = a->cache;
  p.n_freq = a->n_freq;
  p.interleaved = a->interleaved ? 1 : 0;
  for (int i = 0; i < a->n_freq; ++i) {
    p.turns[i] = a->freq_turns[i];
    p.axes[i] = a->axes ? a->axes[i] : 0;
  }
  p.heads = a->Hq + a->Hkv + (cached ? a->Hkv : 0);
  // Tokens per block: 8 where that leaves four blocks to an SM, fewer otherwise;
  // with few tokens a block takes 32 heads of one.
  int tpb = kMaxTokens;
  while (tpb > 1 && p.tokens < int64_t(tpb) * 4 * sms) tpb /= 2;
  p.tokens_per_block = tpb;
  p.heads_per_block = p.tokens < 2 * sms ? std::min(p.heads, kRows) : p.heads;
  const int64_t bx = (p.tokens + tpb - 1) / tpb;
  const int by = (p.heads + p.heads_per_block - 1) / p.heads_per_block;
  if (bx > INT32_MAX || by > 65535) return ZL_ERR_UNSUPPORTED;
  qk_norm_rope_kernel<<<dim3(unsigned(bx), unsigned(by)), kThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
