// Writing the 4-bit cache (zl_kv_append_q4) and reading it back (zl_kv_read_q4).
// The row and its roundings are described in include/zl_decode_attn.h.
//
// Both move bytes: per token and kv head 512 bytes of bf16 on one side, 144 on the
// other. A quarter-warp of 8 lanes takes a K or a V row, each lane one block of 16
// elements (32 bytes of bf16, 8 of codes, a scale byte), so that no block is shared
// between lanes and a row's 64 bytes of codes go out side by side. HBM bounds both: 8
// chunks of 512 tokens of 8 heads appended and 2048-8192 tokens read back 43 us for 254 MB,
// 5.9 TB/s where a copy reaches 6.8; 4 prompts of up to 16384 tokens written and read
// 99 us, 6.2 TB/s. (Two rows at a time per thread took 115 where one took 105; divisions
// that the device works out 104.)
#include "q4.cuh"
#include "q4_host.h"
#include "ptx.cuh"

namespace zl {
namespace {

struct AppendQ4 {
  const uint4* k_new;
  const uint4* v_new;
  int64_t k_stride, v_stride;  // per token, in 16-byte chunks
  uint8_t* pool;
  int64_t page_stride, token_stride, head_stride;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  uint32_t* err_flags;
  int q_len, Hkv, page_size, num_pages;
  bool wide;  // rows on 32-byte boundaries
  Divisor heads, page;
};

// Blocks (x, b): the rows (token, head) of sequence b, two to a warp.
__global__ void __launch_bounds__(256) append_q4_kernel(const __grid_constant__ AppendQ4 p) {
  // (what follows waits for this grid before it touches memory, as this grid does here)
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, kv = (lane >> 3) & 1, j = lane & 7;
  const int b = blockIdx.y;
  const int L = p.seq_lens[b];
  const int n = p.new_lens ? p.new_lens[b] : p.q_len;
  if (n < 0 || n > p.q_len || L < n || int64_t(L) > p.bt_stride * p.page_size) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.err_flags)
      atomicOr(p.err_flags, ZL_DEVERR_BAD_SEQ_LEN);
    return;
  }
  const uint32_t rows = uint32_t(n) * uint32_t(p.Hkv);  // (below 2^31: checked on the host)
  const uint4* src = kv ? p.v_new : p.k_new;
  const int64_t stride = kv ? p.v_stride : p.k_stride;
  const uint32_t step = gridDim.x * (blockDim.x >> 4);
  for (uint32_t r = blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4); r < rows; r += step) {
    const uint32_t i = p.heads.quotient(r), h = r - i * uint32_t(p.Hkv);
    const int t = L - n + int(i);
    const uint32_t pg = p.page.quotient(uint32_t(t));
    const int page = p.block_table[b * p.bt_stride + pg];
    const uint4* at = src + (int64_t(b) * p.q_len + i) * stride + int64_t(h) * 16 + 2 * j;
    uint32_t x[2][4];
    if (p.wide) {
      ld_global_v8(at, x[0], x[1]);
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 v = at[c];
        x[c][0] = v.x, x[c][1] = v.y, x[c][2] = v.z, x[c][3] = v.w;
      }
    }
    if (page < 0 || page >= p.num_pages) {
      if (h == 0 && (lane & 15) == 0 && p.err_flags) atomicOr(p.err_flags, ZL_DEVERR_BAD_PAGE);
      continue;
    }
    const Q4Scale s = q4_scale(max(q4_amax8(x[0]), q4_amax8(x[1])));
    uint8_t* row = p.pool + int64_t(page) * p.page_stride +
                   int64_t(t - int(pg) * p.page_size) * p.token_stride +
                   int64_t(h) * p.head_stride;
    *reinterpret_cast<uint2*>(row + kv * kQ4VCodes + 8 * j) =
        make_uint2(q4_codes(x[0], s), q4_codes(x[1], s));
    row[kQ4KScales + 8 * kv + j] = uint8_t(s.byte);
  }
}

struct ReadQ4 {
  const uint8_t* pool;
  int64_t page_stride, token_stride, head_stride;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  uint32_t* err_flags;
  int tokens, Hkv, page_size, num_pages;
  Divisor heads, page;
};

__global__ void __launch_bounds__(256) read_q4_kernel(const __grid_constant__ ReadQ4 p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, kv = (lane >> 3) & 1, j = lane & 7;
  const int b = blockIdx.y;
  const int L = p.seq_lens[b];
  if (L < 0 || L > p.tokens || int64_t(L) > p.bt_stride * p.page_size) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.err_flags)
      atomicOr(p.err_flags, ZL_DEVERR_BAD_SEQ_LEN);
    return;
  }
  const uint32_t rows = uint32_t(L) * uint32_t(p.Hkv);
  __nv_bfloat16* out = kv ? p.v_out : p.k_out;
  const uint32_t step = gridDim.x * (blockDim.x >> 4);
  for (uint32_t r = blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4); r < rows; r += step) {
    const uint32_t t = p.heads.quotient(r), h = r - t * uint32_t(p.Hkv);
    const uint32_t pg = p.page.quotient(t);
    const int page = p.block_table[b * p.bt_stride + pg];
    if (page < 0 || page >= p.num_pages) {
      if (h == 0 && (lane & 15) == 0 && p.err_flags) atomicOr(p.err_flags, ZL_DEVERR_BAD_PAGE);
      continue;
    }
    if (!out) continue;
    const uint8_t* row = p.pool + int64_t(page) * p.page_stride +
                         int64_t(t - pg * uint32_t(p.page_size)) * p.token_stride +
                         int64_t(h) * p.head_stride;
    const uint2 w = *reinterpret_cast<const uint2*>(row + kv * kQ4VCodes + 8 * j);
    const uint32_t sb = row[kQ4KScales + 8 * kv + j];
    const float s = __half2float(__ushort_as_half(uint16_t(sb << 7)));
    uint32_t y[8];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t f[4];
      q4_pairs(c ? w.y : w.x, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f[i]));
        y[4 * c + i] = pack_bf16x2(v.x * s, v.y * s);
      }
    }
    __nv_bfloat16* to = out + ((int64_t(b) * p.tokens + t) * p.Hkv + h) * 128 + 16 * j;
    st_global_v8(to, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
  }
}

// Blocks over the rows (token, head) of B sequences, 16 to a block; with more than
// fill the device a few times over, each block takes several.
dim3 row_grid(int64_t rows, int B, int sms) {
  const int64_t blocks = (rows + 15) / 16;
  const int64_t most = std::max<int64_t>(1, int64_t(sms) * 32 / B);
  return dim3(unsigned(std::min(blocks, most)), unsigned(B));
}

}  // namespace
}  // namespace zl

extern "C" zl_status zl_kv_append_q4(const zl_kv_append_q4_params* a, zl_stream_t stream) {
  using namespace zl;
  if (!a || a->struct_size != sizeof(*a)) return ZL_ERR_INVALID_ARG;
  zl_status st = q4_check_pool(a);
  if (st != ZL_OK) return st;
  if (a->q_len < 1 || !a->k_new || !a->v_new || !aligned_to(a->k_new, 16) ||
      !aligned_to(a->v_new, 16) || !aligned_to(a->new_lens, 4))
    return ZL_ERR_INVALID_ARG;
  if (a->k_stride % 8 || a->v_stride % 8 || a->k_stride < int64_t(a->Hkv) * 128 ||
      a->v_stride < int64_t(a->Hkv) * 128)
    return ZL_ERR_INVALID_ARG;
  if (a->B > 65535 || int64_t(a->q_len) * a->Hkv > INT32_MAX - (1 << 20)) return ZL_ERR_UNSUPPORTED;
  int sms;
  if ((st = sm_count(&sms)) != ZL_OK) return st;
  AppendQ4 p;
  p.k_new = static_cast<const uint4*>(a->k_new);
  p.v_new = static_cast<const uint4*>(a->v_new);
  p.k_stride = a->k_stride / 8;
  p.v_stride = a->v_stride / 8;
  p.pool = static_cast<uint8_t*>(a->pool);
  p.page_stride = a->page_stride;
  p.token_stride = a->token_stride;
  p.head_stride = a->head_stride;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.seq_lens = a->seq_lens;
  p.new_lens = a->new_lens;
  p.err_flags = a->err_flags;
  p.q_len = a->q_len;
  p.Hkv = a->Hkv;
  p.page_size = a->page_size;
  p.num_pages = a->num_pages;
  p.heads = Divisor(uint32_t(a->Hkv));
  p.page = Divisor(uint32_t(a->page_size));
  p.wide = aligned_to(a->k_new, 32) && aligned_to(a->v_new, 32) && a->k_stride % 16 == 0 &&
           a->v_stride % 16 == 0;
  return launch_after(append_q4_kernel, row_grid(int64_t(a->q_len) * a->Hkv, a->B, sms), 256,
                      stream, p);
}

extern "C" zl_status zl_kv_read_q4(const zl_kv_read_q4_params* a, zl_stream_t stream) {
  using namespace zl;
  if (!a || a->struct_size != sizeof(*a)) return ZL_ERR_INVALID_ARG;
  zl_status st = q4_check_pool(a);
  if (st != ZL_OK) return st;
  if (a->tokens < 1 || (!a->k_out && !a->v_out) || !aligned_to(a->k_out, 32) ||
      !aligned_to(a->v_out, 32))
    return ZL_ERR_INVALID_ARG;
  if (a->B > 65535 || int64_t(a->tokens) * a->Hkv > INT32_MAX - (1 << 20))
    return ZL_ERR_UNSUPPORTED;
  int sms;
  if ((st = sm_count(&sms)) != ZL_OK) return st;
  ReadQ4 p;
  p.pool = static_cast<const uint8_t*>(a->pool);
  p.page_stride = a->page_stride;
  p.token_stride = a->token_stride;
  p.head_stride = a->head_stride;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.seq_lens = a->seq_lens;
  p.k_out = static_cast<__nv_bfloat16*>(a->k_out);
  p.v_out = static_cast<__nv_bfloat16*>(a->v_out);
  p.err_flags = a->err_flags;
  p.tokens = a->tokens;
  p.Hkv = a->Hkv;
  p.page_size = a->page_size;
  p.num_pages = a->num_pages;
  p.heads = Divisor(uint32_t(a->Hkv));
  p.page = Divisor(uint32_t(a->page_size));
  return launch_after(read_q4_kernel, row_grid(int64_t(a->tokens) * a->Hkv, a->B, sms), 256,
                      stream, p);
}
