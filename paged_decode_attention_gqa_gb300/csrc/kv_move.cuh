// What the kernels that move cached rows share: the pools as rows of 16-byte
// chunks, and the host checks of their arguments.
#pragma once

#include "../../include/zl_decode_attn.h"

#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

namespace zl {

// K and V pools; row (page, slot, head) starts at page * page_stride + slot *
// token_stride + head * head_stride, in 16-byte chunks; ck and cv chunks each.
struct MovePools {
  uint4* k;
  uint4* v;  // nullptr for a latent-only pool
  int64_t page_stride, token_stride, head_stride;
  int ck, cv, page_size, num_pages;
  __device__ __forceinline__ int64_t row(int page, int slot, int head) const {
    return int64_t(page) * page_stride + int64_t(slot) * token_stride +
           int64_t(head) * head_stride;
  }
};

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// int32 arrays of na elements at a and nb at b overlap.
inline bool overlaps(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  const intptr_t d = reinterpret_cast<intptr_t>(a) - reinterpret_cast<intptr_t>(b);
  return d < nb * 4 && -d < na * 4;
}

// A caller's parameter struct: of this header's size, or of the size it had
// before the fields after `first_size` bytes came (they are zero then).
template <class Params>
bool take_params(const Params* a, size_t first_size, Params* out) {
  if (!a || (a->struct_size != sizeof(Params) && a->struct_size != first_size)) return false;
  std::memset(out, 0, sizeof(Params));
  std::memcpy(out, a, a->struct_size);
  return true;
}

// The checks and conversion of the pool fields (the same names in every
// parameter struct that moves rows).
template <class Params>
zl_status move_pools(const Params* a, MovePools* out) {
  if (a->B < 1 || a->Hkv < 1 || a->page_size < 1 || a->num_pages < 1 ||
      a->block_table_stride < 1 || a->D_k < 8 || a->D_k > 1024 || a->D_k % 8)
    return ZL_ERR_INVALID_ARG;
  if (!a->k_pool || !a->block_table || !a->seq_lens || !a->new_lens) return ZL_ERR_INVALID_ARG;
  if (a->v_pool && (a->D_v < 8 || a->D_v > 1024 || a->D_v % 8)) return ZL_ERR_INVALID_ARG;
  if (!aligned_to(a->k_pool, 16) || !aligned_to(a->v_pool, 16) ||
      !aligned_to(a->block_table, 4) || !aligned_to(a->seq_lens, 4) ||
      !aligned_to(a->new_lens, 4) || !aligned_to(a->err_flags, 4))
    return ZL_ERR_INVALID_ARG;
  if (a->page_stride <= 0 || a->token_stride <= 0 || a->head_stride <= 0 ||
      a->page_stride % 8 || a->token_stride % 8 || a->head_stride % 8)
    return ZL_ERR_INVALID_ARG;
  if (overlaps(a->new_lens, a->B, a->seq_lens, a->B)) return ZL_ERR_INVALID_ARG;
  if (a->B > 65535 || a->Hkv > 65535) return ZL_ERR_UNSUPPORTED;  // grid dimensions
  out->k = static_cast<uint4*>(a->k_pool);
  out->v = static_cast<uint4*>(a->v_pool);
  out->page_stride = a->page_stride / 8;
  out->token_stride = a->token_stride / 8;
  out->head_stride = a->head_stride / 8;
  out->ck = a->D_k / 8;
  out->cv = a->v_pool ? a->D_v / 8 : 0;
  out->page_size = a->page_size;
  out->num_pages = a->num_pages;
  return ZL_OK;
}

}  // namespace zl
