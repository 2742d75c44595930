// Host checks and queries that the entry points over the 4-bit cache share.
#pragma once

#include "kernels.h"
#include "kv_move.cuh"

#include <algorithm>

namespace zl {

// SMs of the current device (api.cu).
zl_status sm_count(int* sms);
// cuTensorMapEncodeTiled without swizzle or element strides (api.cu).
CUresult encode_tiled(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, void* base,
                      const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box);

// The pool and table fields (the same names in every parameter struct).
template <class Params>
zl_status q4_check_pool(const Params* a) {
  if (a->B < 1 || a->Hkv < 1 || a->page_size < 1 || a->num_pages < 1 || a->block_table_stride < 1)
    return ZL_ERR_INVALID_ARG;
  if (!a->pool || !a->block_table || !a->seq_lens) return ZL_ERR_INVALID_ARG;
  if (!aligned_to(a->pool, 16) || !aligned_to(a->block_table, 4) || !aligned_to(a->seq_lens, 4) ||
      !aligned_to(a->err_flags, 4))
    return ZL_ERR_INVALID_ARG;
  if (a->page_stride <= 0 || a->token_stride <= 0 || a->head_stride <= 0 ||
      a->page_stride % 16 || a->token_stride % 16 || a->head_stride % 16)
    return ZL_ERR_INVALID_ARG;
  return ZL_OK;
}

// Launches a kernel that begins with griddep_wait: its blocks may be placed while what
// comes before it in the stream ends. (Append and read-back of 8 chunks of 512 tokens, call
// after call: 49.4 us launched in the ordinary way, 44.4 so.)
template <class Params>
zl_status launch_after(void (*kernel)(Params), dim3 grid, int threads, zl_stream_t stream,
                       const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

}  // namespace zl
