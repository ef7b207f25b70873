// attn_host.h -- host side shared by the two paged-attention translation units.
#pragma once
#include <algorithm>

#include "attn_common.cuh"
#include "qmv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace attn {

// Tensor map of a cache as rows of D values, in boxes of 64 values by a page's
// rows (a key tile's where pages are longer).
inline sv_status encode_cache(CUtensorMap *map, const void *cache, int D, const Args &a,
                              int tile_keys) {
  return qmv::encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cache, (uint64_t)D,
                        ((uint64_t)a.num_pages * a.Hkv) << a.page_shift, (uint64_t)D * 2, 64,
                        (uint32_t)std::min(1 << a.page_shift, tile_keys),
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

// paged_attn_tc.cu: the tensor-core kernel for many rows (D 64 or 128)
size_t tc_partial_bytes(int D);
unsigned tc_take_give_up();
sv_status tc_run(int D, const Args &a, cudaStream_t stream);
// paged_attn_tc256.cu: the same for D 256
size_t tc256_partial_bytes();
unsigned tc256_take_give_up();
sv_status tc256_run(const Args &a, cudaStream_t stream);

}  // namespace attn
}  // namespace sv
