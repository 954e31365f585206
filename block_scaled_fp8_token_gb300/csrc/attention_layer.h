// attention_layer.h -- host-side declarations of the attention layer: the paged KV cache,
// attention over it and the residual stream between blocks.
#pragma once

#include "bfp8_internal.h"

namespace bfp8 {

// As make_tmap_3d, with one dimension more.
int make_tmap_4d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t dim0,
                 uint64_t dim1, uint64_t dim2, uint64_t dim3, uint64_t stride1_bytes,
                 uint64_t stride2_bytes, uint64_t stride3_bytes, uint32_t box0, uint32_t box1,
                 uint32_t box2, uint32_t box3, CUtensorMapSwizzle swizzle);

int launch_kv_plan(const int32_t* ctx, const int32_t* q_len, int64_t B, const int32_t* free_pages,
                   int64_t n_free, int32_t* table, int64_t ld_table, int64_t max_blocks,
                   int32_t page_size, int32_t* q_offsets, int32_t* kv_len, int64_t* slots,
                   int32_t* positions, int64_t T, int32_t* counts, void* stream);
int launch_kv_append(const void* k, int64_t k_ldt, int64_t k_ldh, const void* v, int64_t v_ldt,
                     int64_t v_ldh, const int64_t* slots, int64_t T, const bfp8_kv_cache& cache,
                     void* stream);
size_t kv_attention_workspace_bytes(int64_t B, int64_t T, int64_t max_q, int64_t Hq, int sms);
int launch_kv_attention(const bfp8_kv_attention_args& args, const bfp8_kv_cache& cache,
                        void* stream);
int launch_residual_norm(const bfp8_norm_args& args, int64_t T, int64_t H, void* stream);

// The device error word of the attention kernels, as those of the projections.
int kv_read_clear_error();

}  // namespace bfp8
