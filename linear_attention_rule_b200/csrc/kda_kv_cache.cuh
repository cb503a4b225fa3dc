// The paged key-value cache as the kernels see it, and what appending and attending share.
#pragma once

#include <cuda_fp8.h>

#include "kda_launch.cuh"

template <> __device__ __forceinline__ float to_f32<__nv_fp8_e4m3>(__nv_fp8_e4m3 x) { return static_cast<float>(x); }

namespace kda {
namespace kv {

// include/libkda.h kda_kv_cache with the page size as a shift.
struct Cache {
    void *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *seq_lens;
    int64_t page_stride, head_stride, row_stride, table_stride;
    int32_t num_pages, page_shift, max_pages, Hkv;
};

// Element offset of position pos of sequence n and head h; -1 for a position outside the
// block table or a page outside the cache.
__device__ __forceinline__ int64_t row_offset(const Cache& c, int n, int64_t pos, int h) {
    const int64_t pi = pos >> c.page_shift;
    if (pos < 0 || pi >= c.max_pages) return -1;
    const int32_t page = c.table[n * c.table_stride + pi];
    if (page < 0 || page >= c.num_pages) return -1;
    return page * c.page_stride + h * c.head_stride + (pos & ((1 << c.page_shift) - 1)) * c.row_stride;
}

// The new tokens of sequence n; false (and the status) where its entries are inconsistent.
__device__ __forceinline__ bool seq_tokens(const int32_t* cu, int n, int64_t total, int64_t& t0, int64_t& t1) {
    t0 = n;
    t1 = n + 1;
    if (!cu) return true;
    t0 = cu[n];
    t1 = cu[n + 1];
    if (t0 < 0 || t1 < t0 || t1 > total || (n == 0 && t0 != 0)) {
        kda_set_status(KDA_ERR_BAD_SEQLENS);
        return false;
    }
    return true;
}

}  // namespace kv
}  // namespace kda
