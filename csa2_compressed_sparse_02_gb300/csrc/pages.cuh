// What the paged-cache calls share: the cache as kernels see it, and its host checks.
#pragma once

#include "common.cuh"

namespace csa2 {

struct Pages {
    uint8_t* pool;
    int64_t layer_bytes;
    int32_t* table;
    int32_t* ref;
    int layers, n_pages, page_size, max_seqs, max_pages;
    int row_bytes;
    __host__ __device__ int64_t page_bytes() const { return (int64_t)page_size * row_bytes; }
    __host__ __device__ int64_t max_len() const { return (int64_t)max_pages * page_size; }
};

// Checks params and cache for the call `name` and fills *out; CSA2_OK or the error.
int check_pages(const char* name, const csa2_params* p, const csa2_pages* c, Pages* out);

}  // namespace csa2
