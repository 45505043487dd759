// The paged key-value cache as the kernels see it: byte strides, and the division
// of a slot by the page size as one multiplication.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace q4k {

struct KvView {
    uint8_t *k, *v;
    const int32_t *table;
    int64_t ld_table;
    int64_t page_bytes, head_bytes, slot_bytes;  // strides
    int64_t n_pages;
    int32_t batch, max_pages, page_size, heads;
    int32_t capacity;     // max_pages * page_size
    uint32_t div_mul;     // slot / page_size = slot * div_mul >> div_shift for 0 <= slot < 2^31:
    uint32_t div_shift;   // div_shift = 31 + ceil(log2 d), div_mul = ceil(2^div_shift / d)
    int32_t dim;          // values of a head
    int32_t e4m3;
    float k_scale, v_scale;
    unsigned int *status;
};

__device__ __forceinline__ uint32_t page_of(const KvView &c, uint32_t slot) {
    return (uint32_t)(((uint64_t)slot * c.div_mul) >> c.div_shift);
}

// Byte offset (in either pool) of a slot's row of head h, given its page's id.
__device__ __forceinline__ int64_t row_bytes_at(const KvView &c, int32_t page, int h, uint32_t slot_in_page) {
    return page * c.page_bytes + h * c.head_bytes + slot_in_page * c.slot_bytes;
}

__device__ __forceinline__ bool page_ok(const KvView &c, int32_t page) { return page >= 0 && page < c.n_pages; }

}  // namespace q4k
