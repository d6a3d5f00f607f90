// Device helpers shared by the kernels of the paged int8 key/value cache: the
// sequences of packed tokens and the pages of their positions.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "llmint8.h"

namespace llmint8 {

// The cache and its sequences as the kernels see them. The kernel before may
// write any of it while this one starts: no loads that take it as constant
// (__ldg), and absmax, whose lines are written by several CTAs, past L1 (__ldcg).
struct KvView {
    int8_t *k, *v;
    float *ka, *va;
    int pages, heads, page_size, page_shift, batch, table_width;
    int64_t table_stride;
    const int32_t *table, *lens, *cu;
    uint32_t *status;
};

// The sequence whose rows include packed row t: the last b with cu[b] <= t
// (rows at and behind cu[batch] belong to none: -1).
__device__ __forceinline__ int sequence_of(const KvView &c, int64_t t)
{
    int lo = 0, hi = c.batch; // cu[lo] <= t < cu[hi], if t has a sequence
    if (t < c.cu[0] || t >= c.cu[c.batch])
        return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c.cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Page of a position of sequence b, or -1 (and the status bit) if the table
// or the cache does not have it.
__device__ __forceinline__ int page_of(const KvView &c, int b, int pos)
{
    const int j = pos >> c.page_shift;
    int page = -1;
    if (j < c.table_width)
        page = c.table[b * c.table_stride + j];
    if ((unsigned)page >= (unsigned)c.pages) {
        atomicOr(c.status, LLMINT8_DEV_BAD_PAGE);
        page = -1;
    }
    return page;
}

} // namespace llmint8
