// Lists of requests and rows of tokens that belong to them, for the kernels that work on page tables.
#pragma once

#include <stdint.h>

#include "kda.h"

namespace kda {

__device__ __forceinline__ int64_t load_index(const void *p, int32_t itype, int64_t i)
{
    return itype == KDA_I32 ? static_cast<int64_t>(static_cast<const int32_t *>(p)[i]) : static_cast<const int64_t *>(p)[i];
}

// Length of a request as the table can hold it.
__device__ __forceinline__ int64_t length_of(const kda_page_table &t, int64_t r)
{
    const int64_t n = t.seq_lens[r], most = t.width * t.page_size;
    return n < 0 ? 0 : n > most ? most : n;
}

// The list entry i with cu[i] <= tok < cu[i + 1], for cu[0] <= tok < cu[count]; by the whole warp, in 33-way steps: two
// looks for a thousand entries.
__device__ __forceinline__ int64_t entry_of(const int32_t *cu, int64_t count, int64_t tok)
{
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = count;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + step * lane;
        const uint32_t below = __ballot_sync(0xffffffffu, at < hi && cu[at] <= tok);  // lane 0 always
        const int64_t from = lo + step * (below != 0 ? __popc(below) - 1 : 0);  // 0 only if the offsets fall somewhere
        hi = from + step < hi ? from + step : hi;
        lo = from;
    }
    return lo;
}

}  // namespace kda
