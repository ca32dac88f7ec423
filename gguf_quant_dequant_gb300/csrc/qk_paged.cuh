// qk_paged.cuh -- geometry of the paged KV pools (include/qk.h, "A paged,
// block-quantized KV cache"): pool [n_pages][n_kv][page][d], rows of d / 32
// blocks.  A page size is a power of two, so a position splits into page and
// offset by shifts.
#pragma once
#include <cstdint>

#include "qk_ptx.cuh"

namespace qk {

struct Pool {
    int64_t n_pages;
    int page_log2;
    int n_kv;
    int row_bytes;   // d / 32 blocks
};

// Byte offset of the row of (page id, kv head, offset in the page).  64-bit:
// a pool of many gigabytes has more bytes than 32 bits count.
__device__ __forceinline__ int64_t pool_row(const Pool& p, int64_t id, int head, int off) {
    return (((id * p.n_kv + head) << p.page_log2) + off) * p.row_bytes;
}

// Page id of position pos of a request with table row `tab`, or -1 where the
// table has no such entry or the id lies outside the pool (recorded in the
// status word).
__device__ __forceinline__ int page_of(const Pool& p, const int32_t* tab, int64_t table_stride, int64_t pos,
                                       unsigned* status) {
    const int64_t i = pos >> p.page_log2;
    const int id = (pos >= 0 && i < table_stride) ? tab[i] : -1;
    if (id >= 0 && id < p.n_pages) return id;
    atomicOr(status, STATUS_BAD_PAGE);
    return -1;
}

}  // namespace qk
