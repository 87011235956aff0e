// kv4_common.cuh -- the 4-bit key/value cache as the kernels see it.
//
// A page holds page_size tokens of every key/value head, one block per head:
//   key codes   [page_size][D/2]  bytes, element 2i in the low nibble of byte i
//   value codes [page_size][D/2]
//   key scales  [page_size] bf16
//   value scales[page_size] bf16
// with code nibble = c + 8, c in -7..7, value = c * scale. One head of one
// page is contiguous (page_size * (D + 4) bytes, a multiple of 16), so a tile
// of tokens is one bulk copy.
#pragma once

#include "divisor.cuh"
#include "tq_internal.h"

namespace tq {

struct Kv4View {
    uint8_t *pages;
    const int32_t *table;  // [batch, max_pages]
    long long page_stride;
    int num_pages, max_pages, batch, kv_heads;
    int lg_ps;  // log2(page_size)
    unsigned *err;

    __host__ __device__ int page_size() const { return 1 << lg_ps; }
    __host__ __device__ int max_len() const { return max_pages << lg_ps; }
    template <int D>
    __host__ __device__ long long head_bytes() const
    {
        return (long long)(D + 4) << lg_ps;
    }
};

// The cached length that a kernel works with, of the one given: a negative one
// is an empty sequence, one beyond the page table is cut to it (and reported).
__device__ __forceinline__ int kv4_cut(const Kv4View &c, int n)
{
    if (n > c.max_len()) {
        atomicOr(c.err, kErrBadPage);
        return c.max_len();
    }
    return max(n, 0);
}

__device__ __forceinline__ int kv4_len(const Kv4View &c, const int32_t *lens, int b)
{
    return kv4_cut(c, lens[b]);
}

}  // namespace tq
