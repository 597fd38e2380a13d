// memq_attn_owner.cuh -- the notes by which memq_attn_paged's join finds the pieces of an item.  Plain C++, so that a test
// on the host runs the same check.
#pragma once

#include <cstdint>

#ifndef MEMQ_HD
#ifdef __CUDACC__
#define MEMQ_HD __host__ __device__ __forceinline__
#else
#define MEMQ_HD inline
#endif
#endif

namespace memq {

// A piece of an item's rows whose keys were shared among several runs, noted by the run that holds its
// first key (`rows` is 0 otherwise): the other pieces are those of the runs up to `last`.
struct alignas(16) AttnOwner {
    int start;        // the sequence's first token
    int row0;         // the item's first row among the t * group rows of (sequence, kv head)
    int first, last;  // runs
    int head, rows;
    int unused[2];
};
static_assert(sizeof(AttnOwner) == 32, "two loads");

// Whether the pieces that a note names, of up to `stride` rows each, and the rows of `out` lie inside their arrays.  Notes
// are of the kernel before, so they do, unless something else wrote to the workspace meanwhile (another call that was given
// the same one): then outputs are lost, but nothing else is.
MEMQ_HD bool attn_owner_ok(const AttnOwner &o, int n_tok, int n_kv, int group, int runs, int stride) {
    if (o.rows < 1 || o.rows > stride || o.row0 < 0 || o.start < 0 || o.start >= n_tok || o.first < 0 || o.first >= runs ||
        o.last < o.first || o.head < 0 || o.head >= n_kv)
        return false;
    const uint32_t last_row = static_cast<uint32_t>(o.row0) + static_cast<uint32_t>(o.rows - 1);
    return last_row / static_cast<uint32_t>(group) < static_cast<uint32_t>(n_tok - o.start);
}

}  // namespace memq
