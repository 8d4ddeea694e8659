// embed.hpp -- what the embedding kernels and their host code share.
//
// The gradient of a lookup is a segment sum of rows by key: the tokens' keys
// (their rows of the table) are sorted stably with their positions, chunks of
// the sorted list are summed, and what a run of one key left in several chunks
// is joined.  A run's rows are added in the order of their positions within a
// chunk; of a run in several chunks eight parts, of as many chunks one after
// another each, are added up in the chunks' order, and then these in theirs.
// So the bits are the same every time.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/libscan.h"

namespace libscan {

constexpr int kSortThreads = 512;
constexpr int kSortTile = 4096;           // keys of a workgroup
constexpr int kSortBits = 9;              // the widest digit
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortMaxPasses = 4;

struct EmbedRowsArgs {
    const void *weight;
    void *out;
    const void *ids;
    int64_t weight_stride, out_stride;
    int dtype, out_dtype, id_bytes;
    uint64_t tokens, rows, width;
    float scale;
    int lanes;                            // lanes of a row
    uint32_t across;                      // workgroups along a row
};
hipError_t launch_embed_rows(EmbedRowsArgs a, hipStream_t stream);

// The sort of a call: its passes, digits and tiles.
struct SortPlan {
    int passes, bits;                     // bits of a digit
    uint32_t tiles;
};
SortPlan sort_plan(uint64_t tokens, uint64_t rows);
// Entries of a chunk of the sorted list.
uint32_t embed_chunk(uint64_t tokens);

struct EmbedGradArgs {
    const void *dout;
    void *dweight;
    const void *ids;
    int64_t dout_stride, dweight_stride;
    int dtype, out_dtype, id_bytes;
    uint32_t tokens;
    uint64_t rows, width;
    float scale;
    bool accumulate;
    SortPlan sort;
    uint32_t *keys[2], *at[2];            // sorted back and forth; the last pass writes [0]
    uint32_t *hist;                       // [passes][tiles][bins], then the current pass's totals [bins]
    uint32_t *totals;
    float *partial;                       // [chunks][2][width]
    uint32_t chunk, chunks;
    uint32_t across;                      // waves along a row
};
size_t embed_grad_body_bytes(uint64_t tokens, uint64_t rows, uint64_t width);
hipError_t launch_embed_grad(EmbedGradArgs a, void *body, hipStream_t stream);

}  // namespace libscan
