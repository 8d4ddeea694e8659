// gatescan.hpp -- what the gated recurrence's kernels and host code share.
//
// Each channel of each sequence is a recurrence of its own,
//
//   forward   h(t) = a(t) h(t-1) + b(t)                      in the tokens' order
//   gradient  G(t) = a(t) (G(t+1) + dout(t))                 in reverse
//
// with dh(t) = dout(t) + G(t+1) the gradient of h(t): a prefix scan of pairs
// under (A, H) o (A', H') = (A A', A' H + H').  A tile is kTile tokens of as
// many channels as 128 bytes hold.  A workgroup reads its tile once, scans it,
// takes what enters it from the tiles before, and writes its outputs once.
//
// What enters a tile is always the chain h <- A h + H over the tiles before,
// from the sequence's first on and in their order: a tile looks back no
// further than the nearest whose chained value is there and goes on from it
// by the same steps that those tiles take.  So the bits do not depend on which
// tiles were ready.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/libscan.h"

namespace libscan {

constexpr int kGateLanes = 8;          // lanes of a row: 16 bytes each
constexpr int kGateThreads = 256;
constexpr int kGateWindow = 12;        // tiles that a look back spans at most
constexpr int kGateGroups = kGateThreads / kGateLanes;

// Counters that tiles are drawn from, one for each die, 128 bytes apart: set i
// has the lines from gate_set(lines, i) on.
constexpr uint32_t kGateSets = 8, kGateCounterStride = 16;
constexpr size_t kGateCounterBytes = kGateSets * kGateCounterStride * sizeof(uint64_t);
__host__ __device__ constexpr uint32_t gate_set(uint32_t lines, uint32_t i)
{
    return (uint32_t)((uint64_t)lines * i / kGateSets);
}

// Tokens of a thread, and of a tile.
constexpr int gate_rows(int dtype, bool grad) { return dtype == LIBSCAN_F32 && !grad ? 8 : 4; }
constexpr int gate_tile(int dtype, bool grad) { return kGateGroups * gate_rows(dtype, grad); }
constexpr int gate_channels(int dtype) { return kGateLanes * (dtype == LIBSCAN_F32 ? 4 : 8); }

struct GateRows {
    const void *p;
    int64_t seq, tok;
};

struct GateArgs {
    GateRows gate, x, dout, h;         // h: the forward pass's outputs (gradient only)
    void *out[2];                      // out; or dgate, dx
    int64_t out_seq[2], out_tok[2];
    int dtype, form;
    bool blend, clear;
    uint32_t seqs;
    uint64_t tokens, width;            // tokens of a sequence, or in all when ends is given
    const uint32_t *ends;
    const float *first;                // h before the first token, or null
    const float *last;                 // gradient of h after the last token, or null
    float *state_out;                  // h after the last token; or the gradient of `first`; or null
    uint32_t blocks;                   // tiles along the width
    uint32_t chains, tiles;            // lines of tiles, and the tiles of each
    bool far;                          // a look back spans kGateWindow tiles, else four
    // Of the chained carry, where there is more than one tile: this launch's tag
    // of its words.
    uint32_t tag;
    uint64_t *counters, *desc;
};

// Lines of tiles and tiles of each; false where a grid cannot hold them.
bool gate_grid(int dtype, bool grad, bool packed, uint32_t seqs, uint64_t tokens, uint64_t width,
               uint32_t *blocks, uint32_t *chains, uint32_t *tiles);
// Whether looks back span kGateWindow tiles, not four.  With few lines a chained
// value moves further in the time of a look than four tiles: lines of 1025 tiles
// (bf16, log, blend) take with twelve 198 us where there is one, 164 with four and
// 234 with 16, with four 268, 230 and 282.  The more lines, the more a look's words
// cost: 2^26 elements in 16 lines take 122 us with twelve and 145 with four, in 32
// and 48 the same, in 64 to 384 with four 1 to 3% less (92.7 and 89.9 in 128; the
// gradient 146.5 and 144.2).  From 64 lines to 127 that is given up.
bool gate_far(uint32_t chains);
size_t gate_desc_bytes(int dtype, uint32_t chains, uint32_t tiles);

hipError_t launch_gatescan(const GateArgs &a, hipStream_t stream);
hipError_t launch_gatescan_grad(const GateArgs &a, hipStream_t stream);

struct GateStepArgs {
    GateRows gate, x;                  // seq is the stride of a row
    void *out;
    int64_t out_seq;
    int dtype, form;
    bool blend;
    uint32_t rows;
    uint64_t width;
    const float *state;
    float *state_out;
    uint64_t pool;
    const int32_t *slots;
};
hipError_t launch_gatescan_step(const GateStepArgs &a, hipStream_t stream);

}  // namespace libscan
