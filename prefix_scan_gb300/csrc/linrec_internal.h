// linrec_internal.h -- host-side pieces shared by the gated linear recurrence's
// translation units: arguments, workspace layout, launcher declarations.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "prefix_scan_recurrence.h"

namespace ps {

constexpr int kLinrecTile = 128;      // tokens of a tile
constexpr int kLinrecWarps = 8;       // warps of a CTA, each with a run of the tile's tokens
constexpr int kLinrecRun = kLinrecTile / kLinrecWarps;

struct LinrecTensor {                 // element strides; channels are contiguous
    const void *p;
    long long seq, tok;
};

// Workspace.  A tile is 128 tokens of the flat index over all sequences' tokens by 32 V channels (V channels a lane);
// what tiles tell one another, for each (tile, channel):
//   flag   one word a tile and block of channels: 0 nothing yet, 1 `map`, 2 `state` (cleared by each call)
//   map    the tile's factor, encoded as in linrec_common.cuh, and what it adds
//   state  the state (backward: the state's gradient) behind the tile
// and in training `start`, the state before each tile, which the backward pass begins from.
struct LinrecArgs {
    long long seqs, tokens, total;    // total: tokens of all sequences
    const int32_t *cu;
    long long channels;
    int tiles, blocks;                // tiles of tokens, blocks of channels
    LinrecTensor x, g, dout;
    const float *h0, *dht;
    float *ht, *dh0;
    void *h, *dx, *dg;
    unsigned *ticket, *flag;
    float2 *map;
    float *state, *start;             // start: nullptr outside of training
};

struct LinrecStepArgs {
    long long seqs, pages, channels;
    int t;
    LinrecTensor x, g;
    float *state;
    const int32_t *slots, *lengths;
    void *h;
};

// vec: two channels a lane (every row starts on a multiple of two elements), else one.
cudaError_t launch_linrec_forward(const LinrecArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s);
cudaError_t launch_linrec_backward(const LinrecArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s);
// vec: four channels a thread.
cudaError_t launch_linrec_step(const LinrecStepArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s);

}  // namespace ps
