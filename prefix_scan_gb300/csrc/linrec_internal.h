// linrec_internal.h -- host-side pieces shared by the gated linear recurrence's
// translation units: arguments, workspace layout, launcher declarations.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "prefix_scan_recurrence.h"

namespace ps {

constexpr int kLinrecTile = 64;       // tokens of the smallest tile
constexpr int kLinrecCtas = 152 * 2;  // two CTAs stay on each SM
// How many tokens are between the states that training keeps: the backward pass's tile.
constexpr int linrec_start_tokens(size_t type_bytes) { return type_bytes == 4 ? 64 : 128; }

struct LinrecTensor {                 // element strides; channels are contiguous
    const void *p;
    long long seq, tok;
    bool flat;                        // seq is tok times the tokens of a sequence
    int piece;                        // rows start on multiples of so many bytes, and hold a multiple of them: 16, 4 or 2
};

// Workspace.  A ticket counter and what tiles tell one another, for each (tile of tokens, block of 64 channels, lane of two
// channels):
//   map    the tile's factors, encoded as in linrec_common.cuh, and what it adds
//   state  the state (backward: the state's gradient) behind the tile
// (set by each call to 0xff bytes, which stands for nothing told yet), and in training `start`, the state before each tile
// of the backward pass, which that begins from.
struct LinrecArgs {
    long long seqs, tokens, total;    // total: tokens of all sequences
    const int32_t *cu;
    long long channels;
    int tiles, blocks;                // tiles of tokens (set by the launchers), blocks of channels
    int start_tokens;
    bool tensor_copies;               // inputs come by tensor copies (set by the launchers)
    bool pairs;                       // outputs' rows start on multiples of two numbers
    LinrecTensor x, g, dout;
    const float *h0, *dht;
    float *ht, *dh0;
    void *h, *dx, *dg;
    unsigned *ticket;                 // the last one taken
    float4 *map;                      // factor and addend of the first channel's pair: (f, f', b, b')
    float2 *state;
    float *start;                     // nullptr outside of training
};
inline unsigned linrec_grid(const LinrecArgs &a) {
    const long long all = (long long)a.tiles * a.blocks;
    return (unsigned)(a.tiles == 1 || all < kLinrecCtas ? all : kLinrecCtas);
}

struct LinrecStepArgs {
    long long seqs, pages, channels;
    int t;
    LinrecTensor x, g;
    float *state;
    const int32_t *slots, *lengths;
    void *h;
};

// Describes tiles of `tokens` by 64 channels of an input for tensor copies; false where its rows are not evenly spaced on
// multiples of 16 bytes, or the driver declines.
bool linrec_tensor_map(CUtensorMap &map, const LinrecTensor &x, const LinrecArgs &a, size_t bytes, bool f16, int tokens);

cudaError_t launch_linrec_forward(const LinrecArgs &a, int type, int gate_type, bool tied, cudaStream_t s);
cudaError_t launch_linrec_backward(const LinrecArgs &a, int type, int gate_type, bool tied, cudaStream_t s);
// vec: four channels a thread.
cudaError_t launch_linrec_step(const LinrecStepArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s);

}  // namespace ps
