// linrec_internal.h -- host-side pieces shared by the gated linear recurrence's
// translation units: arguments, workspace layout, launcher declarations.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "prefix_scan_recurrence.h"

namespace ps {

constexpr int kLinrecWide = 32;       // channels of a tile
constexpr int kLinrecWarps = 8;       // warps of a CTA that compute
constexpr int kLinrecTile = 512 * kLinrecWarps / kLinrecWide;   // tokens of the smallest tile: 128
// How many tokens are between the states that training keeps: the backward pass's tile.
constexpr int linrec_start_tokens(size_t type_bytes, size_t gate_bytes) {
    return kLinrecTile * (2 * type_bytes + gate_bytes > 8 ? 1 : 2);
}

struct LinrecTensor {                 // element strides; channels are contiguous
    const void *p;
    long long seq, tok;
    bool flat;                        // seq is tok times the tokens of a sequence
    int piece;                        // rows start on multiples of so many bytes, and hold a multiple of them: 16, 4 or 2
};

// Workspace.  A ticket counter and what tiles tell one another, for each (tile of tokens, block of 32 channels, pair of channels):
//   map    the tile's factors, encoded as in linrec_common.cuh, and what it adds
//   state  the state (backward: the state's gradient) behind the tile
// (set by each call to 0xff bytes, which stands for nothing told yet), and in training `start`, the state before each tile
// of the backward pass, which that begins from.
struct LinrecArgs {
    long long seqs, tokens, total;    // total: tokens of all sequences
    const int32_t *cu;
    long long channels;
    int tiles, blocks;                // tiles of tokens (set by the launchers), blocks of channels
    int steps;                        // tiles of a sequence where equal sequences take turns (set by the launchers), else 0
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
constexpr int kLinrecSlack = 16;      // tiles' places behind the last one that a look-back's round may read
// Equal sequences of whole tiles take turns, so that the tiles under way at a time are of many chains and few wait for one another.
inline int linrec_steps(const LinrecArgs &a, int tokens) {
    return a.cu == nullptr && a.seqs > 1 && a.tokens % tokens == 0 ? (int)(a.tokens / tokens) : 0;
}
// Tiles of `tokens`: how many, in which order, and where they tell one another what; sets that to nothing told.
inline cudaError_t linrec_prepare(LinrecArgs &a, int tokens, cudaStream_t s) {
    a.tiles = (int)((a.total + tokens - 1) / tokens);
    a.steps = linrec_steps(a, tokens);
    if (a.tiles < 2) return cudaSuccess;
    const size_t places = ((size_t)a.tiles + kLinrecSlack) * (size_t)a.blocks * (kLinrecWide / 2);
    a.map = reinterpret_cast<float4 *>(a.ticket + 64);
    a.state = reinterpret_cast<float2 *>(a.map + places);
    return cudaMemsetAsync(a.ticket, 0xff, 256 + places * 24, s);
}
inline unsigned linrec_grid(const LinrecArgs &a, int ctas_per_sm) {
    const long long all = (long long)a.tiles * a.blocks;
    return (unsigned)(a.tiles == 1 || all < 152 * ctas_per_sm ? all : 152 * ctas_per_sm);
}

struct LinrecStepArgs {
    long long seqs, pages, channels;
    int t;
    LinrecTensor x, g;
    float *state;
    const int32_t *slots, *lengths;
    void *h;
};

// Describes tiles of an input for tensor copies, token by token of `runs` runs of `run` tokens; false where its rows are not
// evenly spaced on multiples of 16 bytes, no run is whole, or the driver declines.
bool linrec_tensor_map(CUtensorMap &map, const LinrecTensor &x, const LinrecArgs &a, size_t bytes, bool f16, int runs, int run);

cudaError_t launch_linrec_forward(const LinrecArgs &a, int type, int gate_type, bool tied, cudaStream_t s);
cudaError_t launch_linrec_backward(const LinrecArgs &a, int type, int gate_type, bool tied, cudaStream_t s);
// vec: four channels a thread.
cudaError_t launch_linrec_step(const LinrecStepArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s);

}  // namespace ps
