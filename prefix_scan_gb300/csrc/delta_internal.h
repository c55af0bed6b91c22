// delta_internal.h -- host-side pieces shared by the gated delta rule's
// translation units: arguments, workspace layout, launcher declarations.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "prefix_scan_delta.h"

namespace ps {

constexpr int kChunk = 64;        // tokens of a chunk
constexpr int kMaxDimK = 128;     // largest key size

struct DeltaTensor {              // element strides; the innermost dimension is contiguous
    const void *p;
    long long seq, tok, head;
};
struct DeltaShape {
    long long seqs, tokens;       // tokens of each sequence, or of all with cu
    const int32_t *cu;
    int hk, hv, k, v;
    float scale;
};

// What the forward kernels leave for each (chunk, value head), in this order; all
// images are swizzled as in delta_common.cuh and kept as pairs hi, lo of bf16.
//   scal   6 x 64 f32: exp(G), exp(G_C - G), beta, G as a sum of two floats, and how many
//          tokens up to here have forgotten the state
//   T - 1  2 x 64 x 64       row i, column j (T's diagonal is 1)
//   P      2 x 64 x 64
// and for the backward pass, for each block of 128 values (rows past the values, to a multiple
// of 16, are 0; further ones are not written)
//   S      2 x 128 x K       row v, column k: the state at the chunk's start
//   U      2 x 128 x 64      row v, column token
// to which the backward chain adds dS (as S: the gradient of the state at the chunk's end) and
// dU (as U).  After all of these come, for each (chunk, key head), the chunk's keys (rows 0-63)
// and queries (rows 64-127) as one image of 128 rows of K, one plane for bf16 and two for other
// types: rows past the sequence's end and columns past K are 0.
struct ChunkLayout {
    size_t scal, t, p, s, u, ds, du, stride;
};
constexpr size_t kSquare = (size_t)kChunk * kChunk * 2;   // bytes of one 64 x 64 plane
constexpr int kBlockV = 128;                              // values of a block
constexpr int pad_k(int k) { return k <= 64 ? 64 : 128; }
constexpr int blocks_v(int v) { return (v + kBlockV - 1) / kBlockV; }
constexpr size_t s_plane(int k) { return (size_t)kBlockV * pad_k(k) * 2; }
constexpr size_t kUPlane = (size_t)kBlockV * kChunk * 2;
constexpr ChunkLayout chunk_layout(int k, int v, bool train) {
    ChunkLayout l{};
    const size_t sb = 2 * s_plane(k) * blocks_v(v), ub = 2 * kUPlane * blocks_v(v);
    size_t at = 0;
    l.scal = at; at += 6 * kChunk * 4;
    l.t = at; at += 2 * kSquare;
    l.p = at; at += 2 * kSquare;
    if (train) {
        l.s = at; at += sb;
        l.u = at; at += ub;
        l.ds = at; at += sb;
        l.du = at; at += ub;
    }
    l.stride = (at + 255) / 256 * 256;
    return l;
}
constexpr size_t kq_stride(int k, int planes) { return (size_t)planes * 2 * kChunk * pad_k(k) * 2; }
constexpr long long delta_slots(long long seqs, long long tokens, bool packed) {
    return packed ? tokens / kChunk + seqs : seqs * ((tokens + kChunk - 1) / kChunk);
}

// Long sequences over few heads are cut into segments of `seg` chunks, so that more CTAs have a
// chain to run.  The state at a segment's end is M S + B, S the state at its start, M a K x K matrix:
// a first pass runs the segments' chains without outputs, B from S = 0 and M as the chain of K
// values that start from the identity and add nothing; a join goes through the segments in order
// (delta_join.cu); a second pass runs every segment from its own start.  The backward pass does the
// same from the other end, with M's transpose.
//   seg_state  [segment slots + 1, hv, K, V] f32: the state at each segment's start; backward, its
//              gradient at each segment's end (one slot further on)
//   seg_h      [seqs, hv, K, V] f32: a copy of h0 that ht takes the place of (of d_ht and dh0): the segment
//              that reads the one and the segment that writes the other run at the same time
//   seg_m      [segment slots, hv] pairs of images of M (row j, column k: M_kj), as S's

// Packed sequences of very different lengths: the chains of the longest are launched first, so that the
// last ones to run are short.  Their order is counted by one CTA of the prepare kernel, in time that grows
// with the square of the sequences' number; with more than kOrdered, chains are many and even out.  48
// sequences of 0 to 35 chunks, 32 heads: 31 us less than in the order in which they come (of 286).
constexpr long long kOrdered = 256;
enum DeltaPass { kPassAll = 0, kPassStates = 1 };
struct DeltaArgs {
    DeltaShape s;
    DeltaTensor q, k, v, g, beta;
    int beta_f32;                 // beta holds f32 and not the inputs' type
    int vec_qk, vec_v;            // rows 16-byte aligned, sizes a multiple of 8
    const float *h0;              // [seqs, hv, k, v] or null
    float *ht;                    // the same, or null
    void *o;                      // contiguous [tokens, hv, v]
    unsigned char *ws, *kq;
    long long slots;
    int train;                    // keep what the backward pass reads
    int seg;                      // chunks of a segment, 0: sequences are not cut
    int pass;
    long long seg_slots;
    float *seg_state, *seg_h;
    int32_t *order;               // [seqs] by falling length, or null: as they come
    int *failed;                  // training: cleared by the prepare kernel, set by a chain whose waits ran out
                                  // (what it kept then is not to be used: all gradients become NaN); else null
    unsigned char *seg_m;
    // backward
    DeltaTensor dout;
    int vec_do;
    const float *dht;
    float *dh0, *dg;
    void *dq, *dk, *dv, *dbeta;
};

// Type codes: PS_REAL_F32, PS_REAL_BF16, PS_REAL_F16.
cudaError_t launch_delta_prepare(const DeltaArgs &a, int type, cudaStream_t s);
cudaError_t launch_delta_chain(const DeltaArgs &a, int type, cudaStream_t s);
cudaError_t launch_delta_chain_backward(const DeltaArgs &a, int type, cudaStream_t s);
cudaError_t launch_delta_join(const DeltaArgs &a, bool backward, cudaStream_t s);
cudaError_t launch_delta_gradients(const DeltaArgs &a, int type, cudaStream_t s);

constexpr size_t seg_m_bytes(int k) { return 2 * s_plane(k); }
// Chunks of a segment, for `chains` chains of `chunks` chunks on average; 0 where cutting does not pay.
// A chain takes a CTA, of which 152 run at once.  n segments cost the waves of the first pass (n - 1
// chains for B, n - 2 for M) and of the second, in chunks of time, and about a chunk's time for each
// step of the join; the backward pass has no M to find.
inline int segment_chunks(long long chains, long long chunks, bool train) {
    if (chains <= 0 || chunks < 8) return 0;
    auto waves = [](long long ctas) { return (ctas + 151) / 152; };
    long long best = chunks * waves(chains) * (train ? 2 : 1), best_len = 0;
    for (long long n = 3; n <= 64 && n * 4 <= chunks; ++n) {
        const long long len = (chunks + n - 1) / n;
        long long cost = len * (waves(chains * (2 * n - 3)) + waves(chains * n)) + n;
        if (train) cost += len * (waves(chains * (n - 1)) + waves(chains * n)) + n;
        if (cost < best) { best = cost; best_len = len; }
    }
    return (int)best_len;
}
constexpr long long segment_slots(long long slots, long long seqs, int seg) { return seg ? slots / seg + seqs : 0; }

struct DeltaStepArgs {
    long long seqs, pages;
    int t, hk, hv, k, v;
    float scale;
    DeltaTensor q, kk, vv, g, beta;
    int beta_f32;
    float *state;                 // [pages, hv, k, v]
    const int32_t *slots, *lengths;   // [seqs] or null
    void *o;                      // contiguous [seqs, t, hv, v]
};
cudaError_t launch_delta_step(const DeltaStepArgs &a, int type, cudaStream_t s);

}  // namespace ps
