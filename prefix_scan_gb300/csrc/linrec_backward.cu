// linrec_backward.cu -- gradients of the gated linear recurrence (notation and
// tiles in linrec_common.cuh).
//
// Bound by memory: x, g and dh are read once, dx and dg are written once.  The states are not read: the forward pass keeps
// the one before each tile (in 32 bits, 1/128 of a number an element), and the tile is scanned again from there, so that
// 16-bit types, too, get the gradient of g from states of 32 bits.  What runs backward is mu, a state's gradient handed to
// the token before; its look-back goes over the tiles from the last one.
#include "linrec_common.cuh"

namespace ps {

namespace {

template <typename TX, typename TG, int V, bool TIED>
__global__ void __launch_bounds__(kLrThreads, 2) linrec_backward_kernel(const LinrecArgs a) {
    __shared__ Marks marks;
    __shared__ Sums<V> sums;                           // of mu
    __shared__ float sum_h[kLinrecWarps][32 * V];      // what the runs add to h
    __shared__ float behind[32 * V];
    __shared__ unsigned ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) ticket = a.tiles > 1 ? atomicAdd(a.ticket, 1u) : blockIdx.x;
    __syncthreads();
    const int k = (int)(ticket / (unsigned)a.blocks), block = (int)(ticket % (unsigned)a.blocks), tile = a.tiles - 1 - k;
    const uint32_t n0 = (uint32_t)tile * kLinrecTile, first = n0 + warp * kLinrecRun, total = (uint32_t)a.total;
    const long long c0 = (long long)block * (32 * V), ch = c0 + lane * V;
    const bool in = ch < a.channels;

    Lanes<TX, V> x[kLinrecRun], dh[kLinrecRun];
    Lanes<TG, V> g[kLinrecRun];
    load_run<TG, V>(g, a.g, first, total, (uint32_t)a.tokens, ch, a.channels);
    load_run<TX, V>(x, a.x, first, total, (uint32_t)a.tokens, ch, a.channels);
    load_run<TX, V>(dh, a.dout, first, total, (uint32_t)a.tokens, ch, a.channels);
    float h[V], s[V], mu[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = in ? a.start[tile * a.channels + ch + v] : 0.f;
    mark_tile(marks, a, n0, tile == a.tiles - 1, a.dht, a.dh0, c0, 32 * V);
    const uint32_t starts = run_bits(marks.start, warp), ends = run_bits(marks.end, warp);
    auto start = [&](float (&y)[V], int i) {
        const float *p = a.h0 + marks.start_seq[warp * kLinrecRun + i] * a.channels + ch;
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = a.h0 && in ? p[v] : 0.f;
    };
    auto end = [&](float (&y)[V], int i) {
        const float *p = a.dht + marks.end_seq[warp * kLinrecRun + i] * a.channels + ch;
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = a.dht && in ? p[v] : 0.f;
    };

    float f[kLinrecRun][V], add[V];
#pragma unroll
    for (int v = 0; v < V; ++v) add[v] = s[v] = mu[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kLinrecRun; ++i) {
        if (starts >> i & 1) start(add, i);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float gi = to_f32<TG>(g[i].v[v]), xi = to_f32<TX>(x[i].v[v]);
            f[i][v] = factor(gi);
            s[v] += gi;
            add[v] = apply(f[i][v], add[v], TIED ? forgotten(f[i][v]) * xi : xi);
        }
    }
#pragma unroll
    for (int i = kLinrecRun - 1; i >= 0; --i) {
        if (ends >> i & 1) end(mu, i);
#pragma unroll
        for (int v = 0; v < V; ++v) mu[v] = apply(f[i][v], to_f32<TX>(dh[i].v[v]) + mu[v], 0.f);
        if (starts >> i & 1) {   // dh0 takes it
#pragma unroll
            for (int v = 0; v < V; ++v) mu[v] = 0.f;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sums.s[warp][lane * V + v] = s[v];
        sums.b[warp][lane * V + v] = mu[v];
        sum_h[warp][lane * V + v] = add[v];
    }
    __syncthreads();
    auto cut = [&](int w) { return (run_bits(marks.start, w) | run_bits(marks.end, w)) != 0; };
    if (warp == 0) {
        float carry[V];
        tile_carry<V>(carry, a, k, block, sums, cut, any_bits(marks.start) || any_bits(marks.end),
                      marks.end[kLinrecTile / 32 - 1] >> 31 == 0, true);
#pragma unroll
        for (int v = 0; v < V; ++v) behind[lane * V + v] = carry[v];
    }
    // the states before each token; with tied inputs less the token's x, as the gradient of g needs them
    for (int w = 0; w < warp; ++w) {
        const bool reset = run_bits(marks.start, w) != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = sum_h[w][lane * V + v];
            h[v] = reset ? b : apply(factor_of_sum(sums.s[w][lane * V + v]), h[v], b);
        }
    }
    float was[kLinrecRun][V];
#pragma unroll
    for (int i = 0; i < kLinrecRun; ++i) {
        if (starts >> i & 1) start(h, i);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float xi = to_f32<TX>(x[i].v[v]);
            was[i][v] = TIED ? h[v] - xi : h[v];
            h[v] = apply(f[i][v], h[v], TIED ? forgotten(f[i][v]) * xi : xi);
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) mu[v] = behind[lane * V + v];
    for (int w = kLinrecWarps - 1; w > warp; --w) {
        const bool reset = cut(w);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = sums.b[w][lane * V + v];
            mu[v] = reset ? b : apply(factor_of_sum(sums.s[w][lane * V + v]), mu[v], b);
        }
    }
    TX *dx = static_cast<TX *>(a.dx) + (long long)first * a.channels + ch;
    TG *dg = static_cast<TG *>(a.dg) + (long long)first * a.channels + ch;
    const uint32_t held = marks.hi > marks.lo ? marks.hi - marks.lo : 0;
#pragma unroll
    for (int i = kLinrecRun - 1; i >= 0; --i) {
        if (ends >> i & 1) end(mu, i);
        float gx[V], gg[V];
        const bool counts = first + i - marks.lo < held;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float lam = to_f32<TX>(dh[i].v[v]) + mu[v];
            mu[v] = apply(f[i][v], lam, 0.f);
            gx[v] = counts ? TIED ? forgotten(f[i][v]) * lam : lam : 0.f;
            gg[v] = counts ? mu[v] * was[i][v] : 0.f;
        }
        if (in && first + i < total) {
            store_lanes<TX, V>(dx + i * a.channels, gx);
            store_lanes<TG, V>(dg + i * a.channels, gg);
        }
        if (starts >> i & 1) {
            if (a.dh0 != nullptr && in) {
                float *p = a.dh0 + marks.start_seq[warp * kLinrecRun + i] * a.channels + ch;
#pragma unroll
                for (int v = 0; v < V; ++v) p[v] = mu[v];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) mu[v] = 0.f;
        }
    }
}

template <typename TX, typename TG> cudaError_t launch(const LinrecArgs &a, bool tied, bool vec, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.tiles * (long long)a.blocks);
    if (vec) {
        if (tied) linrec_backward_kernel<TX, TG, 2, true><<<grid, kLrThreads, 0, s>>>(a);
        else linrec_backward_kernel<TX, TG, 2, false><<<grid, kLrThreads, 0, s>>>(a);
    } else {
        if (tied) linrec_backward_kernel<TX, TG, 1, true><<<grid, kLrThreads, 0, s>>>(a);
        else linrec_backward_kernel<TX, TG, 1, false><<<grid, kLrThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linrec_backward(const LinrecArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s) {
#define CALL(TX, TG) launch<TX, TG>(a, tied, vec, s)
    PS_LINREC_DISPATCH(CALL);
#undef CALL
}

}  // namespace ps
