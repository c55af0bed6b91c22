// linrec_forward.cu -- the gated linear recurrence over whole sequences
// (notation and tiles in linrec_common.cuh).
//
// Bound by memory: x and g are read once, h is written once.  Every run is scanned twice in registers, first from 0 for
// what it adds, then from the state before it.
#include "linrec_common.cuh"

namespace ps {

namespace {

// One token: h becomes a h + w x.
template <int V, bool TIED> __device__ __forceinline__ void token(float (&h)[V], const float (&f)[V], const float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = apply(f[v], h[v], TIED ? forgotten(f[v]) * x[v] : x[v]);
}

template <typename TX, typename TG, int V, bool TIED>
__global__ void __launch_bounds__(kLrThreads, 2) linrec_forward_kernel(const LinrecArgs a) {
    __shared__ Marks marks;
    __shared__ Sums<V> sums;
    __shared__ float before[32 * V];
    __shared__ unsigned ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) ticket = a.tiles > 1 ? atomicAdd(a.ticket, 1u) : blockIdx.x;
    __syncthreads();
    const int k = (int)(ticket / (unsigned)a.blocks), block = (int)(ticket % (unsigned)a.blocks);
    const uint32_t n0 = (uint32_t)k * kLinrecTile, first = n0 + warp * kLinrecRun, total = (uint32_t)a.total;
    const long long c0 = (long long)block * (32 * V), ch = c0 + lane * V;
    const bool in = ch < a.channels;

    Lanes<TX, V> x[kLinrecRun];
    Lanes<TG, V> g[kLinrecRun];
    load_run<TG, V>(g, a.g, first, total, (uint32_t)a.tokens, ch, a.channels);
    load_run<TX, V>(x, a.x, first, total, (uint32_t)a.tokens, ch, a.channels);
    mark_tile(marks, a, n0, k == a.tiles - 1, a.h0, a.ht, c0, 32 * V);
    const uint32_t starts = run_bits(marks.start, warp), ends = run_bits(marks.end, warp);
    auto start = [&](float (&h)[V], int i) {
        const float *p = a.h0 + marks.start_seq[warp * kLinrecRun + i] * a.channels + ch;
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = a.h0 && in ? p[v] : 0.f;
    };

    float f[kLinrecRun][V], h[V], s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = s[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kLinrecRun; ++i) {
        float xi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float gi = to_f32<TG>(g[i].v[v]);
            f[i][v] = factor(gi);
            s[v] += gi;
            xi[v] = to_f32<TX>(x[i].v[v]);
        }
        if (starts >> i & 1) start(h, i);
        token<V, TIED>(h, f[i], xi);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sums.s[warp][lane * V + v] = s[v];
        sums.b[warp][lane * V + v] = h[v];
    }
    __syncthreads();
    if (warp == 0) {
        float carry[V];
        tile_carry<V>(carry, a, k, block, sums, [&](int w) { return run_bits(marks.start, w) != 0; }, any_bits(marks.start),
                      (marks.start[0] & 1) == 0, false);
#pragma unroll
        for (int v = 0; v < V; ++v) before[lane * V + v] = carry[v];
        if (a.start != nullptr && in) {
#pragma unroll
            for (int v = 0; v < V; ++v) a.start[k * a.channels + ch + v] = carry[v];
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = before[lane * V + v];
    for (int w = 0; w < warp; ++w) {
        const bool reset = run_bits(marks.start, w) != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = sums.b[w][lane * V + v];
            h[v] = reset ? b : apply(factor_of_sum(sums.s[w][lane * V + v]), h[v], b);
        }
    }
    TX *out = static_cast<TX *>(a.h) + (long long)first * a.channels + ch;
    const uint32_t held = marks.hi > marks.lo ? marks.hi - marks.lo : 0;
#pragma unroll
    for (int i = 0; i < kLinrecRun; ++i) {
        float xi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) xi[v] = to_f32<TX>(x[i].v[v]);
        if (starts >> i & 1) start(h, i);
        token<V, TIED>(h, f[i], xi);
        if (in && first + i - marks.lo < held) store_lanes<TX, V>(out + i * a.channels, h);
        if ((ends >> i & 1) && a.ht != nullptr && in) {
            float *p = a.ht + marks.end_seq[warp * kLinrecRun + i] * a.channels + ch;
#pragma unroll
            for (int v = 0; v < V; ++v) p[v] = h[v];
        }
    }
}

template <typename TX, typename TG> cudaError_t launch(const LinrecArgs &a, bool tied, bool vec, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.tiles * (long long)a.blocks);
    if (vec) {
        if (tied) linrec_forward_kernel<TX, TG, 2, true><<<grid, kLrThreads, 0, s>>>(a);
        else linrec_forward_kernel<TX, TG, 2, false><<<grid, kLrThreads, 0, s>>>(a);
    } else {
        if (tied) linrec_forward_kernel<TX, TG, 1, true><<<grid, kLrThreads, 0, s>>>(a);
        else linrec_forward_kernel<TX, TG, 1, false><<<grid, kLrThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linrec_forward(const LinrecArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s) {
#define CALL(TX, TG) launch<TX, TG>(a, tied, vec, s)
    PS_LINREC_DISPATCH(CALL);
#undef CALL
}

}  // namespace ps
