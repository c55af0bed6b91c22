// linrec_step.cu -- the gated linear recurrence for the next token or few, on
// states in a pool of pages (notation in linrec_common.cuh).
//
// Bound by memory: a state is read once and written once, whatever the number of tokens.  A thread holds four groups of V
// neighbouring channels of a sequence, whose loads are under way together, and those of the first token
// before the page is known.  4096 sequences of 8192 bf16 channels: 70 us, 6.7 TB/s (two groups: 74 us, one: 73, and 64 sequences of
// 4096 channels, which one group spreads over more SMs, 2.0 against 1.8 us).
#include "linrec_common.cuh"

namespace ps {

namespace {

constexpr int kStepThreads = 128, kGroups = 4;

template <typename T, int V> struct alignas(sizeof(T) * V) Wide { T v[V]; };

template <typename TX, typename TG, int V, bool TIED>
__global__ void __launch_bounds__(kStepThreads) linrec_step_kernel(const LinrecStepArgs a, const int blocks) {
    const long long seq = blockIdx.x / (uint32_t)blocks;
    long long ch[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
        ch[k] = ((blockIdx.x - seq * blocks) * kGroups + k) * kStepThreads * V + threadIdx.x * V;
    const TX *x = static_cast<const TX *>(a.x.p) + seq * a.x.seq;
    const TG *g = static_cast<const TG *>(a.g.p) + seq * a.g.seq;
    TX *out = static_cast<TX *>(a.h) + seq * a.t * a.channels;
    Wide<TX, V> xi[kGroups];
    Wide<TG, V> gi[kGroups];
    Wide<float, V> h[kGroups];
    auto load = [&](long long i) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
            if (ch[k] < a.channels) {
                xi[k] = *reinterpret_cast<const Wide<TX, V> *>(x + i * a.x.tok + ch[k]);
                gi[k] = *reinterpret_cast<const Wide<TG, V> *>(g + i * a.g.tok + ch[k]);
            }
    };
    load(0);   // on their way while the page is found
    const long long page = a.slots ? a.slots[seq] : seq;
    int count = a.lengths ? a.lengths[seq] : a.t;
    count = count < 0 ? 0 : count > a.t ? a.t : count;
    if (page < 0 || page >= a.pages) count = 0;
    if (count > 0) {
        float *state = a.state + page * a.channels;
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
            if (ch[k] < a.channels) h[k] = *reinterpret_cast<const Wide<float, V> *>(state + ch[k]);
        for (long long i = 0; i < count; ++i) {
            if (i > 0) load(i);
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                if (ch[k] >= a.channels) continue;
                Wide<TX, V> o;
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    constexpr int N = V > 1;   // a channel alone takes the place of both
                    const Token t = Token::of(make_float2(to_f32<TG>(gi[k].v[v]), to_f32<TG>(gi[k].v[v + N])));
                    const float2 y = make_float2(to_f32<TX>(xi[k].v[v]), to_f32<TX>(xi[k].v[v + N]));
                    const float2 next = t.apply(make_float2(h[k].v[v], h[k].v[v + N]), t.weigh(y, TIED));
                    h[k].v[v] = next.x;
                    h[k].v[v + N] = next.y;
                    o.v[v] = from_f32<TX>(next.x);
                    o.v[v + N] = from_f32<TX>(next.y);
                }
                *reinterpret_cast<Wide<TX, V> *>(out + i * a.channels + ch[k]) = o;
            }
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
            if (ch[k] < a.channels) *reinterpret_cast<Wide<float, V> *>(state + ch[k]) = h[k];
    }
    Wide<TX, V> zero;
#pragma unroll
    for (int v = 0; v < V; ++v) zero.v[v] = from_f32<TX>(0.f);
    for (long long i = count; i < a.t; ++i)
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
            if (ch[k] < a.channels) *reinterpret_cast<Wide<TX, V> *>(out + i * a.channels + ch[k]) = zero;
}

template <typename TX, typename TG> cudaError_t launch(const LinrecStepArgs &a, bool tied, bool vec, cudaStream_t s) {
    const int per = kStepThreads * kGroups * (vec ? 4 : 1);
    const int blocks = (int)((a.channels + per - 1) / per);
    const unsigned grid = (unsigned)(a.seqs * blocks);
    if (vec) {
        if (tied) linrec_step_kernel<TX, TG, 4, true><<<grid, kStepThreads, 0, s>>>(a, blocks);
        else linrec_step_kernel<TX, TG, 4, false><<<grid, kStepThreads, 0, s>>>(a, blocks);
    } else {
        if (tied) linrec_step_kernel<TX, TG, 1, true><<<grid, kStepThreads, 0, s>>>(a, blocks);
        else linrec_step_kernel<TX, TG, 1, false><<<grid, kStepThreads, 0, s>>>(a, blocks);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linrec_step(const LinrecStepArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s) {
#define CALL(TX, TG) launch<TX, TG>(a, tied, vec, s)
    PS_LINREC_DISPATCH(CALL);
#undef CALL
}

}  // namespace ps
