// linrec_step.cu -- the gated linear recurrence for the next token or few, on
// states in a pool of pages (notation in linrec_common.cuh).
//
// Bound by memory: a state is read once and written once, whatever the number of tokens.  A thread holds V neighbouring
// channels of a sequence.
#include "linrec_common.cuh"

namespace ps {

namespace {

constexpr int kStepThreads = 128;

template <typename T, int V> struct alignas(sizeof(T) * V) Wide { T v[V]; };

template <typename TX, typename TG, int V, bool TIED>
__global__ void __launch_bounds__(kStepThreads) linrec_step_kernel(const LinrecStepArgs a, const int blocks) {
    const long long seq = blockIdx.x / blocks;
    const long long ch = ((long long)(blockIdx.x % blocks) * kStepThreads + threadIdx.x) * V;
    if (ch >= a.channels) return;
    const long long page = a.slots ? a.slots[seq] : seq;
    int count = a.lengths ? a.lengths[seq] : a.t;
    count = count < 0 ? 0 : count > a.t ? a.t : count;
    if (page < 0 || page >= a.pages) count = 0;
    const TX *x = static_cast<const TX *>(a.x.p) + seq * a.x.seq + ch;
    const TG *g = static_cast<const TG *>(a.g.p) + seq * a.g.seq + ch;
    TX *out = static_cast<TX *>(a.h) + seq * a.t * a.channels + ch;
    if (count > 0) {
        float *state = a.state + page * a.channels + ch;
        Wide<float, V> h = *reinterpret_cast<const Wide<float, V> *>(state);
        for (long long i = 0; i < count; ++i) {
            const Wide<TX, V> xi = *reinterpret_cast<const Wide<TX, V> *>(x + i * a.x.tok);
            const Wide<TG, V> gi = *reinterpret_cast<const Wide<TG, V> *>(g + i * a.g.tok);
            Wide<TX, V> o;
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                constexpr int N = V > 1;   // a channel alone takes the place of both
                const Token t = Token::of(make_float2(to_f32<TG>(gi.v[v]), to_f32<TG>(gi.v[v + N])));
                const float2 y = make_float2(to_f32<TX>(xi.v[v]), to_f32<TX>(xi.v[v + N]));
                const float2 next = t.apply(make_float2(h.v[v], h.v[v + N]), t.weigh(y, TIED));
                h.v[v] = next.x;
                h.v[v + N] = next.y;
                o.v[v] = from_f32<TX>(next.x);
                o.v[v + N] = from_f32<TX>(next.y);
            }
            *reinterpret_cast<Wide<TX, V> *>(out + i * a.channels) = o;
        }
        *reinterpret_cast<Wide<float, V> *>(state) = h;
    }
    Wide<TX, V> zero;
#pragma unroll
    for (int v = 0; v < V; ++v) zero.v[v] = from_f32<TX>(0.f);
    for (long long i = count; i < a.t; ++i) *reinterpret_cast<Wide<TX, V> *>(out + i * a.channels) = zero;
}

template <typename TX, typename TG> cudaError_t launch(const LinrecStepArgs &a, bool tied, bool vec, cudaStream_t s) {
    const int per = kStepThreads * (vec ? 4 : 1);
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
