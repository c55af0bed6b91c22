// linrec_step.cu -- the gated linear recurrence for the next token or few, on
// states in a pool of pages (notation in linrec_common.cuh).
//
// Bound by memory: a state is read once and written once, whatever the number of tokens.  A thread holds some groups of V
// neighbouring channels, whose loads are under way together, and those of the first token before the page is known.
//
// Many channels: four groups a thread, of one sequence.  4096 sequences of 8192 bf16 channels: 70 us, 6.7 TB/s (two groups: 74 us,
// one: 73; 64 sequences of 4096 channels, which one group spreads over more SMs, 2.0 against 1.8 us).
// Few channels, up to the 256 groups of a CTA: two groups a thread, of as many sequences as the CTA can hold.  196170 sequences of
// 104 channels: 57 us, 5.7 TB/s (a CTA a sequence: 231), 20000 of 704: 40 (44).  For many channels this takes more registers and
// addresses than it is worth: 82 instead of 70 us of the first.
#include "linrec_common.cuh"

namespace ps {

namespace {

constexpr int kStepThreads = 128, kGroups = 4, kNarrowGroups = 2;

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
                    const Token t = Token::of<kWeights<TX, TIED>>(make_float2(to_f32<TG>(gi[k].v[v]), to_f32<TG>(gi[k].v[v + N])));
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

// Sequences of few channels: as many of them a CTA as are whole in it.
struct Spread {
    uint32_t each, together, factor;   // groups of a sequence, sequences of a CTA; x * factor / 2^20 is x / each for x < 512
};

template <typename TX, typename TG, int V, bool TIED>
__global__ void __launch_bounds__(kStepThreads) linrec_step_narrow_kernel(const LinrecStepArgs a, const Spread d) {
    long long seq[kNarrowGroups], ch[kNarrowGroups];
    int count[kNarrowGroups];
    bool in[kNarrowGroups];
    Wide<TX, V> xi[kNarrowGroups];
    Wide<TG, V> gi[kNarrowGroups];
    Wide<float, V> h[kNarrowGroups];
    float *state[kNarrowGroups];
#pragma unroll
    for (int k = 0; k < kNarrowGroups; ++k) {
        const uint32_t l = k * kStepThreads + threadIdx.x, r = l * d.factor >> 20, group = l - r * d.each;
        seq[k] = (long long)blockIdx.x * d.together + r;
        ch[k] = (long long)group * V;
        in[k] = r < d.together && seq[k] < a.seqs;
    }
    auto load = [&](int k, long long i) {
        xi[k] = *reinterpret_cast<const Wide<TX, V> *>(static_cast<const TX *>(a.x.p) + seq[k] * a.x.seq + i * a.x.tok + ch[k]);
        gi[k] = *reinterpret_cast<const Wide<TG, V> *>(static_cast<const TG *>(a.g.p) + seq[k] * a.g.seq + i * a.g.tok + ch[k]);
    };
#pragma unroll
    for (int k = 0; k < kNarrowGroups; ++k)
        if (in[k]) load(k, 0);   // on their way while the pages are found
#pragma unroll
    for (int k = 0; k < kNarrowGroups; ++k) {
        const long long page = !in[k] ? -1 : a.slots ? a.slots[seq[k]] : seq[k];
        const int n = in[k] && a.lengths ? a.lengths[seq[k]] : a.t;
        count[k] = page < 0 || page >= a.pages || n < 0 ? 0 : n > a.t ? a.t : n;
        state[k] = a.state + page * a.channels + ch[k];
    }
#pragma unroll
    for (int k = 0; k < kNarrowGroups; ++k)
        if (count[k] > 0) h[k] = *reinterpret_cast<const Wide<float, V> *>(state[k]);
    for (int i = 0; i < a.t; ++i) {
        if (i > 0) {
#pragma unroll
            for (int k = 0; k < kNarrowGroups; ++k)
                if (i < count[k]) load(k, i);
        }
#pragma unroll
        for (int k = 0; k < kNarrowGroups; ++k) {
            if (!in[k]) continue;
            Wide<TX, V> o;
            if (i < count[k]) {
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    constexpr int N = V > 1;   // a channel alone takes the place of both
                    const Token t = Token::of<kWeights<TX, TIED>>(make_float2(to_f32<TG>(gi[k].v[v]), to_f32<TG>(gi[k].v[v + N])));
                    const float2 y = make_float2(to_f32<TX>(xi[k].v[v]), to_f32<TX>(xi[k].v[v + N]));
                    const float2 next = t.apply(make_float2(h[k].v[v], h[k].v[v + N]), t.weigh(y, TIED));
                    h[k].v[v] = next.x;
                    h[k].v[v + N] = next.y;
                    o.v[v] = from_f32<TX>(next.x);
                    o.v[v + N] = from_f32<TX>(next.y);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) o.v[v] = from_f32<TX>(0.f);
            }
            *reinterpret_cast<Wide<TX, V> *>(static_cast<TX *>(a.h) + (seq[k] * a.t + i) * a.channels + ch[k]) = o;
        }
    }
#pragma unroll
    for (int k = 0; k < kNarrowGroups; ++k)
        if (count[k] > 0) *reinterpret_cast<Wide<float, V> *>(state[k]) = h[k];
}

template <typename TX, typename TG, int V, bool TIED> cudaError_t launch(const LinrecStepArgs &a, cudaStream_t s) {
    const long long each = a.channels / V;
    if (each <= kStepThreads * kNarrowGroups) {
        const uint32_t together = kStepThreads * kNarrowGroups / (uint32_t)each;
        const Spread d{(uint32_t)each, together, (1u << 20) / (uint32_t)each + 1};
        linrec_step_narrow_kernel<TX, TG, V, TIED><<<(unsigned)((a.seqs + together - 1) / together), kStepThreads, 0, s>>>(a, d);
    } else {
        const int blocks = (int)((each + kStepThreads * kGroups - 1) / (kStepThreads * kGroups));
        linrec_step_kernel<TX, TG, V, TIED><<<(unsigned)(a.seqs * blocks), kStepThreads, 0, s>>>(a, blocks);
    }
    return cudaGetLastError();
}
template <typename TX, typename TG> cudaError_t launch(const LinrecStepArgs &a, bool tied, bool vec, cudaStream_t s) {
    if (vec) return tied ? launch<TX, TG, 4, true>(a, s) : launch<TX, TG, 4, false>(a, s);
    return tied ? launch<TX, TG, 1, true>(a, s) : launch<TX, TG, 1, false>(a, s);
}

}  // namespace

cudaError_t launch_linrec_step(const LinrecStepArgs &a, int type, int gate_type, bool tied, bool vec, cudaStream_t s) {
#define CALL(TX, TG) launch<TX, TG>(a, tied, vec, s)
    PS_LINREC_DISPATCH(CALL);
#undef CALL
}

}  // namespace ps
