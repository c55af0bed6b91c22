// beam.cu -- beam search's choice (include/prefix_scan_beam.h).
//
// Two kernels.  The first reads each row of logits once, a part of it a CTA, into registers: the part's maximum and sum of
// exponentials, and its `width` best tokens in order.  The second, a CTA an item, joins the sums of each row's parts, and
// chooses among what the parts offer.  Bound by memory: a logit is read once and costs an exponential.
//
// The best of many, in both: the maxima of 128 groups of numbers are ranked; at least `width` numbers reach the
// width-th largest of them, T, and as a rule few more do.  Those are gathered and ranked one against all.  Where more reach T
// than there is room for (many equal numbers), the best are taken one after the other instead.
//
// How a row is cut into parts, threads and sums goes by places in the row alone, so that equal rows have equal sums.
#include <climits>
#include <cmath>
#include <cstdint>

#include "delta_common.cuh"
#include "prefix_scan_beam.h"
#include "scan_internal.h"

namespace ps {

namespace {

constexpr int kBeamThreads = 512, kBeamWarps = kBeamThreads / 32, kGroups = kBeamThreads / 4;
typedef unsigned long long u64;

struct BeamArgs {
    long long batch, vocab, item_stride, beam_stride;
    int beams, width, eos, parts;
    const void *logits;
    const float *scores;
    const uint8_t *ended;
    float *out_scores;
    int32_t *out_parents, *out_tokens;
    uint8_t *out_ended;
    double *sums;      // [rows, parts]
    float *tops;       // [rows, parts]
    u64 *best;         // [rows, parts, width], 0 where there is none
};

// Numbers as integers that rise with them (NaN apart); -0 as 0.
__device__ __forceinline__ uint32_t rising(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float number_of(uint32_t r) {
    return __uint_as_float(r & 0x80000000u ? r ^ 0x80000000u : ~r);
}
__device__ __forceinline__ u64 rising(double x) {
    const u64 b = (u64)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// The k-th largest of the 128 groups' maxima (-infinity if there are fewer above that).  All threads; `groups` are set.
__device__ __forceinline__ float kth_largest(const float (&groups)[kGroups], int k, float &slot) {
    if (threadIdx.x < kGroups) {
        const float mine = groups[threadIdx.x];
        int above = 0, reach = 0;
#pragma unroll 8
        for (int i = 0; i < kGroups; i += 4) {
            const float4 g = *reinterpret_cast<const float4 *>(&groups[i]);
            above += (g.x > mine) + (g.y > mine) + (g.z > mine) + (g.w > mine);
            reach += (g.x >= mine) + (g.y >= mine) + (g.z >= mine) + (g.w >= mine);
        }
        if (above < k && k <= reach) slot = mine;
    }
    __syncthreads();
    return slot;
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// ---- a part of a row ---------------------------------------------------------------------

// N numbers a thread: 16-byte pieces where the rows allow (VEC numbers each), else one by one; thread t's i-th piece is
// piece i * 512 + t of the part.
template <typename T, int N, int VEC> struct Part {
    static constexpr int kTokens = kBeamThreads * N;
    __device__ static long long token(long long part, int i) {   // of the thread's i-th number
        return part * kTokens + ((long long)(i / VEC) * kBeamThreads + threadIdx.x) * VEC + i % VEC;
    }
};
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Piece { T v[VEC]; };

template <typename T, int N, int VEC>
__global__ void __launch_bounds__(kBeamThreads) beam_part_kernel(const BeamArgs a) {
    typedef Part<T, N, VEC> P;
    __shared__ float tops[kBeamWarps];
    __shared__ double sums[kBeamWarps];
    __shared__ __align__(16) float groups[kGroups];
    __shared__ u64 found[kBeamThreads];
    __shared__ float slot;
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    if ((a.ended != nullptr && a.ended[row] != 0) || !finite(a.scores[row])) return;   // nothing of it is read
    const T *x = static_cast<const T *>(a.logits) + row / a.beams * a.item_stride + row % a.beams * a.beam_stride;
    const float none = __int_as_float(0xff800000);

    Piece<T, VEC> v[N / VEC];
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        const long long t = P::token(part, i);
        if (t + VEC <= a.vocab) {
            v[i / VEC] = *reinterpret_cast<const Piece<T, VEC> *>(x + t);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i / VEC].v[e] = t + e < a.vocab ? x[t + e] : from_f32<T>(none);
        }
    }
    if (tid == 0) {
        count = 0;
        slot = none;
    }
    float top = none;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, to_f32<T>(v[i / VEC].v[i % VEC]));
    {
        const float q = quad_max(top);
        if ((lane & 3) == 0) groups[tid / 4] = q;
        float w = q;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, d));
        if (lane == 0) tops[warp] = w;
    }
    __syncthreads();
    float m = tops[lane % kBeamWarps];
#pragma unroll
    for (int d = 1; d < kBeamWarps; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float t = kth_largest(groups, a.width, slot);

    // the sum of exponentials: 32 bits over a thread's numbers, 64 beyond
    float sum = 0.f;
    const float base = -m * 1.44269504088896341f;   // its rounding is put right at the end
    if (fabsf(m) < 0x1p100f) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(to_f32<T>(v[i / VEC].v[i % VEC]), 1.44269504088896341f, base)));
            sum += e;
        }
    } else {   // the base overflows, or all are -infinity, or NaN among them
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = to_f32<T>(v[i / VEC].v[i % VEC]);
            if (!(y <= none)) sum += exp2f((y - m) * 1.44269504088896341f);
        }
    }
    double s = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) sums[warp] = s;

    auto key = [&](float y, long long token) { return (u64)rising(y) << 32 | (uint32_t)(0xffffffffu - (uint32_t)token); };
    if (top >= t && top > none) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = to_f32<T>(v[i / VEC].v[i % VEC]);
            if (y >= t && y > none) {
                const int at = atomicAdd(&count, 1);
                if (at < kBeamThreads) found[at] = key(y, P::token(part, i));
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        double all = 0.0;
        for (int i = 0; i < kBeamWarps; ++i) all += sums[i];
        if (fabsf(m) < 0x1p100f) all *= exp2(-(double)m * (double)1.44269504088896341f - (double)base);
        a.sums[row * a.parts + part] = all;
        a.tops[row * a.parts + part] = m;
    }
    u64 *best = a.best + (row * a.parts + part) * a.width;
    const int n = count;
    if (n <= kBeamThreads) {
        if (tid < n) {
            const u64 mine = found[tid];
            int rank = 0;
            for (int i = 0; i < n; ++i) rank += found[i] > mine;
            if (rank < a.width) best[rank] = mine;
        } else if (tid < a.width) {
            best[tid] = 0;
        }
        return;
    }
    // one after the other: the largest key below the last one taken
    u64 last = ~0ull;
    for (int k = 0; k < a.width; ++k) {
        u64 mine = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = to_f32<T>(v[i / VEC].v[i % VEC]);
            const u64 z = y > none ? key(y, P::token(part, i)) : 0;
            if (z < last && z > mine) mine = z;
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, d));
        __syncthreads();
        if (lane == 0) found[warp] = mine;
        __syncthreads();
        last = found[lane % kBeamWarps];
#pragma unroll
        for (int d = 1; d < kBeamWarps; d <<= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
        if (tid == 0) best[k] = last;
        if (last == 0) last = 1;   // nothing is below: zeros from here on
    }
}

// ---- an item -----------------------------------------------------------------------------

struct Candidate {
    u64 total, key;
    int beam;
};
__device__ __forceinline__ bool before(const Candidate &x, const Candidate &y) {
    if (x.total != y.total) return x.total > y.total;
    return x.beam != y.beam ? x.beam < y.beam : x.key > y.key;
}

__global__ void __launch_bounds__(kBeamThreads) beam_item_kernel(const BeamArgs a) {
    __shared__ double log_sum[PS_BEAM_MAX_BEAMS];   // of exp(logit - top)
    __shared__ float near_log[PS_BEAM_MAX_BEAMS], largest[PS_BEAM_MAX_BEAMS], score[PS_BEAM_MAX_BEAMS];
    __shared__ uint8_t ended[PS_BEAM_MAX_BEAMS];
    __shared__ __align__(16) float groups[kGroups];
    __shared__ Candidate found[kBeamThreads];
    __shared__ float slot, sizes[kBeamWarps];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long item = blockIdx.x;
    const float none = __int_as_float(0xff800000);
    if (tid == 0) {
        count = 0;
        slot = none;
    }
    for (int b = warp; b < a.beams; b += kBeamWarps) {
        const long long row = item * a.beams + b;
        const float sc = a.scores[row];
        const bool end = a.ended != nullptr && a.ended[row] != 0;
        double all = __longlong_as_double(0x7ff8000000000000ll), l = all;   // NaN: offers nothing
        float m = none;
        if (finite(sc) && !end) {
            for (int i = lane; i < a.parts; i += 32) m = fmaxf(m, a.tops[row * a.parts + i]);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            all = 0.0;
            for (int i = lane; i < a.parts; i += 32) {
                const float t = a.tops[row * a.parts + i];
                const double s = a.sums[row * a.parts + i];
                all += t == m || s != s ? s : s * exp((double)t - (double)m);
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
            l = log(all);
        }
        if (lane == 0) {
            log_sum[b] = l;
            near_log[b] = (float)l;
            largest[b] = m;
            score[b] = sc;
            ended[b] = end && finite(sc);
        }
    }
    __syncthreads();

    // A candidate is a place in the parts' lists; an ended beam's is the first of its places.
    const int per_beam = a.parts * a.width;
    const long long places = (long long)a.beams * per_beam;
    const u64 *best = a.best + item * places;
    struct Place {
        int beam;
        u64 key;
        bool there;
    };
    auto place = [&](long long c) {
        Place p;
        p.beam = (int)(c / per_beam);
        p.there = ended[p.beam] ? c % per_beam == 0 : near_log[p.beam] == near_log[p.beam];
        p.key = p.there && !ended[p.beam] ? best[c] : 0;
        p.there = p.there && (ended[p.beam] || p.key != 0);
        return p;
    };
    auto near_total = [&](const Place &p) {
        return ended[p.beam] ? score[p.beam]
                             : score[p.beam] + ((number_of((uint32_t)(p.key >> 32)) - largest[p.beam]) - near_log[p.beam]);
    };
    auto candidate = [&](const Place &p) {
        const double t = ended[p.beam] ? (double)score[p.beam]
                                       : (double)score[p.beam] + (((double)number_of((uint32_t)(p.key >> 32)) - (double)largest[p.beam]) -
                                                                      log_sum[p.beam]);
        return Candidate{rising(t), p.key, p.beam};
    };
    // T from totals of 32 bits, each off by at most 2^-23 of the magnitudes that it is made of; what is gathered reaches T less
    // 2^-20 of the largest
    float top = none, size = 0.f;
    for (long long c = tid; c < places; c += kBeamThreads) {
        const Place p = place(c);
        if (!p.there) continue;
        top = fmaxf(top, near_total(p));
        size = fmaxf(size, fabsf(score[p.beam]) + (ended[p.beam] ? 0.f : largest[p.beam] - number_of((uint32_t)(p.key >> 32)) + fabsf(near_log[p.beam])));
    }
    {
        const float q = quad_max(top);
        if ((lane & 3) == 0) groups[tid / 4] = q;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
        if (lane == 0) sizes[warp] = size;
    }
    __syncthreads();
    size = sizes[lane % kBeamWarps];
#pragma unroll
    for (int d = 1; d < kBeamWarps; d <<= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
    const float t = kth_largest(groups, a.width, slot) - size * 0x1p-20f;
    if (top >= t) {
        for (long long c = tid; c < places; c += kBeamThreads) {
            const Place p = place(c);
            if (p.there && near_total(p) >= t) {
                const int at = atomicAdd(&count, 1);
                if (at < kBeamThreads) found[at] = candidate(p);
            }
        }
    }
    __syncthreads();
    const int n = count;
    auto take = [&](int rank, const Candidate &c) {
        const long long to = item * a.width + rank;
        const bool end = ended[c.beam];
        const int32_t token = end ? a.eos : (int32_t)(0xffffffffu - (uint32_t)c.key);
        const u64 b = c.total >> 63 ? c.total ^ 1ull << 63 : ~c.total;
        a.out_scores[to] = (float)__longlong_as_double((long long)b);
        a.out_parents[to] = (int32_t)(item * a.beams + c.beam);
        a.out_tokens[to] = token;
        if (a.out_ended) a.out_ended[to] = end || (a.eos >= 0 && token == a.eos);
    };
    auto leave = [&](int rank) {
        const long long to = item * a.width + rank;
        a.out_scores[to] = none;
        a.out_parents[to] = a.out_tokens[to] = -1;
        if (a.out_ended) a.out_ended[to] = 0;
    };
    if (n <= kBeamThreads) {
        if (tid < n) {
            const Candidate mine = found[tid];
            int rank = 0;
            for (int i = 0; i < n; ++i) rank += before(found[i], mine);
            if (rank < a.width) take(rank, mine);
        } else if (tid < a.width) {
            leave(tid);
        }
        return;
    }
    // one after the other
    __syncthreads();
    Candidate last{~0ull, ~0ull, -1};
    for (int k = 0; k < a.width; ++k) {
        Candidate mine{0, 0, INT_MAX};
        for (long long c = tid; c < places; c += kBeamThreads) {
            const Place p = place(c);
            if (!p.there) continue;
            const Candidate z = candidate(p);
            if (before(last, z) && before(z, mine)) mine = z;
        }
        auto better = [&](int d) {
            Candidate y;
            y.total = __shfl_xor_sync(0xffffffffu, mine.total, d);
            y.key = __shfl_xor_sync(0xffffffffu, mine.key, d);
            y.beam = __shfl_xor_sync(0xffffffffu, mine.beam, d);
            if (before(y, mine)) mine = y;
        };
        for (int d = 1; d < 32; d <<= 1) better(d);
        __syncthreads();
        if (lane == 0) found[warp] = mine;
        __syncthreads();
        mine = found[lane % kBeamWarps];
        for (int d = 1; d < kBeamWarps; d <<= 1) better(d);
        if (tid == 0) {
            if (mine.total != 0) take(k, mine);
            else leave(k);
        }
        last = mine;
    }
}

// ---- host --------------------------------------------------------------------------------

// Numbers of a thread: 32 KiB of logits a CTA, or 8 where rows are few, so that more SMs read them.
template <typename T> constexpr int big() { return 64 / (int)sizeof(T); }
long long part_tokens(const ps_beam_shape *d) {
    const int es = d->type == PS_REAL_F32 ? 4 : 2, most = 64 / es;
    const long long rows = d->batch * d->beams;
    const bool few = rows * ((d->vocab + kBeamThreads * most - 1) / (kBeamThreads * most)) < 152;
    return (long long)kBeamThreads * (few ? 16 / es : most);
}

template <typename T, int VEC> cudaError_t launch(const BeamArgs &a, bool few, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.batch * a.beams * a.parts);
    if (few) beam_part_kernel<T, 16 / sizeof(T), VEC><<<grid, kBeamThreads, 0, s>>>(a);
    else beam_part_kernel<T, 64 / sizeof(T), VEC><<<grid, kBeamThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        beam_item_kernel<<<(unsigned)a.batch, kBeamThreads, 0, s>>>(a);
        e = cudaGetLastError();
    }
    return e;
}
template <typename T> cudaError_t launch(const BeamArgs &a, bool few, bool pieces, cudaStream_t s) {
    return pieces ? launch<T, 16 / sizeof(T)>(a, few, s) : launch<T, 1>(a, few, s);
}

struct Bytes {
    uintptr_t a, b;
};
Bytes span(const void *p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + bytes : a};
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
bool valid(const ps_beam_shape *d) {
    if (d == nullptr || (d->type != PS_REAL_F32 && d->type != PS_REAL_BF16 && d->type != PS_REAL_F16)) return false;
    if (d->batch < 0 || d->beams < 1 || d->beams > PS_BEAM_MAX_BEAMS || d->width < 1 || d->width > PS_BEAM_MAX_WIDTH) return false;
    if (d->vocab < 1 || d->vocab > INT_MAX - 65536 || d->eos_token < -1) return false;
    if (d->batch > INT_MAX / d->beams || d->batch > INT_MAX / d->width) return false;
    const long long tokens = part_tokens(d);
    return d->batch * d->beams <= INT_MAX / ((d->vocab + tokens - 1) / tokens);
}
struct Parts {
    long long parts;
    size_t sums, tops, best, total;
};
Parts parts_of(const ps_beam_shape *d) {
    Parts p;
    const long long tokens = part_tokens(d);
    p.parts = (d->vocab + tokens - 1) / tokens;
    const size_t n = (size_t)(d->batch * d->beams * p.parts);
    p.sums = 0;
    p.tops = up(n * 8);
    p.best = p.tops + up(n * 4);
    p.total = p.best + up(n * (size_t)d->width * 8);
    return p;
}

}  // namespace

}  // namespace ps

using namespace ps;

extern "C" size_t ps_beam_workspace_size(const ps_beam_shape *d) {
    if (!valid(d) || d->batch == 0) return 0;
    return parts_of(d).total;
}

extern "C" ps_status ps_beam_select(const ps_beam_shape *d, const void *logits, const float *scores, const uint8_t *ended,
                                    float *out_scores, int32_t *out_parents, int32_t *out_tokens, uint8_t *out_ended, void *ws,
                                    size_t ws_bytes, ps_stream_t stream) {
    if (!valid(d)) return PS_ERR_INVALID_ARG;
    if (d->batch == 0) return PS_OK;
    const size_t es = d->type == PS_REAL_F32 ? 4 : 2;
    auto on = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    if (logits == nullptr || scores == nullptr || out_scores == nullptr || out_parents == nullptr || out_tokens == nullptr || ws == nullptr)
        return PS_ERR_INVALID_ARG;
    if (!on(logits, es) || !on(scores, 4) || !on(out_scores, 4) || !on(out_parents, 4) || !on(out_tokens, 4) || !on(ws, 256))
        return PS_ERR_INVALID_ARG;
    const Parts p = parts_of(d);
    if (ws_bytes < p.total) return PS_ERR_WORKSPACE_TOO_SMALL;
    const size_t rows = (size_t)(d->batch * d->beams), picks = (size_t)(d->batch * d->width);
    int64_t lo = 0, hi = 0;
    (d->item_stride < 0 ? lo : hi) += d->item_stride * (d->batch - 1);
    (d->beam_stride < 0 ? lo : hi) += d->beam_stride * (d->beams - 1);
    const uintptr_t x = reinterpret_cast<uintptr_t>(logits);
    const Bytes in[] = {{x + lo * (int64_t)es, x + (hi + d->vocab) * (int64_t)es}, span(scores, rows * 4), span(ended, rows)};
    const Bytes out[] = {span(out_scores, picks * 4), span(out_parents, picks * 4), span(out_tokens, picks * 4), span(out_ended, picks),
                        span(ws, p.total)};
    for (int i = 0; i < 5; ++i) {
        for (int j = i + 1; j < 5; ++j)
            if (out[i].a < out[j].b && out[j].a < out[i].b) return PS_ERR_OVERLAP;
        for (const Bytes &y : in)
            if (out[i].a < y.b && y.a < out[i].b) return PS_ERR_OVERLAP;
    }
    unsigned char *w = static_cast<unsigned char *>(ws);
    BeamArgs a{};
    a.batch = d->batch;
    a.vocab = d->vocab;
    a.item_stride = d->item_stride;
    a.beam_stride = d->beam_stride;
    a.beams = d->beams;
    a.width = d->width;
    a.eos = d->eos_token;
    a.parts = (int)p.parts;
    a.logits = logits;
    a.scores = scores;
    a.ended = ended;
    a.out_scores = out_scores;
    a.out_parents = out_parents;
    a.out_tokens = out_tokens;
    a.out_ended = out_ended;
    a.sums = reinterpret_cast<double *>(w + p.sums);
    a.tops = reinterpret_cast<float *>(w + p.tops);
    a.best = reinterpret_cast<u64 *>(w + p.best);
    const bool few = part_tokens(d) * (long long)es == kBeamThreads * 16ll;
    const bool pieces = on(logits, 16) && (d->batch == 1 || d->item_stride * (int64_t)es % 16 == 0) &&
                        (d->beams == 1 || d->beam_stride * (int64_t)es % 16 == 0);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = d->type == PS_REAL_F32    ? launch<float>(a, few, pieces, s)
                          : d->type == PS_REAL_BF16 ? launch<__nv_bfloat16>(a, few, pieces, s)
                                                    : launch<__half>(a, few, pieces, s);
    if (e == cudaSuccess) return PS_OK;
    note_cuda_error(e);
    return PS_ERR_CUDA;
}
