// beam.cu -- beam search's choice (include/prefix_scan_beam.h).
//
// Two kernels.  The first reads each row of logits once, a part of it a CTA, into registers: the part's maximum and sum of
// exponentials, and its `width` best tokens in order.  The second, a CTA an item, joins the sums of each row's parts, and
// chooses among what the parts' lists offer.
//
// The best of many, in both: some numbers are ranked (of a part's the maxima of 32 groups, 128 where the width is above 16; of
// the lists' entries those of 512); at least `width` numbers reach the width-th largest of these, T, and as a rule few more
// do.  Those are gathered and ranked one against all.  Where more reach T than there is room for (many equal numbers, say), the
// best are taken one after the other instead.
//
// Memory bounds it from below (a logit is read once); in fact a part's chain of loads, barriers and shuffles does, which five
// other CTAs on its SM cover in part (two thirds of the issue slots are in use).  A pair of 16-bit logits takes six instructions for its exponentials, two for the maximum
// and three to see whether it reaches T, and a warp some 250 besides for its 1024 logits.  64 x 8 beams over 128000 bf16 logits
// (131 MB, of which a fifth, at their end, is not read): parts 33 us (105 MB, 3.2 TB/s; five CTAs an SM instead of the six that 40 registers allow: 41 instead of
// 35; T found by one warp in steps of a bit: 35; parts twice as long, on four CTAs: 37; parts to come fetched into L2: no
// difference), items 9 us.  12 x 16 beams over 50021 f16 logits with 32 candidates: 14 and 15 us (128 groups against 32: 14 us
// against 25, as 37 instead of 110 numbers reach T; 512 threads an item against 256: 15 against 17).
//
// How a row is cut into parts, threads and sums goes by places in the row alone, so that equal rows have equal sums.  A row's
// logarithm of the sum of exponentials is off by 2^-19 at most and by 2^-22 or so as a rule: an exponential by 2^-22 of itself (and
// 2^-25.4 by its argument), a part's sum by 17 roundings of 2^-24, its share in the row's by 2^-22, the logarithm by 2^-23; the
// parts' shares are added, and totals compared, in 64 bits.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "delta_common.cuh"
#include "prefix_scan_beam.h"
#include "scan_internal.h"

namespace ps {

namespace {

constexpr int kPartThreads = 256, kPartWarps = kPartThreads / 32, kItemThreads = 512, kItemWarps = kItemThreads / 32;

constexpr int kRoom = 512;                             // candidates that are ranked one against all
constexpr int kFewGroups = 32, kMostGroups = 128;      // of numbers: as many as the width at least
typedef unsigned long long u64;

// Division of numbers below 2^31: a multiplication, as divisions would be a tenth of a part's instructions.
struct Divisor {
    uint32_t factor, shift;
};
Divisor divisor(uint32_t d) {   // d < 2^31: s the least with 2^s >= d, then factor = ceil(2^(31 + s) / d) < 2^32 is off by less than
    uint32_t s = 0;             // 2^s / d parts in 2^31 of what it should be, and x < 2^31
    while ((1ull << s) < d) ++s;
    return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s};
}
__device__ __forceinline__ uint32_t operator/(uint32_t x, Divisor d) { return (uint32_t)((u64)x * d.factor >> 31 >> d.shift); }

struct BeamArgs {
    long long batch, vocab, item_stride, beam_stride, part_tokens;
    int beams, width, eos, parts;
    Divisor by_parts, by_beams, by_list;   // by_list: parts * width
    const void *logits;
    const float *scores;
    const uint8_t *ended;
    float *out_scores;
    int32_t *out_parents, *out_tokens;
    uint8_t *out_ended;
    float *sums;       // [rows, parts]: of 2^(x log2 e + base_of(top))
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

// Of a warp's share of N numbers in shared memory (a WARPS-th), the least that fewer than k of all N exceed, as an integer that
// rises with it; ~0 if there is none.  The least of all warps' is the k-th largest number.
template <int N, int WARPS> __device__ __forceinline__ uint32_t reached_by(const float *x, int k) {
    constexpr int LANES = 32 * WARPS / N;   // that compare a number with all
    const int lane = threadIdx.x & 31;
    const float mine = x[(threadIdx.x >> 5) * (N / WARPS) + lane / LANES];
    int above = 0;
#pragma unroll
    for (int i = 0; i < N; i += 4 * LANES) {
        const float4 y = *reinterpret_cast<const float4 *>(&x[i + lane % LANES * 4]);
        above += (y.x > mine) + (y.y > mine) + (y.z > mine) + (y.w > mine);
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) above += __shfl_xor_sync(0xffffffffu, above, d);
    return __reduce_min_sync(0xffffffffu, above < k ? rising(mine) : 0xffffffffu);
}

// ---- a part of a row ---------------------------------------------------------------------

// N numbers a thread: 16-byte pieces where the rows allow (VEC numbers each), else one by one; thread t's i-th piece is
// piece i * 256 + t of the part.
template <int VEC> __device__ __forceinline__ int place_in_part(int i) {   // of the thread's i-th number
    return (i / VEC * kPartThreads + (int)threadIdx.x) * VEC + i % VEC;
}

// A thread's numbers as words, two to a word for 16-bit types.
template <typename T> __device__ __forceinline__ float2 pair_of(const uint32_t *w, int i);   // numbers 2 i and 2 i + 1
template <> __device__ __forceinline__ float2 pair_of<float>(const uint32_t *w, int i) {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}
template <> __device__ __forceinline__ float2 pair_of<__nv_bfloat16>(const uint32_t *w, int i) {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 pair_of<__half>(const uint32_t *w, int i) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
}
// The larger numbers of two words.
template <typename T> __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t larger<float>(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
template <> __device__ __forceinline__ uint32_t larger<__nv_bfloat16>(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <> __device__ __forceinline__ uint32_t larger<__half>(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
// Whether number 2 i or 2 i + 1 is at least t, itself a number of type T.
template <typename T> __device__ __forceinline__ bool either_reaches(const uint32_t *w, int i, float t) {
    const float2 y = pair_of<T>(w, i);
    return y.x >= t || y.y >= t;
}
template <> __device__ __forceinline__ bool either_reaches<__nv_bfloat16>(const uint32_t *w, int i, float t) {
    return __hge2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), __float2bfloat162_rn(t)) != 0;
}
template <> __device__ __forceinline__ bool either_reaches<__half>(const uint32_t *w, int i, float t) {
    return __hge2_mask(*reinterpret_cast<const __half2 *>(&w[i]), __float2half2_rn(t)) != 0;
}
template <typename T> __device__ __forceinline__ uint32_t bits_of(T x) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(x);
    else return *reinterpret_cast<const unsigned short *>(&x);
}
// Number i becomes x (words start as 0).
template <typename T> __device__ __forceinline__ void set_number(uint32_t *w, int i, T x) {
    if (sizeof(T) == 4) w[i] = bits_of(x);
    else w[i / 2] |= bits_of(x) << (16 * (i & 1));
}
// 2^(x log2 e + base)
__device__ __forceinline__ float2 exps_of(float2 x, float base) {
    float2 y, e;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(y.x), "=f"(y.y) : "f"(x.x), "f"(x.y), "f"(1.44269504088896341f), "f"(base));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
    return e;
}

// What is added to x log2 e for the exponentials of a part whose largest number is m, rounded to 32 bits.  Of no
// use where all numbers are -infinity (or NaN), or where what the rounding leaves would overflow the exponentials.
__device__ __forceinline__ bool base_is_used(float m) { return fabsf(m) < 0x1p20f; }
__device__ __forceinline__ float base_of(float m) { return -m * 1.44269504088896341f; }

// Numbers are taken out of their words again for what follows: kept apart they would not fit into registers.
template <int W> __device__ __forceinline__ void again(uint32_t (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

template <typename T, int N, int VEC>
__global__ void __launch_bounds__(kPartThreads, 6) beam_part_kernel(const BeamArgs a) {
    __shared__ float tops[kPartWarps], sums[kPartWarps];
    __shared__ __align__(16) float groups[kMostGroups];
    __shared__ u64 found[kRoom];
    __shared__ int count;
    __shared__ uint32_t reach[kPartWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row = blockIdx.x / a.by_parts, part = blockIdx.x - row * a.parts, item = row / a.by_beams;
    if ((a.ended != nullptr && a.ended[row] != 0) || !finite(a.scores[row])) return;   // nothing of it is read
    const T *x = static_cast<const T *>(a.logits) + item * a.item_stride + (row - item * a.beams) * a.beam_stride;
    const float none = __int_as_float(0xff800000);

    constexpr int WORDS = N * (int)sizeof(T) / 4;
    const long long first = part * a.part_tokens;
    const int here = (int)min(a.part_tokens, a.vocab - first);
    x += first;
    const uint32_t empty = bits_of(from_f32<T>(none)) * (sizeof(T) == 4 ? 1u : 0x10001u);
    uint32_t v[WORDS];
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        const int at = place_in_part<VEC>(i);
        if (VEC > 1) {
            const int w = i * WORDS / N;
            uint4 y = make_uint4(empty, empty, empty, empty);
            if (at + VEC <= here) y = __ldcs(reinterpret_cast<const uint4 *>(x + at));
            v[w] = y.x; v[w + 1] = y.y; v[w + 2] = y.z; v[w + 3] = y.w;
        } else {
            if ((i * WORDS) % N == 0) v[i * WORDS / N] = 0;
            set_number<T>(v, i, at < here ? x[at] : from_f32<T>(none));
        }
    }
    if (VEC > 1 && here % VEC != 0 && (here / VEC) % kPartThreads == tid) {   // the row's last piece is not whole: one thread's
#pragma unroll
        for (int i = 0; i < N; i += VEC) {
            const int at = place_in_part<VEC>(i);
            if (at < here && at + VEC > here) {
                asm volatile("" ::: "memory");
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (((i + e) * WORDS) % N == 0) v[(i + e) * WORDS / N] = 0;
                    set_number<T>(v, i + e, at + e < here ? x[at + e] : from_f32<T>(none));
                }
                asm volatile("" ::: "memory");
            }
        }
    }
    if (tid == 0) count = 0;
    again(v);
    const bool many = a.width > kFewGroups / 2;
    float top;
    {
        uint32_t w = v[0];
#pragma unroll
        for (int i = 1; i < WORDS; ++i) w = larger<T>(w, v[i]);
        if (sizeof(T) == 4) {
            top = fmaxf(__uint_as_float(w), none);
        } else {
            const float2 y = pair_of<T>(&w, 0);
            top = fmaxf(fmaxf(y.x, y.y), none);   // none where all are NaN
        }
    }
    {
        float w = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (many && (lane & 1) == 0) groups[tid / 2] = w;
        w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 2));
        w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 4));
        if (!many && (lane & 7) == 0) groups[tid / 8] = w;
        w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 8));
        w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 16));
        if (lane == 0) tops[warp] = w;
    }
    __syncthreads();
    float m = tops[lane % kPartWarps];
#pragma unroll
    for (int d = 1; d < kPartWarps; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const uint32_t least = many ? reached_by<kMostGroups, kPartWarps>(groups, a.width) : reached_by<kFewGroups, kPartWarps>(groups, a.width);
    if (lane == 0) reach[warp] = least;

    // The sum of exponentials, in a tree of 32-bit sums: 17 additions deep for 32 numbers a thread.  64 bits would cost more than
    // all else here, as the machine adds two such numbers a cycle and SM (8192 parts of 8000 numbers: 57 us, against 40).
    float sum = 0.f;
    if (base_is_used(m)) {
        const float base = base_of(m);
        float2 s2[2] = {};
#pragma unroll
        for (int i = 0; i < N; i += 2) s2[i / 2 % 2] = add_pair(s2[i / 2 % 2], exps_of(pair_of<T>(v, i / 2), base));
        s2[0] = add_pair(s2[0], s2[1]);
        sum = s2[0].x + s2[0].y;
    } else {
#pragma unroll 1
        for (int i = 0; i < N; ++i) {   // read again, as below
            const int at = place_in_part<VEC>(i);
            const float y = at < here ? to_f32(x[at]) : none;
            if (!(y <= none)) sum += exp2f((y - m) * 1.44269504088896341f);
        }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    const float t = number_of(__reduce_min_sync(0xffffffffu, reach[lane % kPartWarps]));

    again(v);
    uint32_t low = 0xffffffffu - (uint32_t)(first + place_in_part<VEC>(0));
    auto key = [&](float y, int i) {
        return (u64)rising(y) << 32 | (low - (uint32_t)(i / VEC * kPartThreads * VEC + i % VEC));
    };
    if (top >= t && top > none) {
        auto gather = [&](float y, int i) {
            if (y >= t && y > none) {
                const int at = atomicAdd(&count, 1);
                if (at < kRoom) found[at] = key(y, i);
            }
        };
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if (!either_reaches<T>(v, i / 2, t)) continue;
            const float2 y = pair_of<T>(v, i / 2);
            gather(y.x, i);
            gather(y.y, i + 1);
        }
    }
    __syncthreads();
    if (warp == 0) {
        float all = sums[lane % kPartWarps];
#pragma unroll
        for (int d = 1; d < kPartWarps; d <<= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
        if (lane == 0) {
            a.sums[blockIdx.x] = all;
            a.tops[blockIdx.x] = m;
        }
    }
    u64 *best = a.best + (size_t)blockIdx.x * a.width;
    const int n = count;
    if (n <= kRoom) {
        for (int c = tid; c < max(n, a.width); c += kPartThreads) {
            if (c >= n) {
                best[c] = 0;
                continue;
            }
            const u64 mine = found[c];
            int rank = 0;
            for (int i = 0; i < n; ++i) rank += found[i] > mine;
            if (rank < a.width) best[rank] = mine;
        }
        return;
    }
    // One after the other: every thread has its largest key below the last one taken; whose that was looks for its next, and
    // reads its numbers again (a list of them in registers, gone through in so many places, would not stay there).
    u64 last = ~0ull, mine = last;
    for (int k = 0; k < a.width; ++k) {
        if (mine == last) {
            mine = 0;
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                const int at = place_in_part<VEC>(i);
                const float y = at < here ? to_f32(x[at]) : none;
                const u64 z = y > none ? key(y, i) : 0;
                if (z < last && z > mine) mine = z;
            }
        }
        u64 most = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        __syncthreads();
        if (lane == 0) found[warp] = most;
        __syncthreads();
        last = found[lane % kPartWarps];
#pragma unroll
        for (int d = 1; d < kPartWarps; d <<= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
        if (tid == 0) best[k] = last;
        if (last == 0) last = 1;   // nothing is left: zeros from here on
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

__device__ __forceinline__ u64 warp_max(u64 x, bool &mine) {   // `mine`: whether it is the lane's
    const uint32_t hi = (uint32_t)(x >> 32), most = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == most ? (uint32_t)x : 0u);
    const u64 m = (u64)most << 32 | lo;
    mine = x == m;
    return m;
}
// The first of a warp's candidates: whether it is the lane's (none's if there are none, with total 0).
__device__ __forceinline__ bool first_of(const Candidate &c) {
    bool mine;
    const u64 total = warp_max(c.total, mine);
    uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (total == 0) return false;
    if (who & (who - 1)) {   // of equal totals the lowest beam's, then the largest key
        const uint32_t beam = __reduce_min_sync(0xffffffffu, mine ? (uint32_t)c.beam : 0xffffffffu);
        mine = mine && (uint32_t)c.beam == beam;
        bool largest;
        warp_max(mine ? c.key : 0, largest);   // an ended beam's is 0, and alone
        who = __ballot_sync(0xffffffffu, mine && largest);
    }
    return (threadIdx.x & 31) == __ffs(who) - 1;
}

constexpr int kLists = 4;   // of a lane

__global__ void __launch_bounds__(kItemThreads) beam_item_kernel(const BeamArgs a) {
    __shared__ double shift[PS_BEAM_MAX_BEAMS];     // score - log sum exp(logit - largest)
    __shared__ float largest[PS_BEAM_MAX_BEAMS], score[PS_BEAM_MAX_BEAMS];
    __shared__ float2 near[PS_BEAM_MAX_BEAMS];      // largest and shift in 32 bits; (0, -infinity) of a beam that offers no tokens
    __shared__ uint8_t state[PS_BEAM_MAX_BEAMS];    // 0: offers nothing, 1: tokens, 2: itself, ended
    __shared__ Candidate chosen[kItemWarps + 1][PS_BEAM_MAX_WIDTH];   // by warp, and of all so far; total 0 where there is none
    static_assert(sizeof(chosen) >= sizeof(Candidate) * kRoom, "one place for both ways");
    Candidate *const found = chosen[0];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long item = blockIdx.x;
    const float none = __int_as_float(0xff800000);
    if (tid == 0) count = 0;
    cudaGridDependencySynchronize();   // the parts are done
    for (int b = warp; b < a.beams; b += kItemWarps) {
        const long long row = item * a.beams + b;
        const float sc = a.scores[row];
        const bool end = a.ended != nullptr && a.ended[row] != 0;
        float m = none;
        double all = 0.0;
        if (finite(sc) && !end) {
            float t = lane < a.parts ? a.tops[row * a.parts + lane] : none, s = lane < a.parts ? a.sums[row * a.parts + lane] : 0.f;
            m = t;
            for (int i = lane + 32; i < a.parts; i += 32) m = fmaxf(m, a.tops[row * a.parts + i]);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            for (int i = lane; i < a.parts; i += 32) {
                if (i >= 32) {
                    t = a.tops[row * a.parts + i];
                    s = a.sums[row * a.parts + i];
                }
                // The sum is one of exponentials of x - t - d ln 2, d the base's rounding: exact, as a product's is in 32 bits.
                const float d = base_is_used(t) ? fmaf(-t, 1.44269504088896341f, -base_of(t)) * 0.693147180559945309f : 0.f;
                all += s != s || s == 0.f ? (double)s : (double)s * (double)expf(t - m + d);   // off by 2^-22 of itself
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
        }
        if (lane == 0) {
            // the 32-bit logarithm, and once Newton's step from it: off by what expf is, 2^-23
            const float y = logf((float)all);
            const double sh = (double)sc - ((double)y + (all * (double)expf(-y) - 1.0));
            const int st = !finite(sc) ? 0 : end ? 2 : all == all && m > none ? 1 : 0;   // NaN: NaN or +infinity among the logits
            shift[b] = sh;
            largest[b] = m;
            score[b] = sc;
            state[b] = st;
            near[b] = st == 1 ? make_float2(m, (float)sh) : make_float2(0.f, none);
        }
    }
    __syncthreads();

    auto take = [&](int k, const Candidate &c) {
        const long long to = item * a.width + k;
        if (c.total != 0) {
            const bool end = state[c.beam] == 2;
            const int32_t token = end ? a.eos : (int32_t)(0xffffffffu - (uint32_t)c.key);
            const u64 b = c.total >> 63 ? c.total ^ 1ull << 63 : ~c.total;
            a.out_scores[to] = (float)__longlong_as_double((long long)b);
            a.out_parents[to] = (int32_t)(item * a.beams + c.beam);
            a.out_tokens[to] = token;
            if (a.out_ended) a.out_ended[to] = end || (a.eos >= 0 && token == a.eos);
        } else {
            a.out_scores[to] = none;
            a.out_parents[to] = a.out_tokens[to] = -1;
            if (a.out_ended) a.out_ended[to] = 0;
        }
    };
    const uint32_t lists = (uint32_t)a.beams * a.parts;
    const u64 *best = a.best + item * lists * a.width;
    // Totals of 32 bits: T is the width-th largest of the maxima of 512 groups.  A total near T is made of a score, a distance
    // from the row's largest and a logarithm that are no larger than `size`; 32 bits lose less than 2^-20 of it.  Distances
    // beyond 2^126 are taken for that, of which no T above -2^124 with scores below 2^120 knows; else all are gathered.
    const uint32_t keys = (uint32_t)min((u64)lists * a.width, 1ull << 31);   // of more, those behind are left to the other way
    auto near_total = [&](uint32_t i) {
        const float2 c = near[i / a.by_list];
        const uint32_t hi = reinterpret_cast<const uint32_t *>(best)[2 * (size_t)i + 1];
        return hi != 0 && c.y > none ? fmaxf(fmaxf(number_of(hi) - c.x, -0x1p126f) + c.y, -FLT_MAX) : none;
    };
    float mine = none, size = 0.f;
#pragma unroll 4
    for (uint32_t i = tid; i < keys; i += kItemThreads) mine = fmaxf(mine, near_total(i));
    for (int b = tid; b < a.beams; b += kItemThreads)
        if (state[b] == 2) mine = fmaxf(mine, score[b]);
    for (int b = lane; b < a.beams; b += 32)
        if (state[b] != 0) size = fmaxf(size, fabsf(score[b]) + (state[b] == 1 ? fabsf(near[b].y) : 0.f));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
    uint32_t reach = 0;   // its leading 24 bits: somewhat more than `width` may reach it
    const uint32_t order = mine >= -FLT_MAX ? rising(mine) : 0;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit >= 1u << 8; bit >>= 1)
        if (__syncthreads_count(order >= (reach | bit)) >= a.width) reach |= bit;
    float t = none;
    if (reach != 0) {
        t = number_of(reach);
        t -= (2.f * size + fabsf(t)) * 0x1p-20f;
        if (!(t > -0x1p124f && size < 0x1p120f)) t = none;
    }
#pragma unroll 4
    for (uint32_t i = tid; i < keys; i += kItemThreads) {
        const float y = near_total(i);
        if (!(y >= t) || y == none) continue;
        const int at = atomicAdd(&count, 1), b = (int)(i / a.by_list);
        if (at >= kRoom) continue;
        const u64 key = best[i];
        found[at] = {rising(((double)number_of((uint32_t)(key >> 32)) - (double)largest[b]) + shift[b]), key, b};
    }
    for (int b = tid; b < a.beams; b += kItemThreads)
        if (state[b] == 2) {
            const int at = atomicAdd(&count, 1);
            if (at < kRoom) found[at] = {rising((double)score[b]), 0, b};
        }
    __syncthreads();
    const int n = count;
    if (n <= kRoom && keys < 1u << 31) {
        for (int c = tid; c < max(n, a.width); c += kItemThreads) {
            if (c >= n) {
                take(c, {0, 0, 0});
                continue;
            }
            const Candidate x = found[c];
            int rank = 0;
            for (int i = 0; i < n; ++i) rank += before(found[i], x);
            if (rank < a.width) take(rank, x);
        }
        return;
    }
    // More than there is room for: the lists' heads one after the other, of 2048 lists at a time.  A warp merges 128 of them, four
    // a lane; then one warp those of all, and of the lists before.
    for (uint32_t base = 0; base < lists; base += kItemThreads * kLists) {
        Candidate head[kLists];
        u64 after[kLists];      // the key behind the head's, loaded ahead
        int next[kLists] = {}, beam[kLists] = {};
        auto load = [&](int q) {
            const uint32_t l = base + (warp * kLists + q) * 32 + lane;
            after[q] = beam[q] >= 0 && next[q] < a.width ? best[(size_t)l * a.width + next[q]] : 0;
            ++next[q];
        };
        auto advance = [&](int q) {   // the head becomes what was loaded ahead
            const u64 key = after[q];
            load(q);
            head[q] = {0, 0, INT_MAX};
            if (key != 0) {
                const double distance = (double)number_of((uint32_t)(key >> 32)) - (double)largest[beam[q]];
                head[q] = {rising(distance + shift[beam[q]]), key, beam[q]};
            }
        };
        __syncthreads();   // what there was in `chosen` has been read
#pragma unroll
        for (int q = 0; q < kLists; ++q) {
            const uint32_t l = base + (warp * kLists + q) * 32 + lane;
            beam[q] = l < lists ? (int)(l / (uint32_t)a.parts) : -1;
            next[q] = 0;
            if (beam[q] >= 0 && state[beam[q]] != 1) {
                const bool itself = state[beam[q]] == 2 && l % (uint32_t)a.parts == 0;   // an ended beam is the head of its first list
                head[q] = itself ? Candidate{rising((double)score[beam[q]]), 0, beam[q]} : Candidate{0, 0, INT_MAX};
                beam[q] = -1;
                load(q);
            } else {
                load(q);
                advance(q);
            }
        }
        const int warps = (int)min((lists - base + 32 * kLists - 1) / (32 * kLists), (uint32_t)kItemWarps);
        if (warp < warps) {
            for (int k = 0; k < a.width; ++k) {
                Candidate mine = head[0];
                int from = 0;
#pragma unroll
                for (int q = 1; q < kLists; ++q)
                    if (before(head[q], mine)) {
                        mine = head[q];
                        from = q;
                    }
                const bool won = first_of(mine);
                if (__ballot_sync(0xffffffffu, won) == 0) {   // no more
                    for (int i = k + lane; i < a.width; i += 32) chosen[warp][i] = {0, 0, INT_MAX};
                    break;
                }
                if (won) {
                    chosen[warp][k] = mine;
#pragma unroll
                    for (int q = 0; q < kLists; ++q)
                        if (q == from) advance(q);
                }
            }
        }
        __syncthreads();
        if (warps == 1 && base == 0 && lists <= 32 * kLists) break;   // warp 0 has them all
        if (warp == 0) {
            const bool list = lane < warps || (lane == kItemWarps && base > 0);
            int at = 0;
            Candidate mine = list ? chosen[lane][0] : Candidate{0, 0, INT_MAX}, result[PS_BEAM_MAX_WIDTH / 32];
            for (int k = 0; k < a.width; ++k) {
                const bool won = first_of(mine);
                const uint32_t who = __ballot_sync(0xffffffffu, won);
                Candidate c{0, 0, INT_MAX};
                if (who) {
                    const int from = __ffs(who) - 1;
                    c.total = __shfl_sync(0xffffffffu, mine.total, from);
                    c.key = __shfl_sync(0xffffffffu, mine.key, from);
                    c.beam = __shfl_sync(0xffffffffu, mine.beam, from);
                }
#pragma unroll
                for (int i = 0; i < PS_BEAM_MAX_WIDTH / 32; ++i)
                    if (k == i * 32 + lane) result[i] = c;
                if (won) mine = ++at < a.width ? chosen[lane][at] : Candidate{0, 0, INT_MAX};
            }
            __syncwarp();   // the lists so far have been read
#pragma unroll
            for (int i = 0; i < PS_BEAM_MAX_WIDTH / 32; ++i)
                if (i * 32 + lane < a.width) chosen[kItemWarps][i * 32 + lane] = result[i];
        }
        __syncthreads();
    }
    const Candidate *from = lists <= 32 * kLists ? chosen[0] : chosen[kItemWarps];
    for (int k = tid; k < a.width; k += kItemThreads) take(k, from[k]);
}

// ---- host --------------------------------------------------------------------------------

// Numbers of a thread: 16 KiB of logits a CTA, or 4 where rows are few, so that more SMs read them.
constexpr int kMostBytes = 64, kFewBytes = 16;
bool few_rows(const ps_beam_shape *d) {
    const long long most = (long long)kPartThreads * kMostBytes / (d->type == PS_REAL_F32 ? 4 : 2);
    return d->batch * d->beams * ((d->vocab + most - 1) / most) < 152;
}
struct Cut {
    long long parts, tokens;
};
Cut cut_of(const ps_beam_shape *d) {   // parts of one size, of whole pieces
    const long long most = (long long)kPartThreads * (few_rows(d) ? kFewBytes : kMostBytes) / (d->type == PS_REAL_F32 ? 4 : 2);
    const long long parts = (d->vocab + most - 1) / most, each = (d->vocab + parts - 1) / parts;
    const long long tokens = (each + 7) / 8 * 8;
    return {(d->vocab + tokens - 1) / tokens, tokens};
}

template <typename T, int VEC> cudaError_t launch(const BeamArgs &a, bool few, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.batch * a.beams * a.parts);
    if (few) beam_part_kernel<T, kFewBytes / sizeof(T), VEC><<<grid, kPartThreads, 0, s>>>(a);
    else beam_part_kernel<T, kMostBytes / sizeof(T), VEC><<<grid, kPartThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};   // starts while the parts are on their way, and waits for them
    c.gridDim = dim3((unsigned)a.batch);
    c.blockDim = dim3(kItemThreads);
    c.stream = s;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, beam_item_kernel, a);
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
    return d->batch * d->beams <= INT_MAX / cut_of(d).parts;
}
struct Parts {
    long long parts;
    size_t sums, tops, best, total;
};
Parts parts_of(const ps_beam_shape *d) {
    Parts p;
    p.parts = cut_of(d).parts;
    const size_t n = (size_t)(d->batch * d->beams * p.parts);
    p.sums = 0;
    p.tops = up(n * 4);
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
    a.part_tokens = cut_of(d).tokens;
    a.by_parts = divisor((uint32_t)a.parts);
    a.by_beams = divisor((uint32_t)a.beams);
    a.by_list = divisor((uint32_t)a.parts * (uint32_t)a.width);
    a.logits = logits;
    a.scores = scores;
    a.ended = ended;
    a.out_scores = out_scores;
    a.out_parents = out_parents;
    a.out_tokens = out_tokens;
    a.out_ended = out_ended;
    a.sums = reinterpret_cast<float *>(w + p.sums);
    a.tops = reinterpret_cast<float *>(w + p.tops);
    a.best = reinterpret_cast<u64 *>(w + p.best);
    const bool few = few_rows(d);
    // short rows number by number, so that every thread has some
    const bool pieces = d->vocab >= 4096 && on(logits, 16) && (d->batch == 1 || d->item_stride * (int64_t)es % 16 == 0) &&
                        (d->beams == 1 || d->beam_stride * (int64_t)es % 16 == 0);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = d->type == PS_REAL_F32    ? launch<float>(a, few, pieces, s)
                          : d->type == PS_REAL_BF16 ? launch<__nv_bfloat16>(a, few, pieces, s)
                                                    : launch<__half>(a, few, pieces, s);
    if (e == cudaSuccess) return PS_OK;
    note_cuda_error(e);
    return PS_ERR_CUDA;
}
