// linrec_common.cuh -- pieces shared by the gated linear recurrence's kernels:
// decays and how a factor is encoded, tiles and how they are loaded, where
// sequences start and end inside a tile, the look-back among tiles.
//
//     h_t = a_t h_{t-1} + w_t x_t,  a = exp(g),  w = 1 or 1 - a
//     backward, from the last token:  lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,
//     dx_t = w_t lam_t,  dg_t = mu_t (h_{t-1} - [tied] x_t),  dh0 = mu_1
//
// A tile is 32 channels by 512, 256 or 128 tokens, as much as three CTAs an SM can hold, in 16 runs of R = 32, 16 or 8 tokens.  A
// lane has a run and two neighbouring channels; a warp of eight has two runs of all 32 channels.  What a run costs beside its
// tokens (joining, the look-back's share) is some 300 instructions a lane, so longer runs are better (32 tokens instead of 16,
// forward, one sequence of 131072 tokens by 512 bf16 channels: 143 us instead of 170); shared memory bounds them, as two CTAs an
// SM with runs twice as long were slower (backward, 4 x 8192 tokens by 4096 bf16 channels, trained, now 458 us: 546 instead of 495
// then).  Wide tiles have long rows in memory (copies of 32 and 64 bf16 channels run at 5.9 and 6.0 TB/s, of 16 at 5.0), narrow
// ones make more chains, so that fewer of the tiles under way wait for one another: with 16, 32 and 64 channels earlier kernels
// took 283, 265 and 254 us for 48 ragged prompts (24571 tokens by 4096 channels, now 214), 180, 189 and 210 for the long one (now
// 141), 733, 630 and 615 for the training.  Sequences are cut out of the flat index over all tokens: where one
// starts the state is set, not multiplied, so short sequences fill tiles as long ones do.
//
// Each tile tells the ones behind it its map h -> a h + b, and the state behind it once it knows that.  A tile that
// needs the state before it takes the nearest state that is known and applies the maps since then in order
// (look-back).  The state behind a tile is always its map applied to the state before it, by the same three operations
// wherever this is done, so results do not depend on which states were known when: they repeat bit for bit, which sums
// composed in the order of arrival would not.
//
// CTAs stay and take tiles by ticket, in the order of the recurrence.  Eight warps compute; a ninth takes tickets, has
// tiles loaded as soon as the one before is done with, finds starts and ends, and looks back, which it begins while the tile's first pass still runs.
//
// Factors.  exp(g) of a slow decay rounds to 2^-24 of 1, and what a state forgets in a token, 1 - exp(g), may be not much
// more than that: an error to one side adds up over the state's whole memory (a thousand tokens and more).  So a factor
// near 1 is kept as its distance from 1 (sign bit set) and applied as h + (f h + b); others are kept as they are
// (sign bit clear), so that a closed gate forgets even a large state.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "delta_common.cuh"
#include "linrec_internal.h"
#include "scan_pipeline.cuh"

namespace ps {

namespace {

constexpr int kLrWarps = kLinrecWarps;
constexpr int kLrCompute = 32 * kLrWarps, kLrThreads = kLrCompute + 32;
constexpr int kLrWide = kLinrecWide, kLrPairs = kLrWide / 2;   // channels of a tile, and pairs of them
constexpr int kLrGroups = 32 / kLrPairs;                       // runs of a warp
static_assert(kLrGroups == 2, "as joining assumes");
constexpr int kLrRuns = kLrWarps * kLrGroups;                  // of a tile

__device__ __forceinline__ int lr_pair() { return threadIdx.x % kLrPairs; }
__device__ __forceinline__ int lr_group() { return threadIdx.x % 32 / kLrPairs; }
__device__ __forceinline__ int lr_run() { return threadIdx.x / kLrPairs; }   // of a compute warp's lane

// ---- pairs of f32 ------------------------------------------------------------------------

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float nan_f32() { return __uint_as_float(0x7fffffffu); }

// ---- factors ---------------------------------------------------------------------------

__device__ __forceinline__ bool near_one(float f) { return __float_as_int(f) < 0; }
__device__ __forceinline__ float exp2_fast(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
// Whether g is in (bound, -0]: the bits of negative numbers, as signed integers, rise with their magnitude.
__device__ __forceinline__ bool just_below_zero(float g, float bound) { return __float_as_int(g) < __float_as_int(bound); }
// The factors exp(g) of one token.  Above -1/16 the series up to g^4 / 24 leaves less than 2^-22.9 of the distance (with f32's
// roundings 2^-22.3); the hardware's 2^x, off by some 2^-22 of 1, serves elsewhere: there a state's memory is at most 16 tokens (and
// 2^0 is 1).
// Tied inputs are weighted by 1 - exp(g), of which 2^-22 of 1 would be 2^-18 just below -1/16 (with all roundings 2^-17.4).  For them
// the distance is g (1 + g q(g)), q such that the largest relative error is least.  Inputs of 16 bits: q of degree 2 above -5/32
// (with f32's roundings 2^-22.8), which is as many operations as the series; below, 2^x leaves 2^-19.4 of the weight (2^-18.7).
// Inputs of 32 bits: of degree 3 above -7/16 (2^-22.7); below, 2^-20.9 (2^-20.2).  (Degree 3 for all: one sequence of 131072 tokens by
// 512 bf16 channels 149 us instead of 141.)
// `one`: 1 where the factor is near one, 0 elsewhere.
enum class Weights { one, tied16, tied32 };   // 1, or tied inputs of 16 or 32 bits
template <typename TX, bool TIED> constexpr Weights kWeights = !TIED ? Weights::one : sizeof(TX) == 4 ? Weights::tied32 : Weights::tied16;

struct Token {
    float2 f, one;
    template <Weights W> __device__ __forceinline__ static Token of(float2 g) {
        const float2 y = mul2(g, both(1.44269504088896341f));
        float2 d;
        if (W == Weights::one) {
            d = fma2(g, both(1.f / 24.f), both(1.f / 6.f));
            d = fma2(g, d, both(0.5f));
        } else if (W == Weights::tied16) {
            d = fma2(g, both(0x1.417b94p-5f), both(0x1.54e304p-3f));
            d = fma2(g, d, both(0x1.fffe86p-2f));
        } else {
            d = fma2(g, both(0x1.c983bap-8f), both(0x1.515aaep-5f));
            d = fma2(g, d, both(0x1.553086p-3f));
            d = fma2(g, d, both(0x1.ffff2ap-2f));
        }
        d = fma2(g, d, both(1.f));
        d = mul2(g, d);   // -0 stays -0
        constexpr float FROM = W == Weights::one ? -1.f / 16.f : W == Weights::tied16 ? -5.f / 32.f : -7.f / 16.f;
        const bool x = just_below_zero(g.x, FROM), z = just_below_zero(g.y, FROM);
        return {make_float2(x ? d.x : exp2_fast(y.x), z ? d.y : exp2_fast(y.y)), make_float2(x ? 1.f : 0.f, z ? 1.f : 0.f)};
    }
    __device__ __forceinline__ static Token from(float2 f) {
        return {f, make_float2(near_one(f.x) ? 1.f : 0.f, near_one(f.y) ? 1.f : 0.f)};
    }
    __device__ __forceinline__ float2 weigh(float2 x, bool tied) const {   // x, or (1 - a) x
        return tied ? mul2(make_float2(1.f - one.x - f.x, 1.f - one.y - f.y), x) : x;
    }
    __device__ __forceinline__ float2 apply(float2 h, float2 b) const { return fma2(one, h, fma2(f, h, b)); }   // a h + b
    __device__ __forceinline__ float2 decayed(float2 h) const { return fma2(one, h, mul2(f, h)); }              // a h
};
// The factors of many tokens from the sums of their log decays: the same with a series up to s^8 / 8! above -1/2, because
// errors add up over the factors of a state's memory in runs and tiles.
__device__ __forceinline__ float2 factor_of_sum(float2 s) {
    const float2 y = mul2(s, both(1.44269504088896341f));
    float2 d = fma2(s, both(1.f / 40320.f), both(1.f / 5040.f));
    d = fma2(s, d, both(1.f / 720.f));
    d = fma2(s, d, both(1.f / 120.f));
    d = fma2(s, d, both(1.f / 24.f));
    d = fma2(s, d, both(1.f / 6.f));
    d = fma2(s, d, both(0.5f));
    d = fma2(s, d, both(1.f));
    d = mul2(s, d);
    return make_float2(just_below_zero(s.x, -0.5f) ? d.x : exp2_fast(y.x), just_below_zero(s.y, -0.5f) ? d.y : exp2_fast(y.y));
}
// a h + b
__device__ __forceinline__ float2 apply(float2 f, float2 h, float2 b) {
    const float2 t = fma2(f, h, b);
    return add2(t, make_float2(near_one(f.x) ? h.x : 0.f, near_one(f.y) ? h.y : 0.f));
}
// ---- numbers in memory -------------------------------------------------------------------

template <typename T> struct Pair;
template <> struct Pair<float> {
    typedef float2 type;
    __device__ static float2 get(float2 x) { return x; }
    __device__ static float2 put(float2 x) { return x; }
};
template <> struct Pair<__nv_bfloat16> {
    typedef uint32_t type;
    __device__ static float2 get(uint32_t x) { return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); }
    __device__ static uint32_t put(float2 x) {
        const __nv_bfloat162 y = __float22bfloat162_rn(x);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
};
template <> struct Pair<__half> {
    typedef uint32_t type;
    __device__ static float2 get(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }
    __device__ static uint32_t put(float2 x) {
        const __half2 y = __float22half2_rn(x);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
};
// Token i of a lane's run in a tile in shared memory: there the runs' first tokens come first, then their second ones, and so
// on, so that a warp reads neighbouring words.
template <typename T> __device__ __forceinline__ float2 pair_at(const T *tile, int i) {
    return Pair<T>::get(reinterpret_cast<const typename Pair<T>::type *>(tile)[i * kLrCompute + threadIdx.x]);
}
template <typename T> __device__ __forceinline__ void set_pair_at(T *tile, int i, float2 x) {
    reinterpret_cast<typename Pair<T>::type *>(tile)[i * kLrCompute + threadIdx.x] = Pair<T>::put(x);
}
// Log decays of 32 bits give their place to the token's factor once that is known, for the second pass.
template <Weights W, typename TG> __device__ __forceinline__ Token token_at(const TG *gs, int i) {
    if constexpr (sizeof(TG) == 4) return Token::from(pair_at(gs, i));
    else return Token::of<W>(pair_at(gs, i));
}
template <typename TG> __device__ __forceinline__ void keep(TG *gs, int i, const Token &t) {
    if (sizeof(TG) == 4) set_pair_at(gs, i, t.f);
}
// A lane's two channels of a row in global memory; `whole`: both are there and the row starts on a multiple of two.
template <typename T> __device__ __forceinline__ void put_pair(T *p, float2 x, bool whole, bool in0, bool in1) {
    if (whole) {
        *reinterpret_cast<typename Pair<T>::type *>(p) = Pair<T>::put(x);
    } else {
        if (in0) p[0] = from_f32<T>(x.x);
        if (in1) p[1] = from_f32<T>(x.y);
    }
}
__device__ __forceinline__ float2 get_f32(const float *p, bool in0, bool in1) {
    return make_float2(p && in0 ? p[0] : 0.f, p && in1 ? p[1] : 0.f);
}
__device__ __forceinline__ void put_f32(float *p, float2 x, bool in0, bool in1) {
    if (in0) p[0] = x.x;
    if (in1) p[1] = x.y;
}

// ---- loads -----------------------------------------------------------------------------

template <int BYTES> __device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool there) {
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The tokens from n0 on of a tensor, channels from c0 on, to a tile in shared memory, in pieces of N numbers, by the threads of
// the compute warps; 0 past the ends.
template <typename T, int R, int N, int UNROLL>
__device__ __forceinline__ void load_pieces(T *tile, const LinrecTensor &x, const LinrecArgs &a, uint32_t n0, long long c0) {
    constexpr int PER = kLrWide / N, STEP = kLrCompute / PER, ROWS = kLrRuns * R;   // pieces of a row, rows at a time
    const int col = threadIdx.x % PER * N, row0 = threadIdx.x / PER;
    const bool in = c0 + col < a.channels;
    const T *base = static_cast<const T *>(x.p), *src = base + c0 + col;
    uint32_t n = n0 + row0, t = 0;
    if (x.flat) {
        src += (long long)n * x.tok;
    } else {
        const uint32_t seq = n / (uint32_t)a.tokens;
        t = n - seq * (uint32_t)a.tokens;
        src += seq * x.seq + (long long)t * x.tok;
    }
    const long long step = STEP * x.tok;
    auto next = [&] {
        n += STEP;
        src += step;
        if (!x.flat) {
            for (t += STEP; t >= (uint32_t)a.tokens; t -= (uint32_t)a.tokens) src += x.seq - (long long)a.tokens * x.tok;
        }
    };
    auto place = [&](int row) { return tile + (row % R * kLrRuns + row / R) * kLrWide + col; };
    if constexpr (N * sizeof(T) == 2) {   // 16 under way at a time (3001 tokens by 1001 f16 channels, trained: 63 us; 8: 66, 4: 80)
        static_assert(ROWS / STEP % UNROLL == 0, "whole rounds");
#pragma unroll 1
        for (int row = row0; row < ROWS; row += STEP * UNROLL) {
            T y[UNROLL];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k, next()) y[k] = in && n < (uint32_t)a.total ? *src : from_f32<T>(0.f);
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) *place(row + k * STEP) = y[k];
        }
    } else {
#pragma unroll(UNROLL)
        for (int row = row0; row < ROWS; row += STEP, next()) {
            const bool there = in && n < (uint32_t)a.total;
            copy_async<N * sizeof(T)>(smem_u32(place(row)), there ? src : base, there);
        }
    }
}
template <typename T, int R>
__device__ __forceinline__ void load_tile(T *tile, const LinrecTensor &x, const LinrecArgs &a, uint32_t n0, long long c0) {
    if (x.piece == 16) load_pieces<T, R, 16 / sizeof(T), 1>(tile, x, a, n0, c0);
    else if (sizeof(T) == 4 || x.piece == 4) load_pieces<T, R, 4 / sizeof(T), 2>(tile, x, a, n0, c0);
    else load_pieces<T, R, 1, 16>(tile, x, a, n0, c0);
}

// Inputs whose rows are evenly spaced, on multiples of 16 bytes, come by tensor copies of whole tiles, one thread's doing
// (their maps count channels, runs and tokens of a run; a last run that is not whole is left out, and read by its own lanes);
// others in pieces of 16, 4 or 2 bytes by all compute warps.
struct LinrecMaps {
    CUtensorMap g, x, d;
};
__device__ __forceinline__ void tile_copy(void *tile, const CUtensorMap &map, int run, int c0, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(smem_u32(tile)), "l"(&map), "r"(c0), "r"(run), "r"(0), "r"(smem_u32(bar)) : "memory");
}
// The last run's tokens, if it is not whole (a lane of the run; it alone reads them).
template <typename T, int R>
__device__ __forceinline__ void load_last_run(T *tile, const LinrecTensor &x, const LinrecArgs &a, uint32_t first, long long ch) {
    const T *p = static_cast<const T *>(x.p) + first * x.tok + ch;
    for (int i = 0; first + i < (uint32_t)a.total; ++i, p += x.tok)
        set_pair_at(tile, i, make_float2(ch < a.channels ? to_f32<T>(p[0]) : 0.f, ch + 1 < a.channels ? to_f32<T>(p[1]) : 0.f));
}

// ---- starts and ends -------------------------------------------------------------------

template <int TOKENS> struct Marks {
    uint32_t start[TOKENS / 32], end[TOKENS / 32];      // bits of tokens that are a sequence's first, its last (if there is any)
    int32_t seq[TOKENS];                                // whose they are
    uint32_t lo, held;                                  // tokens lo ... lo + held - 1 are sequences'
    int starts, ends;                                   // whether there is any
};
__device__ __forceinline__ uint32_t offset_at(const LinrecArgs &a, long long i) {
    const int32_t c = a.cu[i];
    return c < 0 ? 0u : min((uint32_t)c, (uint32_t)a.total);
}
// How many of the seqs + 1 offsets are below `n`, by 32 probes a round (all lanes of a warp).
__device__ __forceinline__ long long offsets_below(const LinrecArgs &a, uint32_t n) {
    long long lo = 0, hi = a.seqs + 1;   // the answer is in [lo, hi]
    while (lo < hi) {
        const long long step = (hi - lo + 31) / 32, at = lo + step * (threadIdx.x & 31);
        const bool below = at < hi && offset_at(a, at) < n;
        const int k = __popc(__ballot_sync(0xffffffffu, below));   // of never-falling offsets the first k are
        if (k == 0) return lo;
        const long long last = lo + step * (k - 1);
        hi = min(hi, last + step);
        lo = last + 1;
    }
    return lo;
}
// Fills `m` for the tile whose first token is `n0` (one warp).  Empty sequences' states go from `from` (nullptr: 0) to `to`
// (nullptr: nowhere) here, for the tile's channels: in the tile at their offset, or in the last one.
template <int TOKENS>
__device__ __forceinline__ void mark_tile(Marks<TOKENS> &m, const LinrecArgs &a, uint32_t n0, bool last_tile, const float *from,
                                          float *to, long long c0) {
    const int lane = threadIdx.x & 31;
    if (a.cu == nullptr) {
        const uint32_t tokens = (uint32_t)a.tokens, first = n0 / tokens, t0 = n0 - first * tokens;
        uint32_t any_s = 0, any_e = 0;
        if (t0 == 0 || t0 + TOKENS >= tokens) {   // not inside of one sequence
            for (int i = 0; i < TOKENS / 32; ++i) {
                const uint32_t n = n0 + 32 * i + lane, seq = n / tokens, t = n - seq * tokens;
                const bool in = n < (uint32_t)a.total;
                const uint32_t s = __ballot_sync(0xffffffffu, in && t == 0), e = __ballot_sync(0xffffffffu, in && t == tokens - 1);
                m.seq[32 * i + lane] = (int32_t)seq;
                any_s |= s;
                any_e |= e;
                if (lane == 0) {
                    m.start[i] = s;
                    m.end[i] = e;
                }
            }
        }
        if (lane == 0) {
            m.lo = 0;
            m.held = (uint32_t)a.total;
            m.starts = any_s != 0;
            m.ends = any_e != 0;
        }
        __syncwarp();
        return;
    }
    const uint32_t n1 = n0 + TOKENS;
    if (lane < TOKENS / 32) m.start[lane] = m.end[lane] = 0;
    __syncwarp();
    const long long below = offsets_below(a, n0);
    bool any_s = false, any_e = false;
    for (long long i0 = below > 0 ? below - 1 : 0; i0 < a.seqs; i0 += 32) {
        const long long i = i0 + lane;
        bool past = false;
        if (i < a.seqs) {
            const uint32_t s = offset_at(a, i), e = offset_at(a, i + 1);
            past = s >= n1;
            if (e > s) {
                if (s >= n0 && s < n1) {
                    atomicOr(&m.start[(s - n0) / 32], 1u << ((s - n0) & 31));
                    m.seq[s - n0] = (int32_t)i;
                    any_s = true;
                }
                if (e > n0 && e <= n1) {
                    atomicOr(&m.end[(e - 1 - n0) / 32], 1u << ((e - 1 - n0) & 31));
                    m.seq[e - 1 - n0] = (int32_t)i;
                    any_e = true;
                }
            } else if (to != nullptr && s >= n0 && (s < n1 || last_tile)) {
                for (long long c = c0; c < min(c0 + (long long)kLrWide, a.channels); ++c)
                    to[i * a.channels + c] = from ? from[i * a.channels + c] : 0.f;
            }
        }
        if (__any_sync(0xffffffffu, past) && !last_tile) break;
    }
    any_s = __any_sync(0xffffffffu, any_s);
    any_e = __any_sync(0xffffffffu, any_e);
    if (lane == 0) {
        const uint32_t lo = offset_at(a, 0), hi = offset_at(a, a.seqs);
        m.lo = lo;
        m.held = hi > lo ? hi - lo : 0;
        m.starts = any_s;
        m.ends = any_e;
    }
    __syncwarp();
}
// The bits of a run's tokens.
template <int R, int N> __device__ __forceinline__ uint32_t run_bits(const uint32_t (&bits)[N], int run) {
    static_assert(N * 32 == kLrRuns * R && 32 % R == 0, "a bit a token");
    return bits[run * R / 32] >> (run * R % 32) & (R == 32 ? 0xffffffffu : (1u << (R % 32)) - 1);
}

// Whether one of warp w's runs forgets what came before.
template <int R, bool BACKWARD, int TOKENS> __device__ __forceinline__ bool warp_cut(const Marks<TOKENS> &m, int w) {
    uint32_t x = 0;
#pragma unroll
    for (int g = 0; g < kLrGroups; ++g) {
        x |= m.starts ? run_bits<R>(m.start, w * kLrGroups + g) : 0u;
        if (BACKWARD) x |= m.ends ? run_bits<R>(m.end, w * kLrGroups + g) : 0u;
    }
    return x != 0;
}
// Where a tile is: the tile of tokens (-1: there is none) and the block of channels.
struct Place {
    int tile, block;
};
// A lane's run of a tile, and its channels.
template <int R> struct Run {
    uint32_t first, starts, ends;
    long long ch;
    bool in0, in1, whole;   // whether the channels are there; whether outputs' pairs are, and on multiples of two numbers
    bool marked, plain;     // of any run of the warp: has a start or end; neither, all tokens held and all pairs whole
    template <int TOKENS> __device__ __forceinline__ Run(const LinrecArgs &a, const Marks<TOKENS> &m, const Place &at) {
        first = (uint32_t)at.tile * TOKENS + lr_run() * R;
        ch = (long long)at.block * kLrWide + 2 * lr_pair();
        in0 = ch < a.channels;
        in1 = ch + 1 < a.channels;
        whole = in1 && a.pairs;
        starts = m.starts ? run_bits<R>(m.start, lr_run()) : 0u;
        ends = m.ends ? run_bits<R>(m.end, lr_run()) : 0u;
        marked = __any_sync(0xffffffffu, (starts | ends) != 0);
        plain = !marked && __all_sync(0xffffffffu, (whole || !in0) && first - m.lo < m.held && first - m.lo + R <= m.held);
    }
    template <int TOKENS> __device__ __forceinline__ float2 start(const LinrecArgs &a, const Marks<TOKENS> &m, int i) const {
        return get_f32(a.h0 ? a.h0 + m.seq[lr_run() * R + i] * a.channels + ch : nullptr, in0, in1);
    }
    template <int TOKENS> __device__ __forceinline__ float2 end(const LinrecArgs &a, const Marks<TOKENS> &m, int i) const {
        return get_f32(a.dht ? a.dht + m.seq[lr_run() * R + i] * a.channels + ch : nullptr, in0, in1);
    }
};

// ---- look-back -------------------------------------------------------------------------

// What a tile tells, its map and the state behind it, is 32-bit words that hold kUntold until then: a reader that finds
// another bit pattern in a word has the number, without flags, and so without the fences that would order a flag behind
// the numbers (a fence also waits for the outputs that its SM has under way).  No result is kUntold: a NaN with
// that pattern is told as another.
constexpr uint32_t kUntold = 0xffffffffu;

__device__ __forceinline__ bool told(float x) { return __float_as_uint(x) != kUntold; }
__device__ __forceinline__ float telling(float x) { return told(x) ? x : nan_f32(); }
__device__ __forceinline__ bool told(float2 x) { return told(x.x) && told(x.y); }
__device__ __forceinline__ bool told(float4 x) { return told(x.x) && told(x.y) && told(x.z) && told(x.w); }
__device__ __forceinline__ void tell(float2 *p, float2 x) {
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" :: "l"(p), "f"(telling(x.x)), "f"(telling(x.y)) : "memory");
}
__device__ __forceinline__ void tell(float4 *p, float2 f, float2 b) {
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};"
                 :: "l"(p), "f"(telling(f.x)), "f"(telling(f.y)), "f"(telling(b.x)), "f"(telling(b.y)) : "memory");
}
__device__ __forceinline__ float2 ask(const float2 *p) {
    float2 x;
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "l"(p) : "memory");
    return x;
}
__device__ __forceinline__ float4 ask(const float4 *p) {
    float4 x;
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p) : "memory");
    return x;
}
// What the warps' runs come to together.
struct Sums {
    float2 s[kLrWarps][kLrPairs], f[kLrWarps][kLrPairs];   // sums of log decays, their factors
    float2 b[kLrWarps][kLrPairs];                          // what the runs add
};
// What a warp's runs before a lane's come to (the state before the run is a h + b of the one before the warp's first), in the
// direction of the recurrence.  `cut`: whether one of them forgets what came before.
struct Ahead {
    float2 f, b;
    bool cut;
};
__device__ __forceinline__ float2 from_group(float2 x, int group) {
    return make_float2(__shfl_sync(0xffffffffu, x.x, group * kLrPairs + lr_pair()), __shfl_sync(0xffffffffu, x.y, group * kLrPairs + lr_pair()));
}
// A warp joins its runs, of which a lane knows its own: the sum of log decays s, its factor f, the addend b, whether it is
// `cut`; and leaves the whole's in the places [warp][pair] that are given.
template <bool BACKWARD>
__device__ __forceinline__ Ahead join_runs(float2 s, float2 f, float2 b, bool cut, bool any, float2 (*sum)[kLrPairs],
                                           float2 (*factors)[kLrPairs], float2 (*adds)[kLrPairs]) {
    const int warp = threadIdx.x >> 5, first = BACKWARD ? 1 : 0;   // the run that comes first
    const float2 fs = from_group(s, first), ff = from_group(f, first), fb = from_group(b, first);
    const bool fc = any && __shfl_sync(0xffffffffu, (int)cut, first * kLrPairs);
    const bool second = lr_group() != first;
    Ahead a{both(0.f), both(0.f), false};
    if (second) {
        a = {ff, fb, fc};
        if (!cut) b = apply(f, a.b, b);
        s = add2(fs, s);
        f = factor_of_sum(s);
        if (sum != nullptr) sum[warp][lr_pair()] = s;
        if (factors != nullptr) factors[warp][lr_pair()] = f;
        adds[warp][lr_pair()] = b;
    }
    return a;
}
// The state before a lane's run from the one before the tile.  `cut(w)`: whether warp w's runs forget what came before.
template <bool BACKWARD, typename Cut>
__device__ __forceinline__ float2 before_run(float2 h, const Ahead &a, const float2 (*factors)[kLrPairs], const float2 (*adds)[kLrPairs],
                                             bool any, Cut cut) {
    const int warp = threadIdx.x >> 5;
    for (int i = 0; i < (BACKWARD ? kLrWarps - 1 - warp : warp); ++i) {
        const int w = BACKWARD ? kLrWarps - 1 - i : i;
        const float2 b = adds[w][lr_pair()];
        h = any && cut(w) ? b : apply(factors[w][lr_pair()], h, b);
    }
    return lr_group() == (BACKWARD ? 1 : 0) ? h : a.cut ? a.b : apply(a.f, h, a.b);
}

// How long anything is waited for; two seconds, which no correct launch takes.  (Tests of what follows then set another limit.)
#ifndef PS_LINREC_WAIT_LIMIT_NS
#define PS_LINREC_WAIT_LIMIT_NS 2000000000ull
#endif
constexpr unsigned long long kLrWaitLimitNs = PS_LINREC_WAIT_LIMIT_NS;
// Waits for a phase in tries of up to `ns` nanoseconds; false if that ran out.
__device__ __forceinline__ bool mbar_wait_limited(uint64_t *bar, uint32_t parity, uint32_t ns, unsigned long long limit = kLrWaitLimitNs) {
    if (mbar_try_wait_for(bar, parity, ns)) return true;
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 0; i < kMbarSpinCap; ++i) {
        if (mbar_try_wait_for(bar, parity, ns)) return true;
        if ((i & 15u) == 15u && global_ns() - t0 > limit) break;
    }
    return false;
}

// What a CTA's warps share beside its tiles.
constexpr int kLrWindow = 8;   // tiles that a round of the look-back reads
static_assert(kLrWindow <= kLinrecSlack, "a round stays in the workspace");
template <int R> struct Shared {
    static constexpr int TOKENS = kLrRuns * R;
    Sums sums;
    float2 before[kLrPairs];     // the state before the tile, in the direction of the recurrence
    float4 maps[kLrWindow][kLrPairs];
    float2 states[kLrWindow][kLrPairs];
    Marks<TOKENS> marks[2];
    Place place[2];
    uint64_t landed, summed, done;   // the tile's inputs are there; all runs are summed; the inputs are no longer needed
    volatile int lost;               // a wait for inputs, or for their place, ran out: see wait_for_inputs
    // All lanes, before barriers and anything else.
    __device__ __forceinline__ void init() {
        if (threadIdx.x == 0) {
            mbar_init(&landed, 1);
            mbar_init(&summed, kLrWarps);
            mbar_init(&done, kLrWarps);
            lost = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncthreads();
    }
    // Waits for a tile's inputs (a compute warp's lane).  Where that runs out, the tile and all that the CTA takes after it
    // are lost: nothing is copied any more, what was not read is not written over, and the outputs are NaN.
    __device__ __forceinline__ void wait_for_inputs(int turn) {
        if (!mbar_try_wait_for(&landed, turn, 2000) && !lost && !mbar_wait_limited(&landed, turn, 2000)) lost = 1;
    }
    // Of a whole warp: it needs its inputs no longer, and what it wrote in their place comes before the next copies.
    __device__ __forceinline__ void release() {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&done);
    }
};
// Barriers by number.  1: marks are set, the next tile is known, pieces of tiles have landed; 2: the first tile is known;
// 3: the state before the tile is known; 4: among the compute warps.  The ninth warp never waits at them.
// Whether a phase is over, without waiting (try_wait may hold the warp for some time).
__device__ __forceinline__ bool mbar_over(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void pass_by(int id) { asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(kLrThreads) : "memory"); }
__device__ __forceinline__ void meet(int id) { named_barrier(id, kLrThreads); }

// The ninth warp.  `issue(place)` has a tile loaded (one lane), where tensor copies do.
//
// Tiles have positions in the order of the recurrence: the tile before position p is at p - 1.  Tickets go up the positions, or,
// where equal sequences take turns, up each sequence's; a chain starts at position 0, or at its sequence's first.
//
// Look-back: `at` is the last position before this tile's whose state, h, is known (-1: none yet).  A round reads what a window of
// tiles has told, from at + 1 on, or, with nothing known, further and further back in the chain; the last state told
// replaces h, the maps behind it are applied.  Rounds begin while the tile's inputs are summed; if the state before it is not
// known when they are, the tile's map is told at once, for others to pass over it.  A chain's first tile always tells its
// state.  Waits end after kLrWaitLimitNs, with NaN.
template <int R, bool BACKWARD, typename Issue>
__device__ __forceinline__ void ninth_warp(const LinrecArgs &a, Shared<R> &sm, const float *from, float *to, bool tensor_copies,
                                           Issue issue) {
    constexpr int TOKENS = Shared<R>::TOKENS, AT_ONCE = kLrWindow / kLrGroups;
    constexpr uint32_t FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, pair = lr_pair(), group = lr_group();
    const unsigned all = (unsigned)a.tiles * (unsigned)a.blocks;
    const bool chained = a.tiles > 1;
    const size_t stride = (size_t)a.blocks * kLrPairs;
    auto place_of = [&](unsigned ticket) {
        if (ticket >= all) return Place{-1, 0};
        const unsigned k = ticket / (unsigned)a.blocks;
        const int p = (int)(a.steps ? k % (unsigned)a.seqs * (unsigned)a.steps + k / (unsigned)a.seqs : k);
        return Place{BACKWARD ? a.tiles - 1 - p : p, (int)(ticket % (unsigned)a.blocks)};
    };
    auto take = [&]() { return chained ? atomicAdd(a.ticket, 1u) + 1 : all; };   // from -1 on
    auto copy = [&](const Place &at) {
#ifdef PS_TESTING_LOST_TILE   // of the first block: a tile that is never copied, so that the wait for it runs out
        if (at.tile == PS_TESTING_LOST_TILE && at.block == 0) return;
#endif
        issue(at);
    };
    unsigned ticket = blockIdx.x, next = all;
    if (chained && lane == 0) ticket = take();
    Place place = place_of(__shfl_sync(FULL, ticket, 0));
    if (lane == 0) {
        sm.place[0] = place;
        if (tensor_copies && place.tile >= 0) copy(place);
        next = take();
    }
    int last_turn = 0;   // whose inputs were copied last
    __syncwarp();
    pass_by(2);
    for (int turn = 0, first = 1; place.tile >= 0; turn ^= 1, first = 0) {
        Marks<TOKENS> &m = sm.marks[turn];
        const Sums &sums = sm.sums;
        mark_tile(m, a, (uint32_t)place.tile * TOKENS, place.tile == a.tiles - 1, from, to, (long long)place.block * kLrWide);
        const Place next_place = place_of(__shfl_sync(FULL, next, 0));
        if (lane == 0) sm.place[turn ^ 1] = next_place;
        __syncwarp();
        pass_by(1);
        if (!first && tensor_copies) {
            if (!mbar_wait_limited(&sm.done, turn ^ 1, 1000)) sm.lost = 1;   // with the tile before
            __syncwarp();
            if (!sm.lost) {
                if (lane == 0) copy(place);
                last_turn = turn;
            }
            __syncwarp();
        }
        if (lane == 0) next = take();

        const int p = BACKWARD ? a.tiles - 1 - place.tile : place.tile;
        const int chain = a.steps ? p - p % a.steps : 0;
        const bool any = BACKWARD ? (m.starts | m.ends) != 0 : m.starts != 0;   // a run forgets what came before the tile
        const bool known = p == 0 || any;                                       // so does the state behind it
        const bool needs = p > 0 && (BACKWARD ? !m.ends || m.end[TOKENS / 32 - 1] >> 31 == 0 : !m.starts || (m.start[0] & 1) == 0);
        float2 *const states = a.state + (size_t)place.block * kLrPairs + pair;
        float4 *const maps = a.map + (size_t)place.block * kLrPairs + pair;
        float2 h = both(0.f), f = both(0.f), b = both(0.f);
        int at = needs ? -1 : p - 1, back = max(p - kLrWindow, chain);
        bool have_sums = false, passed = false;
        uint32_t polls = 0;
        unsigned long long t0 = 0;
        while (true) {
            const bool found = at == p - 1;
            bool just = false;
            // Lanes may see a phase end at different times, and all of them shuffle below: so all have seen it, or none has.
            // Sums come after the wait for inputs, and the limit of their wait after its.
            if (!have_sums && (found ? mbar_wait_limited(&sm.summed, turn, 2000, 4 * kLrWaitLimitNs) || true
                                     : __all_sync(FULL, mbar_over(&sm.summed, turn))))
                have_sums = just = true;
            if (found && have_sums && !passed) {   // not before all have their sums: some may still wait for the last tile's state
                passed = true;
                if (group == 0) sm.before[pair] = h;
                __syncwarp();
                pass_by(3);
            }
            if (just) {
                if (chained) {
                    float2 s = both(0.f);
#pragma unroll 4
                    for (int i = 0; i < kLrWarps; ++i) {
                        const int w = BACKWARD ? kLrWarps - 1 - i : i;
                        const float2 bw = sums.b[w][pair];
                        b = any && warp_cut<R, BACKWARD>(m, w) ? bw : apply(sums.f[w][pair], b, bw);
                        s = add2(s, sums.s[w][pair]);
                    }
                    f = factor_of_sum(s);
                    if (group == 0) {
                        if (known) tell(states + p * stride, b);
                        else if (found) tell(states + p * stride, apply(f, h, b));
                        else tell(maps + p * stride, f, b);
                    }
                }
            }
            if (passed) break;
            if (!found) {
                const int j = at >= 0 ? at + 1 : back, n = min(p - j, kLrWindow);
                float2 st[AT_ONCE];
                float4 mp[AT_ONCE];
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) {   // past the tile's own, places are of later tiles, or slack
                    st[i] = ask(states + (j + i * kLrGroups + group) * stride);
                    mp[i] = ask(maps + (j + i * kLrGroups + group) * stride);
                }
                uint32_t told_state = 0, told_map = 0;   // a bit a tile
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) {
                    const uint32_t s = ~__ballot_sync(FULL, told(st[i])), q = ~__ballot_sync(FULL, told(mp[i]));
#pragma unroll
                    for (int g = 0; g < kLrGroups; ++g) {
                        constexpr uint32_t LANES = (1u << kLrPairs) - 1;
                        told_state |= (uint32_t)((s >> (g * kLrPairs) & LANES) == 0) << (i * kLrGroups + g);
                        told_map |= (uint32_t)((q >> (g * kLrPairs) & LANES) == 0) << (i * kLrGroups + g);
                    }
                    sm.states[i * kLrGroups + group][pair] = st[i];
                    sm.maps[i * kLrGroups + group][pair] = mp[i];
                }
                __syncwarp();
                told_state &= FULL >> (32 - n);
                if (told_state) {
                    const int last = 31 - __clz(told_state);
                    h = sm.states[last][pair];
                    at = j + last;
                }
                if (at >= 0) {
                    for (int i = at + 1 - j; i < n && (told_map >> i & 1); ++i) {
                        const float4 x = sm.maps[i][pair];
                        h = apply(make_float2(x.x, x.y), h, make_float2(x.z, x.w));
                        at = j + i;
                    }
                } else {
                    back = back > chain ? max(back - kLrWindow, chain) : max(p - kLrWindow, chain);
                }
                __syncwarp();
                if (!have_sums && at < p - 1) mbar_try_wait_for(&sm.summed, turn, 300);   // others may tell more meanwhile
                if (have_sums && ++polls > 4) {
                    if (polls == 5) t0 = global_ns();
                    if (__shfl_sync(FULL, (int)(global_ns() - t0 > kLrWaitLimitNs), 0)) {
                        h = both(nan_f32());
                        at = p - 1;
                    }
                }
                if (have_sums && at == p - 1 && !known && group == 0) tell(states + p * stride, apply(f, h, b));
            }
        }
        place = next_place;
    }
    if (tensor_copies && sm.lost) mbar_wait_limited(&sm.landed, last_turn, 2000);   // what is under way still writes to this CTA's memory
}

}  // namespace

// Runs CALL(types) for the type codes.
#define PS_LINREC_DISPATCH(CALL)                                                                        \
    do {                                                                                                \
        if (type == PS_REAL_F32) return CALL(float, float);                                             \
        if (type == PS_REAL_BF16 && gate_type == PS_REAL_F32) return CALL(__nv_bfloat16, float);        \
        if (type == PS_REAL_BF16) return CALL(__nv_bfloat16, __nv_bfloat16);                            \
        if (gate_type == PS_REAL_F32) return CALL(__half, float);                                       \
        return CALL(__half, __half);                                                                    \
    } while (0)

}  // namespace ps
