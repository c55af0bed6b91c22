// linrec_common.cuh -- pieces shared by the gated linear recurrence's kernels:
// decays and how a factor is encoded, tiles and how they are loaded, where
// sequences start and end inside a tile, the look-back among tiles.
//
//     h_t = a_t h_{t-1} + w_t x_t,  a = exp(g),  w = 1 or 1 - a
//     backward, from the last token:  lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,
//     dx_t = w_t lam_t,  dg_t = mu_t (h_{t-1} - [tied] x_t),  dh0 = mu_1
//
// A tile is 8 R tokens by 64 channels.  Warp w of eight has tokens R w ... R w + R - 1 of it (a run), a lane two neighbouring
// channels.  Sequences are cut out of the flat index over all tokens: where one starts the state is set, not multiplied, so
// short sequences fill tiles as long ones do.
//
// Each tile tells the ones behind it its map h -> a h + b, and the state behind it once it knows that.  A tile that
// needs the state before it takes the nearest state that is known and applies the maps since then in order
// (look-back).  The state behind a tile is always its map applied to the state before it, by the same three operations
// wherever this is done, so results do not depend on which states were known when: they repeat bit for bit, which sums
// composed in the order of arrival would not.
//
// CTAs stay and take tiles by ticket, in the order of the recurrence.  Eight warps compute; a ninth takes tickets, has
// tiles loaded, finds starts and ends, and looks back, which it begins while the tile's first pass still runs.
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

constexpr int kLrWarps = 8;
constexpr int kLrCompute = 32 * kLrWarps, kLrThreads = kLrCompute + 32;
constexpr int kLrWide = 64;   // channels of a tile

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

// ---- factors ---------------------------------------------------------------------------

__device__ __forceinline__ bool near_one(float f) { return __float_as_int(f) < 0; }
__device__ __forceinline__ float exp2_fast(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
// Whether g is in (bound, -0]: the bits of negative numbers, as signed integers, rise with their magnitude.
__device__ __forceinline__ bool just_below_zero(float g, float bound) { return __float_as_int(g) < __float_as_int(bound); }
// The factors exp(g) of one token.  Above -1/16 the series up to g^4 / 24 leaves less than 2^-22.9 of the distance; the
// hardware's 2^x, off by some 2^-22 of 1, serves elsewhere: there a state's memory is at most 16 tokens (and 2^0 is 1).
__device__ __forceinline__ float2 factor(float2 g) {
    const float2 y = mul2(g, both(1.44269504088896341f));
    float2 d = fma2(g, both(1.f / 24.f), both(1.f / 6.f));
    d = fma2(g, d, both(0.5f));
    d = fma2(g, d, both(1.f));
    d = mul2(g, d);
    return make_float2(just_below_zero(g.x, -0.0625f) ? d.x : exp2_fast(y.x), just_below_zero(g.y, -0.0625f) ? d.y : exp2_fast(y.y));
}
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
// a h
__device__ __forceinline__ float2 decayed(float2 f, float2 h) {
    const float2 t = mul2(f, h);
    return add2(t, make_float2(near_one(f.x) ? h.x : 0.f, near_one(f.y) ? h.y : 0.f));
}
// 1 - a
__device__ __forceinline__ float2 forgotten(float2 f) {
    return make_float2((near_one(f.x) ? 0.f : 1.f) - f.x, (near_one(f.y) ? 0.f : 1.f) - f.y);
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
// A lane's two channels of a row of a tile in shared memory.
template <typename T> __device__ __forceinline__ float2 pair_at(const T *tile, int row) {
    return Pair<T>::get(reinterpret_cast<const typename Pair<T>::type *>(tile)[row * (kLrWide / 2) + (threadIdx.x & 31)]);
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

// Rows n0 ... n0 + ROWS - 1 of a tensor, channels c0 ... c0 + 63, to a tile in shared memory, in pieces of N numbers, by the
// threads of the compute warps; 0 past the ends.
template <typename T, int ROWS, int N, int UNROLL>
__device__ __forceinline__ void load_pieces(T *tile, const LinrecTensor &x, const LinrecArgs &a, uint32_t n0, long long c0) {
    constexpr int PER = kLrWide / N, STEP = kLrCompute / PER;   // pieces of a row, rows at a time
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
    T *dst = tile + row0 * kLrWide + col;
#pragma unroll(UNROLL)
    for (int row = row0; row < ROWS; row += STEP) {
        const bool there = in && n < (uint32_t)a.total;
        if constexpr (N * sizeof(T) == 2) *dst = there ? *src : from_f32<T>(0.f);
        else copy_async<N * sizeof(T)>(smem_u32(dst), there ? src : base, there);
        n += STEP;
        src += step;
        dst += STEP * kLrWide;
        if (!x.flat) {
            for (t += STEP; t >= (uint32_t)a.tokens; t -= (uint32_t)a.tokens) src += x.seq - (long long)a.tokens * x.tok;
        }
    }
}
template <typename T, int ROWS>
__device__ __forceinline__ void load_tile(T *tile, const LinrecTensor &x, const LinrecArgs &a, uint32_t n0, long long c0) {
    if (x.piece == 16) {
        if (x.flat) {
            LinrecTensor y = x;
            y.flat = true;
            load_pieces<T, ROWS, 16 / sizeof(T), 8>(tile, y, a, n0, c0);
        } else {
            load_pieces<T, ROWS, 16 / sizeof(T), 1>(tile, x, a, n0, c0);
        }
    } else if (sizeof(T) == 4 || x.piece == 4) {
        load_pieces<T, ROWS, 4 / sizeof(T), 1>(tile, x, a, n0, c0);
    } else {
        load_pieces<T, ROWS, 1, 1>(tile, x, a, n0, c0);
    }
}

// Inputs whose rows are evenly spaced, on multiples of 16 bytes, come by tensor copies of whole tiles, one thread's doing;
// others in pieces of 16, 4 or 2 bytes by all compute warps.
struct LinrecMaps {
    CUtensorMap g, x, d;
};
__device__ __forceinline__ void tile_copy(void *tile, const CUtensorMap &map, uint32_t n0, int c0, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(smem_u32(tile)), "l"(&map), "r"(c0), "r"((int)n0), "r"(smem_u32(bar)) : "memory");
}

// ---- starts and ends -------------------------------------------------------------------

template <int TOKENS> struct Marks {
    uint32_t start[TOKENS / 32], end[TOKENS / 32];      // bits of tokens that are a sequence's first, its last
    int32_t start_seq[TOKENS], end_seq[TOKENS];         // whose
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
        const bool inside = t0 > 0 && t0 + TOKENS < tokens;   // of one sequence
        for (int i = 0; i < TOKENS / 32; ++i) {
            uint32_t s = 0, e = 0;
            if (!inside) {
                const uint32_t n = n0 + 32 * i + lane, seq = n / tokens, t = n - seq * tokens;
                const bool in = n < (uint32_t)a.total;
                s = __ballot_sync(0xffffffffu, in && t == 0);
                e = __ballot_sync(0xffffffffu, in && t == tokens - 1);
                m.start_seq[32 * i + lane] = m.end_seq[32 * i + lane] = (int32_t)seq;
            }
            any_s |= s;
            any_e |= e;
            if (lane == 0) {
                m.start[i] = s;
                m.end[i] = e;
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
                    m.start_seq[s - n0] = (int32_t)i;
                    any_s = true;
                }
                if (e > n0 && e <= n1) {
                    atomicOr(&m.end[(e - 1 - n0) / 32], 1u << ((e - 1 - n0) & 31));
                    m.end_seq[e - 1 - n0] = (int32_t)i;
                    any_e = true;
                }
            } else if (to != nullptr && s >= n0 && (s < n1 || last_tile)) {
                for (long long c = c0; c < min(c0 + kLrWide, a.channels); ++c)
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
// The bits of the tokens of warp w's run.
template <int R, int N> __device__ __forceinline__ uint32_t run_bits(const uint32_t (&bits)[N], int w) {
    static_assert(N * 32 == kLrWarps * R, "a bit a token");
    return bits[w * R / 32] >> (w * R % 32) & (R == 32 ? 0xffffffffu : (1u << (R % 32)) - 1);
}

// A warp's run of the tile of a ticket, and a lane's channels.
template <int R> struct Run {
    uint32_t first, starts, ends;
    long long ch;
    bool in0, in1, whole;   // whether the lane's channels are there; whether outputs' pairs are, and on multiples of two numbers
    bool plain;             // no start or end, all tokens held, all pairs whole
    int warp;
    template <int TOKENS>
    __device__ __forceinline__ Run(const LinrecArgs &a, const Marks<TOKENS> &m, unsigned ticket, int k, int warp_) : warp(warp_) {
        first = (uint32_t)k * TOKENS + warp * R;
        ch = (long long)(ticket % (unsigned)a.blocks) * kLrWide + 2 * (threadIdx.x & 31);
        in0 = ch < a.channels;
        in1 = ch + 1 < a.channels;
        whole = in1 && a.pairs;
        starts = run_bits<R>(m.start, warp);
        ends = run_bits<R>(m.end, warp);
        plain = (starts | ends) == 0 && __all_sync(0xffffffffu, whole || !in0) && first - m.lo < m.held && first - m.lo + R <= m.held;
    }
    template <int TOKENS> __device__ __forceinline__ float2 start(const LinrecArgs &a, const Marks<TOKENS> &m, int i) const {
        return get_f32(a.h0 ? a.h0 + m.start_seq[warp * R + i] * a.channels + ch : nullptr, in0, in1);
    }
    template <int TOKENS> __device__ __forceinline__ float2 end(const LinrecArgs &a, const Marks<TOKENS> &m, int i) const {
        return get_f32(a.dht ? a.dht + m.end_seq[warp * R + i] * a.channels + ch : nullptr, in0, in1);
    }
};

// ---- look-back -------------------------------------------------------------------------

// What a tile tells, its map and the state behind it, is 32-bit words that hold kUntold until then: a reader that finds
// another bit pattern in a word has the number, without flags, and so without the fences that would order a flag behind
// the numbers (a fence also waits for the outputs that its SM has under way).  No result is kUntold: a NaN with
// that pattern is told as another.
constexpr uint32_t kUntold = 0xffffffffu;

__device__ __forceinline__ bool told(float x) { return __float_as_uint(x) != kUntold; }
__device__ __forceinline__ float telling(float x) { return told(x) ? x : __uint_as_float(0x7fffffffu); }
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
// Of a lane's two channels of the k-th tile of a block of channels.
__device__ __forceinline__ size_t tile_at(const LinrecArgs &a, int k, int block) {
    return ((size_t)k * a.blocks + block) * 32 + (threadIdx.x & 31);
}

// What the runs of a tile come to.
struct Sums {
    float2 s[kLrWarps][32];   // sums of log decays
    float2 f[kLrWarps][32];   // their factors
    float2 b[kLrWarps][32];   // what the run adds
};

// What a CTA's warps share beside its tiles.
template <int R> struct Shared {
    static constexpr int TOKENS = kLrWarps * R;
    Sums sums;
    float2 before[32];           // the state before the tile, in the direction of the recurrence
    Marks<TOKENS> marks[2];
    unsigned ticket[2];
    uint64_t landed, summed;     // the tile's inputs are there; all runs are summed
    uint64_t read;               // and g and x no longer needed (backward; forward they are not when runs are summed)
};
// Barriers by number.  1: marks are set, and pieces of tiles have landed; 2: the next ticket is known (tiles in pieces);
// 3: the state before the tile is known; 4: among the compute warps.  The ninth warp never waits at 1 to 3.
__device__ __forceinline__ void pass_by(int id) { asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(kLrThreads) : "memory"); }
__device__ __forceinline__ void meet(int id) { named_barrier(id, kLrThreads); }

// The ninth warp.  `issue(k, block)` has a tile loaded (one lane), where tensor copies do.
//
// Look-back: `at` is the last tile before this one whose state, h, is known (-1: none yet).  A round reads what eight tiles
// have told, from at + 1 on, or, with nothing known, further and further back; a state told replaces h, a map is
// applied to the state before it.  (Lanes go on by themselves: each has its own two channels.)  Rounds begin while the
// tile's inputs are summed; if the state before it is not known when they are, the tile's map is told at once, for others
// to pass over it.  The first tile always tells its state.  Waits end after about two seconds, with NaN.
template <int R, bool BACKWARD, typename Issue>
__device__ __forceinline__ void ninth_warp(const LinrecArgs &a, Shared<R> &sm, const float *from, float *to, bool tensor_copies,
                                           Issue issue) {
    constexpr int TOKENS = Shared<R>::TOKENS, AT_ONCE = 8;
    const int lane = threadIdx.x & 31;
    const unsigned all = (unsigned)a.tiles * (unsigned)a.blocks;
    const bool chained = a.tiles > 1;
    unsigned mine = blockIdx.x;
    if (chained && lane == 0) mine = atomicAdd(a.ticket, 1u) + 1;   // from -1 on
    unsigned ticket = __shfl_sync(0xffffffffu, mine, 0);
    if (lane == 0) {
        sm.ticket[0] = ticket;
        if (tensor_copies && ticket < all) issue(ticket / (unsigned)a.blocks, ticket % (unsigned)a.blocks);
    }
    __syncwarp();
    pass_by(2);
    for (int turn = 0; ticket < all; turn ^= 1) {
        const int k = (int)(ticket / (unsigned)a.blocks), block = (int)(ticket % (unsigned)a.blocks);
        const int tile = BACKWARD ? a.tiles - 1 - k : k;
        Marks<TOKENS> &m = sm.marks[turn];
        mark_tile(m, a, (uint32_t)tile * TOKENS, tile == a.tiles - 1, from, to, (long long)block * kLrWide);
        pass_by(1);
        unsigned next = all;
        if (chained && lane == 0) next = atomicAdd(a.ticket, 1u) + 1;

        const bool any = BACKWARD ? (m.starts | m.ends) != 0 : m.starts != 0;   // a run forgets what came before the tile
        const bool known = k == 0 || any;                                       // so does the state behind it
        const bool needs = k > 0 && (BACKWARD ? m.end[TOKENS / 32 - 1] >> 31 == 0 : (m.start[0] & 1) == 0);
        const size_t stride = (size_t)a.blocks * 32, place = (size_t)block * 32 + lane;
        float2 *const states = a.state + place;
        float4 *const maps = a.map + place;
        float2 h = both(0.f), f = both(0.f), b = both(0.f);
        int at = needs ? -1 : k - 1, back = k - AT_ONCE;
        bool have_next = false, have_sums = false, issued = !tensor_copies;
        uint32_t polls = 0;
        unsigned long long t0 = 0;
        while (true) {
            const bool found = __all_sync(0xffffffffu, at == k - 1);
            if (have_next && !have_sums && (found ? mbar_wait(&sm.summed, turn) || true : mbar_try_wait(&sm.summed, turn))) {
                have_sums = true;
                if (chained) {
                    float2 s = both(0.f);
#pragma unroll 4
                    for (int i = 0; i < kLrWarps; ++i) {
                        const int w = BACKWARD ? kLrWarps - 1 - i : i;
                        const bool reset = any && (run_bits<R>(m.start, w) | (BACKWARD ? run_bits<R>(m.end, w) : 0u)) != 0;
                        const float2 bw = sm.sums.b[w][lane];
                        b = reset ? bw : apply(sm.sums.f[w][lane], b, bw);
                        s = add2(s, sm.sums.s[w][lane]);
                    }
                    f = factor_of_sum(s);
                    if (known) tell(states + k * stride, b);
                    else if (!found) tell(maps + k * stride, f, b);
                }
            }
            if (have_sums && !issued && (!BACKWARD || (found ? mbar_wait(&sm.read, turn) || true : mbar_try_wait(&sm.read, turn)))) {
                issued = true;
                if (lane == 0 && next < all) issue(next / (unsigned)a.blocks, next % (unsigned)a.blocks);
                __syncwarp();
            }
            if (found && have_sums && issued) break;
            if (!found) {
                const int j = at >= 0 ? at + 1 : back;
                float2 st[AT_ONCE];
                float4 mp[AT_ONCE];
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i)
                    if (j + i >= 0 && j + i < k) {
                        st[i] = ask(states + (j + i) * stride);
                        mp[i] = ask(maps + (j + i) * stride);
                    }
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i)
                    if (j + i >= 0 && j + i < k) {
                        if (told(st[i])) {
                            h = st[i];
                            at = j + i;
                        } else if (at == j + i - 1 && at >= 0 && told(mp[i])) {
                            h = apply(make_float2(mp[i].x, mp[i].y), h, make_float2(mp[i].z, mp[i].w));
                            at = j + i;
                        }
                    }
                if (at < 0) back = back > 0 ? back - AT_ONCE : k - AT_ONCE;
                if (have_sums && ++polls > 4) {
                    if (polls == 5) t0 = global_ns();
                    const bool late = global_ns() - t0 > kMbarWaitLimitNs;
                    if (__shfl_sync(0xffffffffu, (int)late, 0)) {
                        h = both(__uint_as_float(0x7fffffffu));
                        at = k - 1;
                    }
                }
            }
            if (!have_next) {   // the atomic has had the time of a round
                next = __shfl_sync(0xffffffffu, next, 0);
                if (lane == 0) sm.ticket[turn ^ 1] = next;
                have_next = true;
                __syncwarp();
                if (!tensor_copies) pass_by(2);
            }
        }
        if (chained && !known) tell(states + k * stride, apply(f, h, b));
        sm.before[lane] = h;
        __syncwarp();
        pass_by(3);
        ticket = next;
    }
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
