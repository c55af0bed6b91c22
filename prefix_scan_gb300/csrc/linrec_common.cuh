// linrec_common.cuh -- pieces shared by the gated linear recurrence's kernels:
// decays and how a factor is encoded, tile geometry and loads, where sequences
// start and end inside a tile, the look-back among tiles.
//
//     h_t = a_t h_{t-1} + w_t x_t,  a = exp(g),  w = 1 or 1 - a
//     backward, from the last token:  lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,
//     dx_t = w_t lam_t,  dg_t = mu_t (h_{t-1} - [tied] x_t),  dh0 = mu_1
//
// A tile is 128 tokens by 32 V channels.  Warp w of eight holds tokens 16 w ... 16 w + 15, a lane V neighbouring
// channels, so that a warp's loads and stores are whole rows and all of a run's loads are in flight at once.  Sequences are
// cut out of the flat index over all tokens: where one starts the state is set, not multiplied, so short sequences fill
// tiles as long ones do.
//
// Each tile tells the ones behind it its map h -> a h + b, and the state behind it once it knows that.  A tile that
// needs the state before it takes the nearest state that is known and applies the maps since then in order
// (look-back).  The state behind a tile is always its map applied to the state before it, by the same three operations
// wherever this is done, so results do not depend on which states were known when: they repeat bit for bit, which sums
// composed in the order of arrival would not.
//
// Factors.  exp(g) of a slow decay rounds to 2^-24 of 1, and what a state forgets in a token, 1 - exp(g), may be not much
// more than that: an error to one side adds up over the state's whole memory (a thousand tokens and more).  So a factor
// near 1 is kept as its distance from 1 (sign bit set) and applied as h + (w h + b); others are kept as they are
// (sign bit clear), so that a closed gate forgets even a large state.
#pragma once

#include <cstdint>

#include "delta_common.cuh"
#include "linrec_internal.h"
#include "scan_pipeline.cuh"

namespace ps {

namespace {

constexpr int kLrThreads = 32 * kLinrecWarps;

// ---- factors ---------------------------------------------------------------------------

__device__ __forceinline__ bool near_one(float f) { return __float_as_int(f) < 0; }
// The factor exp(g) of one token.  Above -1/16 the series up to g^4 / 24 leaves less than 2^-22.9 of the distance; the
// hardware's 2^x, off by some 2^-22 of 1, serves below, where a state's memory is at most 16 tokens.
__device__ __forceinline__ float factor(float g) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * 1.44269504088896341f));
    const float d = g * fmaf(g, fmaf(g, fmaf(g, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
    return g > -0.0625f && g <= 0.f ? __int_as_float(__float_as_int(d) | 0x80000000) : e;
}
// The factor of many tokens from the sum of their log decays.
__device__ __forceinline__ float factor_of_sum(float s) {
    return s > -0.5f && s <= 0.f ? __int_as_float(__float_as_int(expm1f(s)) | 0x80000000) : expf(s);
}
// a h + b
__device__ __forceinline__ float apply(float f, float h, float b) {
    const float t = fmaf(f, h, b);
    return near_one(f) ? t + h : t;
}
// 1 - a
__device__ __forceinline__ float forgotten(float f) { return near_one(f) ? -f : 1.f - f; }

// ---- loads -----------------------------------------------------------------------------

template <typename T, int V> struct Lanes { T v[V]; };
template <> struct alignas(4) Lanes<__nv_bfloat16, 2> { __nv_bfloat16 v[2]; };
template <> struct alignas(4) Lanes<__half, 2> { __half v[2]; };
template <> struct alignas(8) Lanes<float, 2> { float v[2]; };

// The rows of a strided tensor at consecutive flat tokens.
struct Rows {
    long long off, tok, turn;   // elements
    uint32_t t, tokens;
    __device__ __forceinline__ Rows(const LinrecTensor &x, uint32_t n, uint32_t tokens_) : tok(x.tok), tokens(tokens_) {
        const uint32_t seq = n / tokens;
        t = n - seq * tokens;
        off = (long long)seq * x.seq + (long long)t * tok;
        turn = x.seq - (long long)tokens * tok;
    }
    __device__ __forceinline__ void next() {
        off += tok;
        if (++t == tokens) {
            t = 0;
            off += turn;
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void load_run(Lanes<T, V> (&r)[kLinrecRun], const LinrecTensor &x, uint32_t n0, uint32_t total,
                                         uint32_t tokens, long long ch, long long channels) {
    Rows rows(x, n0, tokens);
    const T *p = static_cast<const T *>(x.p) + ch;
#pragma unroll
    for (int i = 0; i < kLinrecRun; ++i) {
        if (n0 + i < total && ch < channels) {
            r[i] = *reinterpret_cast<const Lanes<T, V> *>(p + rows.off);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) r[i].v[v] = from_f32<T>(0.f);
        }
        rows.next();
    }
}
template <typename T, int V> __device__ __forceinline__ void store_lanes(T *p, const float (&x)[V]) {
    Lanes<T, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = from_f32<T>(x[v]);
    *reinterpret_cast<Lanes<T, V> *>(p) = r;
}

// ---- starts and ends -------------------------------------------------------------------

struct Marks {
    uint32_t start[kLinrecTile / 32], end[kLinrecTile / 32];   // bits of tokens that are a sequence's first, its last
    int32_t start_seq[kLinrecTile], end_seq[kLinrecTile];      // whose
    uint32_t lo, hi;                                           // the tokens that sequences hold
    int64_t from, to;                                          // entries of cu below the tile, and below its end
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
// Fills `m` for the tile whose first token is `n0` (all threads; ends with a barrier).  Empty sequences' states go from
// `from` (nullptr: 0) to `to` (nullptr: nowhere) here, for channels c0 ... c0 + count - 1: in the tile at their offset, or in
// the last one.
__device__ __forceinline__ void mark_tile(Marks &m, const LinrecArgs &a, uint32_t n0, bool last_tile, const float *from,
                                          float *to, long long c0, int count) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.cu == nullptr) {
        if (tid < kLinrecTile) {
            const uint32_t n = n0 + tid, tokens = (uint32_t)a.tokens, seq = n / tokens, t = n - seq * tokens;
            const bool in = n < (uint32_t)a.total;
            const uint32_t s = __ballot_sync(0xffffffffu, in && t == 0), e = __ballot_sync(0xffffffffu, in && t == tokens - 1);
            if (lane == 0) {
                m.start[warp] = s;
                m.end[warp] = e;
            }
            m.start_seq[tid] = m.end_seq[tid] = (int32_t)seq;
        }
        if (tid == 0) {
            m.lo = 0;
            m.hi = (uint32_t)a.total;
        }
        __syncthreads();
        return;
    }
    const uint32_t n1 = n0 + kLinrecTile;
    if (tid < kLinrecTile / 32) m.start[tid] = m.end[tid] = 0;
    if (warp == 1) {
        const long long k = offsets_below(a, n0);
        if (lane == 0) m.from = k;
    } else if (warp == 2) {
        const long long k = last_tile ? a.seqs + 1 : offsets_below(a, n1);
        if (lane == 0) m.to = k;
    } else if (tid == 96) {
        m.lo = offset_at(a, 0);
        m.hi = offset_at(a, a.seqs);
    }
    __syncthreads();
    for (long long i = max(m.from - 1, (int64_t)0) + tid; i < min(m.to, (int64_t)a.seqs); i += kLrThreads) {
        const uint32_t s = offset_at(a, i), e = offset_at(a, i + 1);
        if (e > s) {
            if (s >= n0 && s < n1) {
                atomicOr(&m.start[(s - n0) / 32], 1u << ((s - n0) & 31));
                m.start_seq[s - n0] = (int32_t)i;
            }
            if (e > n0 && e <= n1) {
                atomicOr(&m.end[(e - 1 - n0) / 32], 1u << ((e - 1 - n0) & 31));
                m.end_seq[e - 1 - n0] = (int32_t)i;
            }
        } else if (to != nullptr && s >= n0 && (s < n1 || last_tile)) {
            for (long long c = c0; c < min(c0 + count, a.channels); ++c)
                to[i * a.channels + c] = from ? from[i * a.channels + c] : 0.f;
        }
    }
    __syncthreads();
}
// The 16 bits of warp w's tokens.
__device__ __forceinline__ uint32_t run_bits(const uint32_t (&bits)[kLinrecTile / 32], int w) {
    return bits[w / 2] >> (16 * (w & 1)) & 0xffffu;
}
__device__ __forceinline__ bool any_bits(const uint32_t (&bits)[kLinrecTile / 32]) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kLinrecTile / 32; ++i) x |= bits[i];
    return x != 0;
}

// ---- look-back -------------------------------------------------------------------------

enum { kNothing = 0, kMap = 1, kState = 2 };

__device__ __forceinline__ unsigned flag_acquire(const unsigned *p) {
    unsigned x;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}
// One warp, after its lanes have written what the flag stands for.
__device__ __forceinline__ void publish(unsigned *flag, unsigned what) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;" :: "l"(flag), "r"(what) : "memory");
}
__device__ __forceinline__ size_t tile_at(const LinrecArgs &a, int k, int block) { return (size_t)k * a.blocks + block; }
__device__ __forceinline__ unsigned *flag_of(const LinrecArgs &a, int k, int block) { return a.flag + (size_t)block * a.tiles + k; }

// The state before the k-th tile of a block of channels (k > 0; one warp).  The first tile always publishes its state, so the
// walk ends there at the latest; waits end after about two seconds, with NaN.
template <int V> __device__ __forceinline__ void look_back(float (&carry)[V], const LinrecArgs &a, int k, int block) {
    const int lane = threadIdx.x & 31;
    const unsigned long long t0 = global_ns();
    int pos = k - 1, anchor = -1;
    uint32_t polls = 0;
    while (anchor < 0) {
        const unsigned f = pos - lane >= 0 ? flag_acquire(flag_of(a, pos - lane, block)) : kState;
        const uint32_t states = __ballot_sync(0xffffffffu, f == kState), none = __ballot_sync(0xffffffffu, f == kNothing);
        const int s = __ffs(states), x = __ffs(none);   // 1 + the place, 0 for no such
        if (x != 0 && (s == 0 || x < s)) {
            const bool out = (++polls & 63u) == 0 && global_ns() - t0 > kMbarWaitLimitNs;
            if (__shfl_sync(0xffffffffu, (int)out, 0)) break;
            if (polls > 8) __nanosleep(64);
        } else if (s != 0) {
            anchor = pos - (s - 1);
        } else {
            pos -= 32;
        }
    }
    __syncwarp();
    if (anchor < 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = __int_as_float(0x7fffffff);
        return;
    }
    {
        const float *p = a.state + (tile_at(a, anchor, block) * 32 + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = __ldcg(p + v);
    }
    for (int j = anchor + 1; j < k; j += 8) {
        float2 m[8][V];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j + i < k) {
                const float2 *p = a.map + (tile_at(a, j + i, block) * 32 + lane) * V;
#pragma unroll
                for (int v = 0; v < V; ++v) m[i][v] = __ldcg(p + v);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j + i < k) {
#pragma unroll
                for (int v = 0; v < V; ++v) carry[v] = apply(m[i][v].x, carry[v], m[i][v].y);
            }
    }
}

// What the runs of a tile come to, for one warp's worth of channels: `runs` from the first one in the direction of the
// recurrence, `reset(w)` where the run forgets what came before.
template <int V> struct Sums {
    float s[kLinrecWarps][32 * V];   // sums of log decays
    float b[kLinrecWarps][32 * V];   // what the run adds
};

// Warp 0's part between the two passes: tells the tile's map, finds the state before the tile (or takes it as 0 where the
// tile does not need it) and tells the state behind it.
template <int V, typename Reset>
__device__ __forceinline__ void tile_carry(float (&carry)[V], const LinrecArgs &a, int k, int block, const Sums<V> &sums,
                                           Reset reset, bool any_reset, bool needs, bool backward) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = 0.f;
    if (a.tiles == 1) return;
    float f[V], b[V];
    {
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = b[v] = 0.f;
        for (int i = 0; i < kLinrecWarps; ++i) {
            const int w = backward ? kLinrecWarps - 1 - i : i;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float sw = sums.s[w][lane * V + v], bw = sums.b[w][lane * V + v];
                b[v] = reset(w) ? bw : apply(factor_of_sum(sw), b[v], bw);
                s[v] += sw;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = factor_of_sum(s[v]);
    }
    const size_t at = (tile_at(a, k, block) * 32 + lane) * V;
    const bool known = any_reset || k == 0;
    if (known) {
#pragma unroll
        for (int v = 0; v < V; ++v) __stcg(a.state + at + v, b[v]);
        publish(flag_of(a, k, block), kState);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) __stcg(a.map + at + v, make_float2(f[v], b[v]));
        publish(flag_of(a, k, block), kMap);
    }
    if (k > 0 && needs) look_back<V>(carry, a, k, block);
    if (!known) {
#pragma unroll
        for (int v = 0; v < V; ++v) __stcg(a.state + at + v, apply(f[v], carry[v], b[v]));
        publish(flag_of(a, k, block), kState);
    }
}

}  // namespace

// Runs CALL<types, V, tied> for the type codes.
#define PS_LINREC_DISPATCH(CALL)                                                                        \
    do {                                                                                                \
        if (type == PS_REAL_F32) return CALL(float, float);                                             \
        if (type == PS_REAL_BF16 && gate_type == PS_REAL_F32) return CALL(__nv_bfloat16, float);        \
        if (type == PS_REAL_BF16) return CALL(__nv_bfloat16, __nv_bfloat16);                            \
        if (gate_type == PS_REAL_F32) return CALL(__half, float);                                       \
        return CALL(__half, __half);                                                                    \
    } while (0)

}  // namespace ps
