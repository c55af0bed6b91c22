// linrec_forward.cu -- the gated linear recurrence over whole sequences
// (notation and tiles in linrec_common.cuh).
//
// Memory bounds it from below (x and g are read once, h is written once).  In fact half of the issue slots are in use, and warps
// wait at barriers for a tile's inputs and for the state before it: every run is scanned twice from shared memory, first from 0
// for what it adds, then from the state before it, 33 instructions a number in all (16-bit types).  Kept in registers in between, factors and inputs cost fewer, but so many registers that fewer warps hide each
// other's waits (issue slots 38 instead of 56% in use): one sequence of 131072 tokens 185 us instead of 170 (with runs of 16).  Factors of 32-bit log
// decays take their place in shared memory; those of 16 bits are computed again, as they would be rounded there.
//
// 48 ragged prompts, 24571 tokens by 4096 bf16 channels with f32 log decays: 214 us, 3.8 TB/s.  One sequence of 131072 tokens by
// 512 bf16 channels: 141 us, 2.9 TB/s (its 16 blocks of channels are one chain of 256 tiles each).
#include <type_traits>

#include "linrec_common.cuh"

namespace ps {

namespace {

template <typename TX, typename TG, int R> struct ForwardSpace {
    alignas(128) TG g[kLrRuns * R * kLrWide];
    alignas(128) TX x[kLrRuns * R * kLrWide];
    Shared<R> shared;
};

template <typename TX, typename TG, bool TIED, int R, int CTAS>
__global__ void __launch_bounds__(kLrThreads, CTAS) linrec_forward_kernel(const LinrecArgs a, const __grid_constant__ LinrecMaps maps) {
    typedef ForwardSpace<TX, TG, R> Space;
    constexpr int TOKENS = kLrRuns * R;
    extern __shared__ __align__(128) unsigned char raw[];
    Space &space = *reinterpret_cast<Space *>(raw);
    Shared<R> &sm = space.shared;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool tensor_copies = a.tensor_copies;
    sm.init();

    if (warp == kLrWarps) {
        ninth_warp<R, false>(a, sm, a.h0, a.ht, tensor_copies, [&](const Place &at) {
            mbar_arrive_expect_tx(&sm.landed, sizeof(space.g) + sizeof(space.x));
            tile_copy(space.g, maps.g, at.tile * kLrRuns, at.block * kLrWide, &sm.landed);
            tile_copy(space.x, maps.x, at.tile * kLrRuns, at.block * kLrWide, &sm.landed);
        });
        return;
    }

    TX *const xs = space.x;
    TG *const gs = space.g;
    meet(2);
    Place place = sm.place[0];
    for (int turn = 0; place.tile >= 0; turn ^= 1) {
        const Marks<TOKENS> &m = sm.marks[turn];
        if (tensor_copies) {
            sm.wait_for_inputs(turn);
        } else {
            load_tile<TG, R>(gs, a.g, a, (uint32_t)place.tile * TOKENS, (long long)place.block * kLrWide);
            load_tile<TX, R>(xs, a.x, a, (uint32_t)place.tile * TOKENS, (long long)place.block * kLrWide);
            copies_landed();
        }
        meet(1);
        const Place next_place = sm.place[turn ^ 1];
        Run<R> r(a, m, place);
        if (tensor_copies && r.first < (uint32_t)a.total && r.first + R > (uint32_t)a.total) {
            load_last_run<TG, R>(gs, a.g, a, r.first, r.ch);
            load_last_run<TX, R>(xs, a.x, a, r.first, r.ch);
        }
        float2 h = both(0.f), s = both(0.f);
        if (!r.marked) {
#pragma unroll 4
            for (int i = 0; i < R; ++i) {
                const float2 g = pair_at(gs, i);
                const Token t = Token::of<kWeights<TX, TIED>>(g);
                keep(gs, i, t);
                s = add2(s, g);
                h = t.apply(h, t.weigh(pair_at(xs, i), TIED));
            }
        } else {
#pragma unroll 2
            for (int i = 0; i < R; ++i) {
                const float2 g = pair_at(gs, i);
                const Token t = Token::of<kWeights<TX, TIED>>(g);
                keep(gs, i, t);
                s = add2(s, g);
                if (r.starts >> i & 1) h = r.start(a, m, i);
                h = t.apply(h, t.weigh(pair_at(xs, i), TIED));
            }
        }
        const bool lost = sm.lost;   // whatever was read, h is NaN
        if (lost) h = s = both(nan_f32());
        const Ahead ahead = join_runs<false>(s, factor_of_sum(s), h, r.starts != 0, m.starts != 0, sm.sums.s, sm.sums.f,
                                             sm.sums.b);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.summed);

        meet(3);
        h = before_run<false>(sm.before[lr_pair()], ahead, sm.sums.f, sm.sums.b, m.starts != 0,
                              [&](int w) { return warp_cut<R, false>(m, w); });
        if (lost) {
            h = both(nan_f32());
            r.starts = 0;
        }
        if (a.start != nullptr && (r.first & (a.start_tokens - 1)) == 0 && r.first < (uint32_t)a.total)
            put_f32(a.start + r.first / a.start_tokens * a.channels + r.ch, h, r.in0, r.in1);
        TX *out = static_cast<TX *>(a.h) + (long long)r.first * a.channels + r.ch;
        if (r.plain) {
#pragma unroll 4
            for (int i = 0; i < R; ++i) {
                const Token t = token_at<kWeights<TX, TIED>>(gs, i);
                h = t.apply(h, t.weigh(pair_at(xs, i), TIED));
                if (r.in0) *reinterpret_cast<typename Pair<TX>::type *>(out) = Pair<TX>::put(h);
                out += a.channels;
            }
        } else {
#pragma unroll 2
            for (int i = 0; i < R; ++i) {
                const Token t = token_at<kWeights<TX, TIED>>(gs, i);
                if (r.starts >> i & 1) h = r.start(a, m, i);
                h = t.apply(h, t.weigh(pair_at(xs, i), TIED));
                if (r.first + i - m.lo < m.held) put_pair<TX>(out, h, r.whole, r.in0, r.in1);
                if ((r.ends >> i & 1) && a.ht != nullptr) put_f32(a.ht + m.seq[lr_run() * R + i] * a.channels + r.ch, h, r.in0, r.in1);
                out += a.channels;
            }
        }
        if (tensor_copies) sm.release();
        else named_barrier(4, kLrCompute);
        place = next_place;
    }
}

template <typename TX, typename TG, bool TIED> cudaError_t launch(LinrecArgs a, cudaStream_t s) {
    constexpr int R = sizeof(TX) + sizeof(TG) <= 4 ? 32 : 16, CTAS = 3;
    typedef ForwardSpace<TX, TG, R> Space;
    static_assert((sizeof(Space) + 1024) * CTAS <= 228 * 1024, "room for all CTAs of an SM");
    const cudaError_t e0 = linrec_prepare(a, kLrRuns * R, s);
    if (e0 != cudaSuccess) return e0;
    LinrecMaps maps{};
    a.tensor_copies = linrec_tensor_map(maps.g, a.g, a, sizeof(TG), std::is_same<TG, __half>::value, kLrRuns, R) &&
                      linrec_tensor_map(maps.x, a.x, a, sizeof(TX), std::is_same<TX, __half>::value, kLrRuns, R);
    const auto kernel = linrec_forward_kernel<TX, TG, TIED, R, CTAS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Space));
    if (e != cudaSuccess) return e;
    kernel<<<linrec_grid(a, CTAS), kLrThreads, sizeof(Space), s>>>(a, maps);
    return cudaGetLastError();
}
template <typename TX, typename TG> cudaError_t launch(const LinrecArgs &a, bool tied, cudaStream_t s) {
    return tied ? launch<TX, TG, true>(a, s) : launch<TX, TG, false>(a, s);
}

}  // namespace

cudaError_t launch_linrec_forward(const LinrecArgs &a, int type, int gate_type, bool tied, cudaStream_t s) {
#define CALL(TX, TG) launch<TX, TG>(a, tied, s)
    PS_LINREC_DISPATCH(CALL);
#undef CALL
}

}  // namespace ps
