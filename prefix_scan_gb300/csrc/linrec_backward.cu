// linrec_backward.cu -- gradients of the gated linear recurrence (notation and
// tiles in linrec_common.cuh).
//
// Bound by memory: x, g and dh are read once, dx and dg are written once.  The states are not read: the forward pass keeps
// the one before each tile (in 32 bits), and the tile is scanned again from there, so that 16-bit types, too, get the
// gradient of g from states of 32 bits.  What runs backward is mu, a state's gradient handed to the token before; its
// look-back goes over the tiles from the last one.
#include <type_traits>

#include "linrec_common.cuh"

namespace ps {

namespace {

template <typename TX, typename TG, int R> struct BackwardSpace {
    alignas(128) TG g[2][kLrRuns * R * kLrWide];   // the next tile's are on their way
    alignas(128) TX x[2][kLrRuns * R * kLrWide], dh[2][kLrRuns * R * kLrWide];
    float2 add[kLrWarps][kLrPairs];                // what the warps' runs add to h
    Shared<R> shared;
};

template <typename TX, typename TG, bool TIED, int R>
__global__ void __launch_bounds__(kLrThreads, kLinrecCtasPerSm) linrec_backward_kernel(const LinrecArgs a, const __grid_constant__ LinrecMaps maps) {
    typedef BackwardSpace<TX, TG, R> Space;
    constexpr int TOKENS = kLrRuns * R;
    extern __shared__ __align__(128) unsigned char raw[];
    Space &space = *reinterpret_cast<Space *>(raw);
    Shared<R> &sm = space.shared;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool tensor_copies = a.tensor_copies;
    if (tid == 0) {
        mbar_init(&sm.landed[0], 1);
        mbar_init(&sm.landed[1], 1);
        mbar_init(&sm.summed, kLrWarps);
        mbar_init(&sm.done, kLrWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    if (warp == kLrWarps) {
        ninth_warp<R, true>(a, sm, a.dht, a.dh0, tensor_copies, [&](const Place &at, int stage) {
            const int n = at.tile * kLrRuns, c = at.block * kLrWide;
            mbar_arrive_expect_tx(&sm.landed[stage], sizeof(space.g[0]) + 2 * sizeof(space.x[0]));
            tile_copy(space.g[stage], maps.g, n, c, &sm.landed[stage]);
            tile_copy(space.x[stage], maps.x, n, c, &sm.landed[stage]);
            tile_copy(space.dh[stage], maps.d, n, c, &sm.landed[stage]);
        });
        return;
    }

    auto load = [&](const Place &at, int stage) {
        const uint32_t n = (uint32_t)at.tile * TOKENS;
        const long long c = (long long)at.block * kLrWide;
        load_tile<TG, R>(space.g[stage], a.g, a, n, c);
        load_tile<TX, R>(space.x[stage], a.x, a, n, c);
        load_tile<TX, R>(space.dh[stage], a.dout, a, n, c);
    };
    meet(2);
    Place place = sm.place[0];
    if (!tensor_copies && place.tile >= 0) load(place, 0);
    for (int turn = 0, phase = 0; place.tile >= 0; phase ^= turn, turn ^= 1) {
        const Marks<TOKENS> &m = sm.marks[turn];
        const float2 first = get_f32(a.start + (long long)place.tile * a.channels + (long long)place.block * kLrWide + 2 * lr_pair(),
                                     place.block * kLrWide + 2 * lr_pair() < a.channels, place.block * kLrWide + 2 * lr_pair() + 1 < a.channels);
        bool whole_tile = true;
        if (tensor_copies) whole_tile = mbar_wait(&sm.landed[turn], phase);
        else copies_landed();
        meet(1);
        const Place next_place = sm.place[turn ^ 1];
        if (!tensor_copies && next_place.tile >= 0) load(next_place, turn ^ 1);
        const Run<R> r(a, m, place);
        TG *gs = space.g[turn];
        TX *xs = space.x[turn], *ds = space.dh[turn];
        if (tensor_copies && r.first < (uint32_t)a.total && r.first + R > (uint32_t)a.total) {
            load_last_run<TG, R>(gs, a.g, a, r.first, r.ch);
            load_last_run<TX, R>(xs, a.x, a, r.first, r.ch);
            load_last_run<TX, R>(ds, a.dout, a, r.first, r.ch);
        }
        float2 f[R], was[R], add = both(0.f), s = both(whole_tile ? 0.f : __uint_as_float(0x7fffffffu)), mu = both(0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 g = pair_at(gs, i);
            f[i] = factor(g);
            s = add2(s, g);
        }
        if (!r.marked) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float2 x = pair_at(xs, i);
                add = apply(f[i], add, TIED ? mul2(forgotten(f[i]), x) : x);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) mu = decayed(f[i], add2(pair_at(ds, i), mu));
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float2 x = pair_at(xs, i);
                if (r.starts >> i & 1) add = r.start(a, m, i);
                add = apply(f[i], add, TIED ? mul2(forgotten(f[i]), x) : x);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                if (r.ends >> i & 1) mu = r.end(a, m, i);
                mu = decayed(f[i], add2(pair_at(ds, i), mu));
                if (r.starts >> i & 1) mu = both(0.f);   // dh0 takes it
            }
        }
        const float2 own = factor_of_sum(s);
        const Ahead behind = join_runs<true>(s, own, mu, (r.starts | r.ends) != 0, (m.starts | m.ends) != 0, sm.sums[turn].s,
                                             sm.sums[turn].f, sm.sums[turn].b);
        const Ahead ahead = join_runs<false>(s, own, add, r.starts != 0, m.starts != 0, nullptr, nullptr, space.add);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.summed);
        named_barrier(4, kLrCompute);
        // the states before each token; with tied inputs less the token's x, as the gradient of g needs them
        float2 h = before_run<false>(first, ahead, sm.sums[turn].f, space.add, m.starts != 0, [&](int w) { return warp_cut<R, false>(m, w); });
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 x = pair_at(xs, i);
            if (r.starts >> i & 1) h = r.start(a, m, i);
            was[i] = TIED ? make_float2(h.x - x.x, h.y - x.y) : h;
            h = apply(f[i], h, TIED ? mul2(forgotten(f[i]), x) : x);
        }
        meet(3);
        mu = before_run<true>(sm.before[lr_pair()], behind, sm.sums[turn].f, sm.sums[turn].b, (m.starts | m.ends) != 0,
                              [&](int w) { return warp_cut<R, true>(m, w); });
        TX *dx = static_cast<TX *>(a.dx) + (long long)(r.first + R - 1) * a.channels + r.ch;
        TG *dg = static_cast<TG *>(a.dg) + (long long)(r.first + R - 1) * a.channels + r.ch;
        if (r.plain) {
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const float2 lam = add2(pair_at(ds, i), mu);
                mu = decayed(f[i], lam);
                if (r.in0) {
                    *reinterpret_cast<typename Pair<TX>::type *>(dx) = Pair<TX>::put(TIED ? mul2(forgotten(f[i]), lam) : lam);
                    *reinterpret_cast<typename Pair<TG>::type *>(dg) = Pair<TG>::put(mul2(mu, was[i]));
                }
                dx -= a.channels;
                dg -= a.channels;
            }
        } else {
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                if (r.ends >> i & 1) mu = r.end(a, m, i);
                const float2 lam = add2(pair_at(ds, i), mu);
                mu = decayed(f[i], lam);
                const bool counts = r.first + i - m.lo < m.held;
                if (r.first + i < (uint32_t)a.total) {
                    put_pair<TX>(dx, counts ? TIED ? mul2(forgotten(f[i]), lam) : lam : both(0.f), r.whole, r.in0, r.in1);
                    put_pair<TG>(dg, counts ? mul2(mu, was[i]) : both(0.f), r.whole, r.in0, r.in1);
                }
                if (r.starts >> i & 1) {
                    if (a.dh0 != nullptr) put_f32(a.dh0 + m.start_seq[lr_run() * R + i] * a.channels + r.ch, mu, r.in0, r.in1);
                    mu = both(0.f);
                }
                dx -= a.channels;
                dg -= a.channels;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.done);
        place = next_place;
    }
}

template <typename TX, typename TG, bool TIED> cudaError_t launch(LinrecArgs a, cudaStream_t s) {
    constexpr int R = linrec_start_tokens(sizeof(TX), sizeof(TG)) / kLrRuns;
    typedef BackwardSpace<TX, TG, R> Space;
    static_assert(sizeof(Space) <= 113 * 1024, "two CTAs an SM");
    const cudaError_t e0 = linrec_prepare(a, kLrRuns * R, s);
    if (e0 != cudaSuccess) return e0;
    LinrecMaps maps{};
    a.tensor_copies = linrec_tensor_map(maps.g, a.g, a, sizeof(TG), std::is_same<TG, __half>::value, kLrRuns, R) &&
                      linrec_tensor_map(maps.x, a.x, a, sizeof(TX), std::is_same<TX, __half>::value, kLrRuns, R) &&
                      linrec_tensor_map(maps.d, a.dout, a, sizeof(TX), std::is_same<TX, __half>::value, kLrRuns, R);
    const auto kernel = linrec_backward_kernel<TX, TG, TIED, R>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Space));
    if (e != cudaSuccess) return e;
    kernel<<<linrec_grid(a), kLrThreads, sizeof(Space), s>>>(a, maps);
    return cudaGetLastError();
}
template <typename TX, typename TG> cudaError_t launch(const LinrecArgs &a, bool tied, cudaStream_t s) {
    return tied ? launch<TX, TG, true>(a, s) : launch<TX, TG, false>(a, s);
}

}  // namespace

cudaError_t launch_linrec_backward(const LinrecArgs &a, int type, int gate_type, bool tied, cudaStream_t s) {
#define CALL(TX, TG) launch<TX, TG>(a, tied, s)
    PS_LINREC_DISPATCH(CALL);
#undef CALL
}

}  // namespace ps
