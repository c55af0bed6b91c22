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
    alignas(128) TG g[kLrWarps * R * kLrWide];
    alignas(128) TX x[kLrWarps * R * kLrWide];
    alignas(128) TX dh[2][kLrWarps * R * kLrWide];   // the next tile's while this one's second pass is to come
    Shared<R> shared;
    float2 add[kLrWarps][32];                        // what the runs add to h
};

template <typename TX, typename TG, bool TIED, int R>
__global__ void __launch_bounds__(kLrThreads, 2) linrec_backward_kernel(const LinrecArgs a, const __grid_constant__ LinrecMaps maps) {
    typedef BackwardSpace<TX, TG, R> Space;
    constexpr int TOKENS = kLrWarps * R;
    extern __shared__ __align__(128) unsigned char raw[];
    Space &space = *reinterpret_cast<Space *>(raw);
    Shared<R> &sm = space.shared;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned all = (unsigned)a.tiles * (unsigned)a.blocks;
    const bool tensor_copies = a.tensor_copies;
    if (tid == 0) {
        mbar_init(&sm.landed, 1);
        mbar_init(&sm.summed, kLrWarps);
        mbar_init(&sm.read, kLrWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    if (warp == kLrWarps) {
        int stage = 0;
        ninth_warp<R, true>(a, sm, a.dht, a.dh0, tensor_copies, [&](unsigned k, unsigned block) {
            const uint32_t n = (a.tiles - 1 - k) * TOKENS;
            const int c = (int)(block * kLrWide);
            mbar_arrive_expect_tx(&sm.landed, sizeof(space.g) + 2 * sizeof(space.x));
            tile_copy(space.g, maps.g, n, c, &sm.landed);
            tile_copy(space.x, maps.x, n, c, &sm.landed);
            tile_copy(space.dh[stage], maps.d, n, c, &sm.landed);
            stage ^= 1;
        });
        return;
    }

    auto load = [&](unsigned ticket, int stage) {
        const uint32_t n = (a.tiles - 1 - ticket / (unsigned)a.blocks) * TOKENS;
        const long long c = (long long)(ticket % (unsigned)a.blocks) * kLrWide;
        load_tile<TG, TOKENS>(space.g, a.g, a, n, c);
        load_tile<TX, TOKENS>(space.x, a.x, a, n, c);
        load_tile<TX, TOKENS>(space.dh[stage], a.dout, a, n, c);
    };
    meet(2);
    unsigned ticket = sm.ticket[0];
    if (!tensor_copies && ticket < all) load(ticket, 0);
    for (int turn = 0; ticket < all; turn ^= 1) {
        const Marks<TOKENS> &m = sm.marks[turn];
        const int tile = a.tiles - 1 - (int)(ticket / (unsigned)a.blocks);
        const long long ch = (long long)(ticket % (unsigned)a.blocks) * kLrWide + 2 * lane;
        float2 h = get_f32(a.start + (long long)tile * a.channels + ch, ch < a.channels, ch + 1 < a.channels);
        bool whole_tile = true;
        if (tensor_copies) whole_tile = mbar_wait(&sm.landed, turn);
        else copies_landed();
        meet(1);
        const Run<R> r(a, m, ticket, tile, warp);
        const TG *gs = space.g + warp * R * kLrWide;
        const TX *xs = space.x + warp * R * kLrWide, *ds = space.dh[turn] + warp * R * kLrWide;
        float2 f[R], was[R], add = both(0.f), s = both(whole_tile ? 0.f : __uint_as_float(0x7fffffffu)), mu = both(0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 g = pair_at(gs, i);
            f[i] = factor(g);
            s = add2(s, g);
        }
        if ((r.starts | r.ends) == 0) {
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
        sm.sums.s[warp][lane] = s;
        sm.sums.f[warp][lane] = factor_of_sum(s);
        sm.sums.b[warp][lane] = mu;
        space.add[warp][lane] = add;
        __syncwarp();
        if (lane == 0 && tensor_copies) mbar_arrive(&sm.summed);
        named_barrier(4, kLrCompute);
        // the states before each token; with tied inputs less the token's x, as the gradient of g needs them
        for (int w = 0; w < warp; ++w) {
            const float2 b = space.add[w][lane];
            h = m.starts && run_bits<R>(m.start, w) != 0 ? b : apply(sm.sums.f[w][lane], h, b);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 x = pair_at(xs, i);
            if (r.starts >> i & 1) h = r.start(a, m, i);
            was[i] = TIED ? make_float2(h.x - x.x, h.y - x.y) : h;
            h = apply(f[i], h, TIED ? mul2(forgotten(f[i]), x) : x);
        }
        __syncwarp();
        if (tensor_copies) {
            if (lane == 0) mbar_arrive(&sm.read);
        } else {
            meet(2);   // before the ninth warp may come to its next ticket
            if (lane == 0) mbar_arrive(&sm.summed);
            if (sm.ticket[turn ^ 1] < all) load(sm.ticket[turn ^ 1], turn ^ 1);
        }

        meet(3);
        mu = sm.before[lane];
        for (int w = kLrWarps - 1; w > warp; --w) {
            const float2 b = sm.sums.b[w][lane];
            const bool cut = (m.starts | m.ends) && (run_bits<R>(m.start, w) | run_bits<R>(m.end, w)) != 0;
            mu = cut ? b : apply(sm.sums.f[w][lane], mu, b);
        }
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
                    if (a.dh0 != nullptr) put_f32(a.dh0 + m.start_seq[warp * R + i] * a.channels + r.ch, mu, r.in0, r.in1);
                    mu = both(0.f);
                }
                dx -= a.channels;
                dg -= a.channels;
            }
        }
        ticket = sm.ticket[turn ^ 1];
        named_barrier(4, kLrCompute);   // all have read the sums
    }
}

template <typename TX, typename TG, bool TIED> cudaError_t launch(LinrecArgs a, cudaStream_t s) {
    constexpr int R = linrec_start_tokens(sizeof(TX)) / kLrWarps;
    typedef BackwardSpace<TX, TG, R> Space;
    a.tiles = (int)((a.total + kLrWarps * R - 1) / (kLrWarps * R));
    LinrecMaps maps{};
    a.tensor_copies = linrec_tensor_map(maps.g, a.g, a, sizeof(TG), std::is_same<TG, __half>::value, kLrWarps * R) &&
                      linrec_tensor_map(maps.x, a.x, a, sizeof(TX), std::is_same<TX, __half>::value, kLrWarps * R) &&
                      linrec_tensor_map(maps.d, a.dout, a, sizeof(TX), std::is_same<TX, __half>::value, kLrWarps * R);
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
