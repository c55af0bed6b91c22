// linrec_backward.cu -- gradients of the gated linear recurrence (notation and
// tiles in linrec_common.cuh).
//
// Memory bounds it from below (x, g and dh are read once, dx and dg are written once).  In fact it is 54 instructions a number in
// half of the issue slots, and waits at barriers for a tile's inputs and for what comes from the tile behind it.  The states are not read: the forward pass keeps the one before each tile (in 32 bits), and the tile is scanned again from there,
// so that 16-bit types, too, get the gradient of g from states of 32 bits.  What runs backward is mu, a state's gradient
// handed to the token before; its look-back goes over the tiles from the last one.
//
// A run's first scan is forward only: what it adds to mu is the sum of P_i dh_i, P_i the product of its factors up to token i.
// The second takes eight tokens at a time, the last ones first: forward for the states before them, from what the first
// scan kept there (a state from 0, and P), then backward: a step back from a state would divide by factors near 0.
//
// Runs with starts or ends, which are few as a rule, go backward in rolled loops (their arrays in local memory): the others' code
// then stays in the instruction cache and in registers.  So do all runs of rows whose pairs are not whole or not on multiples of
// two numbers, odd channel counts among them: 8192 tokens by 4097 bf16 channels take 206 us, by 4096 95 (forward 126 and 64, where
// such rows are loaded number by number, too).
//
// 4 sequences of 8192 tokens by 4096 bf16 channels, forward and backward: 458 us, of which this is about 280 (earlier, all in unrolled
// loops 495, rolled by twos 465); 65536 tokens by 512 f32 channels, tied: 278 us.
#include <type_traits>

#include "linrec_common.cuh"

namespace ps {

namespace {

constexpr int kPart = 8;   // tokens

template <typename TX, typename TG, int R> struct BackwardSpace {
    alignas(128) TG g[kLrRuns * R * kLrWide];
    alignas(128) TX x[kLrRuns * R * kLrWide], dh[kLrRuns * R * kLrWide];
    float2 add[kLrWarps][kLrPairs];   // what the warps' runs add to h
    Shared<R> shared;
};

template <typename TX, typename TG, bool TIED, int R, int CTAS>
__global__ void __launch_bounds__(kLrThreads, CTAS) linrec_backward_kernel(const LinrecArgs a, const __grid_constant__ LinrecMaps maps) {
    typedef BackwardSpace<TX, TG, R> Space;
    constexpr int TOKENS = kLrRuns * R;
    extern __shared__ __align__(128) unsigned char raw[];
    Space &space = *reinterpret_cast<Space *>(raw);
    Shared<R> &sm = space.shared;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool tensor_copies = a.tensor_copies;
    sm.init();

    if (warp == kLrWarps) {
        ninth_warp<R, true>(a, sm, a.dht, a.dh0, tensor_copies, [&](const Place &at) {
            const int n = at.tile * kLrRuns, c = at.block * kLrWide;
            mbar_arrive_expect_tx(&sm.landed, sizeof(space.g) + 2 * sizeof(space.x));
            tile_copy(space.g, maps.g, n, c, &sm.landed);
            tile_copy(space.x, maps.x, n, c, &sm.landed);
            tile_copy(space.dh, maps.d, n, c, &sm.landed);
        });
        return;
    }

    TG *const gs = space.g;
    TX *const xs = space.x, *const ds = space.dh;
    meet(2);
    Place place = sm.place[0];
    for (int turn = 0; place.tile >= 0; turn ^= 1) {
        const Marks<TOKENS> &m = sm.marks[turn];
        const long long ch = (long long)place.block * kLrWide + 2 * lr_pair();
        const float2 first = get_f32(a.start + (long long)place.tile * a.channels + ch, ch < a.channels, ch + 1 < a.channels);
        if (tensor_copies) {
            sm.wait_for_inputs(turn);
        } else {
            const uint32_t n = (uint32_t)place.tile * TOKENS;
            const long long c = (long long)place.block * kLrWide;
            load_tile<TG, R>(gs, a.g, a, n, c);
            load_tile<TX, R>(xs, a.x, a, n, c);
            load_tile<TX, R>(ds, a.dout, a, n, c);
            copies_landed();
        }
        meet(1);
        const Place next_place = sm.place[turn ^ 1];
        Run<R> r(a, m, place);
        if (tensor_copies && r.first < (uint32_t)a.total && r.first + R > (uint32_t)a.total) {
            load_last_run<TG, R>(gs, a.g, a, r.first, r.ch);
            load_last_run<TX, R>(xs, a.x, a, r.first, r.ch);
            load_last_run<TX, R>(ds, a.dout, a, r.first, r.ch);
        }
        float2 add = both(0.f), s = both(0.f), mu = both(0.f), p = both(1.f);
        float2 kept_h[R / kPart], kept_p[R / kPart];   // before each part
#pragma unroll
        for (int q = 0; q < R / kPart; ++q) {
            kept_h[q] = add;
            kept_p[q] = p;
            if (!r.marked) {
#pragma unroll 4
                for (int i = q * kPart; i < (q + 1) * kPart; ++i) {
                    const float2 g = pair_at(gs, i);
                    const Token t = Token::of<kWeights<TX, TIED>>(g);
                    keep(gs, i, t);
                    s = add2(s, g);
                    add = t.apply(add, t.weigh(pair_at(xs, i), TIED));
                    p = t.decayed(p);
                    mu = fma2(p, pair_at(ds, i), mu);
                }
            } else {
#pragma unroll 1
                for (int i = q * kPart; i < (q + 1) * kPart; ++i) {
                    const float2 g = pair_at(gs, i);
                    const Token t = Token::of<kWeights<TX, TIED>>(g);
                    keep(gs, i, t);
                    s = add2(s, g);
                    if (r.starts >> i & 1) {
                        add = r.start(a, m, i);
                        p = both(0.f);
                    }
                    add = t.apply(add, t.weigh(pair_at(xs, i), TIED));
                    p = t.decayed(p);
                }
            }
        }
        if (r.marked) {
#pragma unroll 1
            for (int i = R - 1; i >= 0; --i) {
                if (r.ends >> i & 1) mu = r.end(a, m, i);
                mu = token_at<kWeights<TX, TIED>>(gs, i).decayed(add2(pair_at(ds, i), mu));
                if (r.starts >> i & 1) mu = both(0.f);   // dh0 takes it
            }
        }
        if (sm.lost) s = mu = both(nan_f32());   // whatever was read, mu is NaN, and so is all that is made of it
        const float2 own = factor_of_sum(s);
        const Ahead behind = join_runs<true>(s, own, mu, (r.starts | r.ends) != 0, (m.starts | m.ends) != 0, sm.sums.s,
                                             sm.sums.f, sm.sums.b);
        const Ahead ahead = join_runs<false>(s, own, add, r.starts != 0, m.starts != 0, nullptr, nullptr, space.add);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.summed);

        meet(3);
        const float2 H = before_run<false>(first, ahead, sm.sums.f, space.add, m.starts != 0,
                                           [&](int w) { return warp_cut<R, false>(m, w); });
        mu = before_run<true>(sm.before[lr_pair()], behind, sm.sums.f, sm.sums.b, (m.starts | m.ends) != 0,
                              [&](int w) { return warp_cut<R, true>(m, w); });
        if (sm.lost) {
            mu = both(nan_f32());
            r.ends = 0;
        }
        TX *dx = static_cast<TX *>(a.dx) + (long long)(r.first + R - 1) * a.channels + r.ch;
        TG *dg = static_cast<TG *>(a.dg) + (long long)(r.first + R - 1) * a.channels + r.ch;
        auto part = [&](int q, float2 h, auto marked) {
            constexpr int UNROLL = decltype(marked)::value ? 1 : kPart;
            float2 f[kPart], was[kPart];   // the states before each token; with tied inputs less the token's x, as dg needs them
#pragma unroll UNROLL
            for (int i = 0; i < kPart; ++i) {
                const Token t = token_at<kWeights<TX, TIED>>(gs, q * kPart + i);
                const float2 x = pair_at(xs, q * kPart + i);
                if (marked && (r.starts >> (q * kPart + i) & 1)) h = r.start(a, m, q * kPart + i);
                f[i] = t.f;
                was[i] = TIED ? make_float2(h.x - x.x, h.y - x.y) : h;
                h = t.apply(h, t.weigh(x, TIED));
            }
#pragma unroll UNROLL
            for (int i = kPart - 1; i >= 0; --i) {
                if (marked && (r.ends >> (q * kPart + i) & 1)) mu = r.end(a, m, q * kPart + i);
                const float2 lam = add2(pair_at(ds, q * kPart + i), mu);
                const Token t = Token::from(f[i]);
                const float2 gx = t.weigh(lam, TIED);
                mu = t.decayed(lam);
                const float2 gg = mul2(mu, was[i]);
                if (!marked) {
                    if (r.in0) {
                        *reinterpret_cast<typename Pair<TX>::type *>(dx) = Pair<TX>::put(gx);
                        *reinterpret_cast<typename Pair<TG>::type *>(dg) = Pair<TG>::put(gg);
                    }
                } else {
                    const uint32_t n = r.first + q * kPart + i;
                    const bool counts = n - m.lo < m.held;
                    if (n < (uint32_t)a.total) {
                        put_pair<TX>(dx, counts ? gx : both(0.f), r.whole, r.in0, r.in1);
                        put_pair<TG>(dg, counts ? gg : both(0.f), r.whole, r.in0, r.in1);
                    }
                    if (r.starts >> (q * kPart + i) & 1) {
                        if (a.dh0 != nullptr) put_f32(a.dh0 + m.seq[lr_run() * R + q * kPart + i] * a.channels + r.ch, mu, r.in0, r.in1);
                        mu = both(sm.lost ? nan_f32() : 0.f);
                    }
                }
                dx -= a.channels;
                dg -= a.channels;
            }
        };
#pragma unroll
        for (int q = R / kPart - 1; q >= 0; --q) {
            // where a start came before the part P is 0, and whatever was before it, NaN too, is forgotten
            const float2 h = q == 0 ? H : r.starts & ((1u << (q * kPart)) - 1) ? kept_h[q] : fma2(kept_p[q], H, kept_h[q]);
            if (r.plain) part(q, h, std::false_type{});
            else part(q, h, std::true_type{});
        }
        if (tensor_copies) sm.release();
        named_barrier(4, kLrCompute);   // all have read what the warps' runs add
        place = next_place;
    }
}

template <typename TX, typename TG, bool TIED> cudaError_t launch(LinrecArgs a, cudaStream_t s) {
    constexpr int R = linrec_start_tokens(sizeof(TX), sizeof(TG)) / kLrRuns;
    typedef BackwardSpace<TX, TG, R> Space;
    constexpr int CTAS = 3;
    static_assert((sizeof(Space) + 1024) * CTAS <= 228 * 1024, "room for all CTAs of an SM");
    const cudaError_t e0 = linrec_prepare(a, kLrRuns * R, s);
    if (e0 != cudaSuccess) return e0;
    LinrecMaps maps{};
    a.tensor_copies = linrec_tensor_map(maps.g, a.g, a, sizeof(TG), std::is_same<TG, __half>::value, kLrRuns, R) &&
                      linrec_tensor_map(maps.x, a.x, a, sizeof(TX), std::is_same<TX, __half>::value, kLrRuns, R) &&
                      linrec_tensor_map(maps.d, a.dout, a, sizeof(TX), std::is_same<TX, __half>::value, kLrRuns, R);
    const auto kernel = linrec_backward_kernel<TX, TG, TIED, R, CTAS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Space));
    if (e != cudaSuccess) return e;
    kernel<<<linrec_grid(a, CTAS), kLrThreads, sizeof(Space), s>>>(a, maps);
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
