// linrec_forward.cu -- the gated linear recurrence over whole sequences
// (notation and tiles in linrec_common.cuh).
//
// Bound by memory: x and g are read once, h is written once.  A run is scanned once, from 0, and each token's state and the
// factor P of what was there before the run stay in registers; when the state H before the run is known, h + P H goes
// out.  P is a plain product of at most 16 factors: its 2^-20 is of one output alone, as states go from run to run by the
// runs' maps, whose factors come from sums of log decays.
#include <type_traits>

#include "linrec_common.cuh"

namespace ps {

namespace {

template <typename TX, typename TG, int R> struct ForwardSpace {
    alignas(128) TG g[2][kLrRuns * R * kLrWide];   // the next tile's are on their way
    alignas(128) TX x[2][kLrRuns * R * kLrWide];
    Shared<R> shared;
};

template <typename TX, typename TG, bool TIED, int R>
__global__ void __launch_bounds__(kLrThreads, kLinrecCtasPerSm) linrec_forward_kernel(const LinrecArgs a, const __grid_constant__ LinrecMaps maps) {
    typedef ForwardSpace<TX, TG, R> Space;
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
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    if (warp == kLrWarps) {
        ninth_warp<R, false>(a, sm, a.h0, a.ht, tensor_copies, [&](const Place &at, int stage) {
            mbar_arrive_expect_tx(&sm.landed[stage], sizeof(space.g[0]) + sizeof(space.x[0]));
            tile_copy(space.g[stage], maps.g, at.tile * kLrRuns, at.block * kLrWide, &sm.landed[stage]);
            tile_copy(space.x[stage], maps.x, at.tile * kLrRuns, at.block * kLrWide, &sm.landed[stage]);
        });
        return;
    }

    auto load = [&](const Place &at, int stage) {
        load_tile<TG, R>(space.g[stage], a.g, a, (uint32_t)at.tile * TOKENS, (long long)at.block * kLrWide);
        load_tile<TX, R>(space.x[stage], a.x, a, (uint32_t)at.tile * TOKENS, (long long)at.block * kLrWide);
    };
    meet(2);
    Place place = sm.place[0];
    if (!tensor_copies && place.tile >= 0) load(place, 0);
    for (int turn = 0, phase = 0; place.tile >= 0; phase ^= turn, turn ^= 1) {
        const Marks<TOKENS> &m = sm.marks[turn];
        bool whole_tile = true;
        if (tensor_copies) whole_tile = mbar_wait(&sm.landed[turn], phase);
        else copies_landed();
        meet(1);
        const Place next_place = sm.place[turn ^ 1];
        if (!tensor_copies && next_place.tile >= 0) load(next_place, turn ^ 1);
        const Run<R> r(a, m, place);
        TX *xs = space.x[turn];
        TG *gs = space.g[turn];
        if (tensor_copies && r.first < (uint32_t)a.total && r.first + R > (uint32_t)a.total) {
            load_last_run<TG, R>(gs, a.g, a, r.first, r.ch);
            load_last_run<TX, R>(xs, a.x, a, r.first, r.ch);
        }
        float2 hs[R], ps[R], h = both(0.f), p = both(1.f), s = both(whole_tile ? 0.f : __uint_as_float(0x7fffffffu));
        auto token = [&](int i) {
            const float2 g = pair_at(gs, i), x = pair_at(xs, i), f = factor(g);
            s = add2(s, g);
            const float2 one = make_float2(near_one(f.x) ? 1.f : 0.f, near_one(f.y) ? 1.f : 0.f);
            const float2 b = TIED ? mul2(make_float2((near_one(f.x) ? 0.f : 1.f) - f.x, (near_one(f.y) ? 0.f : 1.f) - f.y), x) : x;
            h = fma2(one, h, fma2(f, h, b));
            p = fma2(one, p, mul2(f, p));
            hs[i] = h;
            ps[i] = p;
        };
        if (!r.marked) {
#pragma unroll
            for (int i = 0; i < R; ++i) token(i);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (r.starts >> i & 1) {
                    h = r.start(a, m, i);
                    p = both(0.f);
                }
                token(i);
            }
        }
        const Ahead ahead = join_runs<false>(s, factor_of_sum(s), h, r.starts != 0, m.starts != 0, sm.sums[turn].s, sm.sums[turn].f,
                                             sm.sums[turn].b);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.summed);
        meet(3);
        float2 H = before_run<false>(sm.before[lr_pair()], ahead, sm.sums[turn].f, sm.sums[turn].b, m.starts != 0,
                                     [&](int w) { return warp_cut<R, false>(m, w); });
        if (a.start != nullptr && r.first % a.start_tokens == 0 && r.first < (uint32_t)a.total)
            put_f32(a.start + r.first / a.start_tokens * a.channels + r.ch, H, r.in0, r.in1);
        TX *out = static_cast<TX *>(a.h) + (long long)r.first * a.channels + r.ch;
        if (r.plain) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (r.in0) *reinterpret_cast<typename Pair<TX>::type *>(out) = Pair<TX>::put(fma2(ps[i], H, hs[i]));
                out += a.channels;
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (r.starts >> i & 1) H = both(0.f);   // whatever came before, NaN too, is forgotten
                const float2 y = fma2(ps[i], H, hs[i]);
                if (r.first + i - m.lo < m.held) put_pair<TX>(out, y, r.whole, r.in0, r.in1);
                if ((r.ends >> i & 1) && a.ht != nullptr)
                    put_f32(a.ht + m.end_seq[lr_run() * R + i] * a.channels + r.ch, y, r.in0, r.in1);
                out += a.channels;
            }
        }
        place = next_place;
    }
}

template <typename TX, typename TG, bool TIED> cudaError_t launch(LinrecArgs a, cudaStream_t s) {
    // runs of 8 tokens where 16 of them, twice, leave no room for a second CTA
    constexpr int R = sizeof(TX) + sizeof(TG) <= 6 ? 16 : 8;
    typedef ForwardSpace<TX, TG, R> Space;
    static_assert(sizeof(Space) <= 113 * 1024, "two CTAs an SM");
    const cudaError_t e0 = linrec_prepare(a, kLrRuns * R, s);
    if (e0 != cudaSuccess) return e0;
    LinrecMaps maps{};
    a.tensor_copies = linrec_tensor_map(maps.g, a.g, a, sizeof(TG), std::is_same<TG, __half>::value, kLrRuns, R) &&
                      linrec_tensor_map(maps.x, a.x, a, sizeof(TX), std::is_same<TX, __half>::value, kLrRuns, R);
    const auto kernel = linrec_forward_kernel<TX, TG, TIED, R>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Space));
    if (e != cudaSuccess) return e;
    kernel<<<linrec_grid(a), kLrThreads, sizeof(Space), s>>>(a, maps);
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
