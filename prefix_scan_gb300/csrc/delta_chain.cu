// delta_chain.cu -- the gated delta rule's states, chunk after chunk, and its
// outputs (notation in delta_common.cuh).
//
// One CTA per sequence, value head and block of 128 values.  Everything is held
// transposed: values are the 128 rows of the tensor-memory accumulators, and the
// left operand of each product is the result of the one before it, split into
// pairs of bf16 and put back into tensor memory, while keys, queries, T and P are
// right operands in shared memory:
//     X^T = S^T K^T           U^T = (beta R)^T T^T
//     S'^T = exp(G_C) S^T + (exp(G_C - G) U)^T K
//     O^T = scale exp(G) (S^T Q^T) + U^T P^T
// The state stays in tensor memory from the first chunk to the last.  T and P are
// lower triangular.
//
// A product of 128 rows, 16 inner and up to 128 columns takes 64 clocks however
// few the columns (measured), so keys and queries are one operand of 128 columns,
// and so are the two parts of T: U comes as two accumulators, added on their way out
// (to beta R: the image holds T - 1, so that the greater part of U passes no pair).
//
// Bounded by the chain S -> X -> U -> S' of each chunk: three products and, between
// them, the way of 128 x 128 and twice 128 x 64 numbers through registers.  So the
// warps have roles: one issues products, two load the next chunk (one its values),
// one stores what training keeps, eight convert on the chain (row = lane, half of
// the columns each), and four take the outputs, which the chain does not wait for:
// U^T P^T of a chunk runs while the next one's X is on its way through registers.
//
// Long sequences over few heads come in segments (DeltaArgs::seg): the first of two
// passes takes the states alone, and one more chain per segment finds its matrix M.
//
// Measured at 128 x 128 and bf16: a chunk takes 5600 clocks of its chain, products
// being issued in about half of them (tensor pipe 33 % busy).  12345 tokens in 48
// sequences, 32 heads: 231 us; 4 x 4096 tokens, 16 heads, with what training keeps:
// 246 us; 32768 tokens, 8 heads: two passes of 128 us (uncut, 1.3 ms).
#include "delta_tmem.cuh"

namespace ps {

namespace {

constexpr int kChainThreads = 16 * 32, kFirstConvert = 4, kFirstOut = 12;   // warps
// Tensor-memory columns: S; its pair, later U's two accumulators; X and S^T Q^T; the pair of beta R,
// later of U; the pair of exp(G_C - G) U, later U^T P^T.
constexpr uint32_t kColS = 0, kColSHi = 128, kColSLo = 192, kColU = 128, kColX = 256, kColQ = 320, kColR = 384, kColW = 448;
constexpr uint32_t kColO = kColW;

template <typename T, int KP>
struct ChainSmem {
    static constexpr int NP = Planes<T>::NP;
    static constexpr int kKQ = NP * (KP / 64) * kHalf, kTP = 4 * (int)kSquare;
    static constexpr int kStages = NP == 1 || (KP == 64 && sizeof(T) == 2) ? 2 : 1;   // as many as there is room for
    static constexpr int kScal = 256, kTiles = 2048, kStage = kKQ + kTP;   // barriers and scalars come first
    static constexpr int kVRow = kBlockV * (int)sizeof(T), kVTile = kChunk * kVRow, kV = kTiles + kStages * kStage;
    // outputs; S on its way out in training; U, which at K = 128 takes the place of T and of the queries
    // (both used by then) in its stage
    static constexpr int kOut = kV + kVTile, kSave = kOut + kVTile, kSaveU = kSave + 2 * (KP / 64) * kHalf;
    static constexpr bool kInStage = KP == 128;
    static constexpr int kBytes = kSave, kTrainBytes = kSaveU + (kInStage ? 0 : 2 * kHalf);
    static_assert(kTrainBytes <= 227 * 1024, "too much shared memory");
};
struct ChainBars {
    uint64_t full[2], empty[2], v_full, v_empty, s_ready[2], x_done, q_read, r_ready, u_done, w_ready, u_ready, s_done, o_done, o_read, s_kept, s_free, u_free, drained;
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(ChainBars) <= 256, "barriers precede the scalars");

}  // namespace

template <typename T, int KP>
__global__ void __launch_bounds__(kChainThreads, 1) delta_chain_kernel(const DeltaArgs a) {
    using M = ChainSmem<T, KP>;
    constexpr int NP = M::NP, KH = KP / 64;
    extern __shared__ __align__(1024) unsigned char smem[];
    ChainBars &bar = *reinterpret_cast<ChainBars *>(smem);
    volatile int *gave_up = &bar.gave_up;
    const uint32_t base = smem_addr(smem);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // known to be uniform
    const bool states = a.pass == kPassStates;   // of segments, without outputs
    const int blocks = blocks_v(a.s.v) + states, rep = a.s.hv / a.s.hk;
    const int vb = (int)(blockIdx.x % blocks);
    const int head = (int)(blockIdx.x / blocks % a.s.hv);
    const bool matrix = states && vb == blocks - 1;   // this chain finds M
    Chain chain;
    if (!chain_of(a, blockIdx.x / blocks / a.s.hv, chain)) return;
    if (states && (chain.last || (matrix && chain.first))) return;   // nobody needs it
    const long long seq = chain.seq;
    const Span sp = chain.span;
    const int v0 = matrix ? 0 : vb * kBlockV;
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, a.train != 0);
    const int chunks = (int)((sp.len + kChunk - 1) / kChunk);
    const bool keep = a.train && !states;
    // the state at the start and where it goes at the end
    const size_t one_state = (size_t)a.s.k * a.s.v;
    const float *from = chain.first ? (a.h0 ? a.h0 + (size_t)(seq * a.s.hv + head) * one_state : nullptr)
                        : states   ? nullptr
                                   : a.seg_state + (size_t)(chain.slot * a.s.hv + head) * one_state;
    float *to_state = states ? (matrix ? nullptr : a.seg_state + (size_t)((chain.slot + 1) * a.s.hv + head) * one_state)
                      : chain.last && a.ht ? a.ht + (size_t)(seq * a.s.hv + head) * one_state
                                           : nullptr;
    auto chunk_ws = [&](int c) { return a.ws + (size_t)((sp.slot + c) * a.s.hv + head) * lay.stride; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], states ? 1 : 1 + 4 + (keep && M::kInStage));
        }
        mbar_init(&bar.v_full, 32);
        mbar_init(&bar.v_empty, 8);
        mbar_init(&bar.s_ready[0], 8);
        mbar_init(&bar.s_ready[1], 8);
        mbar_init(&bar.x_done, 1);
        mbar_init(&bar.q_read, 4);
        mbar_init(&bar.r_ready, 8);
        mbar_init(&bar.u_done, 1);
        mbar_init(&bar.w_ready, 8);
        mbar_init(&bar.u_ready, 8);
        mbar_init(&bar.s_done, 1);
        mbar_init(&bar.o_done, 1);
        mbar_init(&bar.o_read, 4);
        mbar_init(&bar.s_kept, 8);
        mbar_init(&bar.s_free, 1);
        mbar_init(&bar.u_free, 1);
        mbar_init(&bar.drained, 1);
        bar.gave_up = base & 1023 ? 1 : 0;   // images need their alignment
        mbar_init_done();
    }
    if (warp == 0) tmem_alloc(smem_addr(&bar.tmem));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    constexpr uint32_t tm = 0;   // all columns are this CTA's
    if (threadIdx.x == 0 && bar.tmem != tm) bar.gave_up = 1;

    if (warp == 0) {
        const uint32_t one = elect_lane();
        {
            // operands: keys and queries by rows, keys by columns, T and P after it
            const uint64_t kq0 = operand(base + M::kTiles, true, 0), kt0 = operand(base + M::kTiles, false, kHalf);
            // U^T P^T, all of it: leaving out that tokens 16 k.. of U reach no earlier ones would save no time,
            // and accumulators of different shapes have no order among them
            auto outputs = [&](int c) {
                const int st = c % M::kStages;
                const uint64_t pp = further(kq0, st * M::kStage + M::kKQ + 2 * (uint32_t)kSquare);
                wait_phase(&bar.u_ready, c & 1, gave_up);
                wait_phase(&bar.s_done, c & 1, gave_up);   // which has read the pair that was in this place
                tmem_fence_after();
#pragma unroll
                for (int t = 0; t < (NP == 1 ? 3 : 4); ++t)   // hi hi, lo hi, hi lo, and lo lo for f16 and f32 (delta_common.cuh says why)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_tmem(one, tm + kColO, tm + kColR + (t & 1 ? 32 : 0) + k * 8,
                                 further(pp, (t & 2 ? (uint32_t)kSquare : 0) + k * 32), shape(kChunk, true), t + k > 0);
                mma_commit(one, &bar.o_done);
                mma_commit(one, &bar.empty[st]);
            };
#pragma unroll 1
            for (int c = 0; c < chunks && !*gave_up; ++c) {
                const int st = c % M::kStages;
                const uint32_t at_stage = st * M::kStage;
                const uint64_t kq = further(kq0, at_stage), kt = further(kt0, at_stage), tt = further(kq, M::kKQ);
                if (M::kStages == 1 && c && !states) outputs(c - 1);
                wait_phase(&bar.full[st], (c / M::kStages) & 1, gave_up);
                if (c && !states) wait_phase(&bar.q_read, (c - 1) & 1, gave_up);
                // S^T [K^T Q^T], by the columns of S that are ready together
#pragma unroll
                for (int r = 0; r < KH; ++r) {
                    wait_busy(&bar.s_ready[r], c & 1, gave_up);
                    tmem_fence_after();
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int k = (i >> 1) * (KP / 32) + 2 * r + (i & 1);   // columns 16 k..
                                mma_tmem(one, tm + kColX, tm + (h ? kColSLo : kColSHi) + k * 8,
                                         further(kq, (p * KH + (k >> 2)) * kHalf + (k & 3) * 32), shape(2 * kChunk, true),
                                         r + p + h + i > 0);
                            }
                }
                mma_commit(one, &bar.x_done);
                if (M::kStages == 2 && c && !states) outputs(c - 1);
                wait_busy(&bar.r_ready, c & 1, gave_up);
                tmem_fence_after();
                // (beta R)^T (T - 1)^T: both parts of beta R with both of T - 1's
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_tmem(one, tm + kColU, tm + kColR + k * 8, further(tt, (k & 3) * 32), shape(2 * kChunk, true), k > 0);
                mma_commit(one, &bar.u_done);
                wait_busy(&bar.w_ready, c & 1, gave_up);
                tmem_fence_after();
                // S^T += (exp(G_C - G) U)^T K
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_tmem(one, tm + kColS, tm + kColW + h * 32 + k * 8,
                                     further(kt, p * KH * kHalf + k * 16 * 128), shape(KP, false), true);
                mma_commit(one, &bar.s_done);
                if (states) mma_commit(one, &bar.empty[st]);
            }
            if (chunks > 0 && !*gave_up && !states) outputs(chunks - 1);
            mma_commit(one, &bar.drained);
            wait_drained(&bar.drained, 0);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && keep) {   // what training keeps
            const int rows = min(kBlockV, (a.s.v - v0 + 15) / 16 * 16);
            for (int c = 0; c < chunks; ++c) {
                unsigned char *w = chunk_ws(c);
                wait_phase(&bar.s_kept, c & 1, gave_up);
#pragma unroll
                for (int p = 0; p < 2 * KH; ++p)
                    bulk_store(w + lay.s + (size_t)(vb * 2 * KH + p) * kHalf, base + M::kSave + p * kHalf, rows * 128);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(&bar.s_free);
                wait_phase(&bar.u_ready, c & 1, gave_up);
                unsigned char *u = w + lay.u + (size_t)vb * 2 * kHalf;
                if (M::kInStage) {
                    const uint32_t tiles = base + M::kTiles + c % M::kStages * M::kStage;
                    bulk_store(u, tiles + M::kKQ, rows * 128);
                    bulk_store(u + kHalf, tiles + kChunk * 128, min(rows, kChunk) * 128);
                    if (rows > kChunk) bulk_store(u + kHalf + kChunk * 128, tiles + kHalf + kChunk * 128, (rows - kChunk) * 128);
                } else {
                    for (int p = 0; p < 2; ++p) bulk_store(u + p * kHalf, base + M::kSaveU + p * kHalf, rows * 128);
                }
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(M::kInStage ? &bar.empty[c % M::kStages] : &bar.u_free);
            }
            bulk_wait();
        }
        __syncwarp();
    } else if (warp == 2) {
        if (lane == 0) {
            int c = 0;
            for (; c < chunks; ++c) {
                const int st = c % M::kStages;
                if (c >= M::kStages) wait_phase(&bar.empty[st], (c / M::kStages - 1) & 1, gave_up);
                if (*gave_up) break;
                unsigned char *w = chunk_ws(c), *to = smem + M::kTiles + st * M::kStage;
                mbar_arrive_expect_tx(&bar.full[st], M::kStage + 3 * kChunk * 4);
                bulk_load(to, a.kq + (size_t)((sp.slot + c) * a.s.hk + head / rep) * kq_stride(a.s.k, NP), M::kKQ, &bar.full[st]);
                bulk_load(to + M::kKQ, w + lay.t, M::kTP, &bar.full[st]);
                bulk_load(smem + M::kScal + st * 3 * kChunk * 4, w + lay.scal, 3 * kChunk * 4, &bar.full[st]);
            }
            for (int i = c < M::kStages ? 0 : c - M::kStages; i < c; ++i)   // copies in flight
                wait_drained(&bar.full[i % M::kStages], (i / M::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 3) {
        const int cols = min(kBlockV, a.s.v - v0);
        int c = 0;
        for (; c < chunks && !matrix; ++c) {
            const int n = (int)min((long long)kChunk, sp.len - (long long)c * kChunk);
            if (c) wait_phase(&bar.v_empty, (c - 1) & 1, gave_up);
            if (*gave_up) break;
            const T *src = row_ptr<T>(a.v, sp, seq, (long long)c * kChunk, head) + v0;
            unsigned char *dst = smem + M::kV;
            if (a.vec_v) {
                constexpr int PIECES = M::kVRow / 16;   // 16-byte pieces of a row
                const int piece = lane % PIECES;
                if (piece * 16 < cols * (int)sizeof(T))
                    for (int i = lane / PIECES; i < n; i += 32 / PIECES)
                        cp_async16(smem_addr(dst) + i * M::kVRow + piece * 16, reinterpret_cast<const char *>(src + i * a.v.tok) + piece * 16, true);
                mbar_arrive_after_copies(&bar.v_full);
            } else {
                for (int i = lane; i < n * kBlockV; i += 32)
                    if (i % kBlockV < cols) reinterpret_cast<T *>(dst)[i] = src[(i / kBlockV) * a.v.tok + i % kBlockV];
                mbar_arrive(&bar.v_full);
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
    } else if (warp >= kFirstConvert && warp < kFirstOut) {
        const int row = 32 * (warp & 3) + lane, half = (warp - kFirstConvert) >> 2, v = v0 + row;   // this thread's value, its half
        const uint32_t at = (uint32_t)(warp & 3) << 21;                                             // lane 32 (warp % 4)
        float x[2][16], y[2][16];
        uint32_t hi[8], lo[8];
        {   // the state at the start: all of its loads in flight at once
            float s[KP / 32][16];
            const float *row_from = from + (size_t)half * (KP / 2) * a.s.v + v;
            const int n = from && !matrix && v < a.s.v ? a.s.k - half * (KP / 2) : 0;
#pragma unroll
            for (int b = 0; b < KP / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[b][i] = matrix && half * (KP / 2) + 16 * b + i == v ? 1.f : 0.f;
                    if (16 * b + i < n) s[b][i] = row_from[(size_t)(16 * b + i) * a.s.v];
                }
#pragma unroll
            for (int b = 0; b < KP / 32; ++b) tmem_st16(at + kColS + half * (KP / 2) + 16 * b, s[b]);
        }
        tmem_wait_st();
        // this half's values of a chunk; rows past the sequence's end and values past V hold anything and count as 0
        auto fetch = [&](int c) {
            if (matrix) {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i >> 4][i & 15] = 0.f;
                return;
            }
            const T *vp = reinterpret_cast<const T *>(smem + M::kV) + 32 * half * kBlockV + row;
            const int n = v < a.s.v ? (int)min((long long)kChunk, sp.len - (long long)c * kChunk) - 32 * half : 0;
            wait_phase(&bar.v_full, c & 1, gave_up);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i >> 4][i & 15] = to_f32<T>(vp[i * kBlockV]);
            if (n < 32)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i >= n) y[i >> 4][i & 15] = 0.f;
            warp_arrive(&bar.v_empty, lane);
        };
        if (chunks > 0) fetch(0);
        for (int c = 0; c < chunks; ++c) {
            const int st = c % M::kStages;
            const float *scal = reinterpret_cast<const float *>(smem + M::kScal + st * 3 * kChunk * 4) + 32 * half;
            wait_phase(&bar.full[st], (c / M::kStages) & 1, gave_up);
            const float eall = scal[kChunk - 1 - 32 * half];
            if (c > 0) {
                if (keep) wait_phase(&bar.s_free, (c - 1) & 1, gave_up);
                wait_phase(&bar.s_done, (c - 1) & 1, gave_up);
                tmem_fence_after();
            }
#pragma unroll 1
            for (int r = 0; r < KH; ++r) {
                const int k16 = half * (KP / 32) + 2 * r;
                tmem_ld16(x[0], at + kColS + 16 * k16, x[1], at + kColS + 16 * k16 + 16);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    split16(x[b], hi, lo);   // what X reads; the state itself goes on in f32
                    tmem_st8(at + kColSHi + 8 * (k16 + b), hi);
                    tmem_st8(at + kColSLo + 8 * (k16 + b), lo);
                    scale16(x[b], eall);
                    tmem_st16(at + kColS + 16 * (k16 + b), x[b]);
                    if (keep) keep16(base + M::kSave, KH * kHalf, row, k16 + b, hi, lo);
                }
                tmem_wait_st();
                tmem_fence_before();
                warp_arrive(&bar.s_ready[r], lane);
            }
            if (keep) {
                fence_async();
                warp_arrive(&bar.s_kept, lane);
            }

            wait_phase(&bar.x_done, c & 1, gave_up);
            tmem_fence_after();
            tmem_ld16(x[0], at + kColX + 32 * half, x[1], at + kColX + 32 * half + 16);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {   // beta R = beta (V - exp(G) X)
                    const float4 eg = *reinterpret_cast<const float4 *>(scal + 16 * b + i);
                    const float4 be = *reinterpret_cast<const float4 *>(scal + 128 + 16 * b + i);
                    const float2 r0 = fma2(make_float2(-eg.x, -eg.y), make_float2(x[b][i], x[b][i + 1]), make_float2(y[b][i], y[b][i + 1]));
                    const float2 r1 = fma2(make_float2(-eg.z, -eg.w), make_float2(x[b][i + 2], x[b][i + 3]), make_float2(y[b][i + 2], y[b][i + 3]));
                    const float2 y0 = mul2(make_float2(be.x, be.y), r0), y1 = mul2(make_float2(be.z, be.w), r1);
                    x[b][i] = y0.x; x[b][i + 1] = y0.y; x[b][i + 2] = y1.x; x[b][i + 3] = y1.y;
                }
            if (c > 0 && !states) wait_phase(&bar.o_done, (c - 1) & 1, gave_up);   // the last chunk's U was there
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                split16(x[b], hi, lo);   // for (T - 1) beta R alone: U adds beta R in f32
                tmem_st8(at + kColR + 16 * half + 8 * b, hi);
                tmem_st8(at + kColR + 32 + 16 * half + 8 * b, lo);
            }
            tmem_wait_st();
            tmem_fence_before();
            warp_arrive(&bar.r_ready, lane);
            if (c + 1 < chunks) fetch(c + 1);

            if (c > 0 && !states) wait_phase(&bar.o_read, (c - 1) & 1, gave_up);   // the last outputs were where the next pair goes
            wait_phase(&bar.u_done, c & 1, gave_up);
            tmem_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {   // U = beta R + (T - 1) beta R: only the second part goes through pairs
                float z[16], w[16];
                tmem_ld16(z, at + kColU + 32 * half + 16 * b, w, at + kColU + kChunk + 32 * half + 16 * b);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 t = fma2(make_float2(1.f, 1.f), make_float2(z[i], z[i + 1]), make_float2(w[i], w[i + 1]));
                    const float2 u = fma2(make_float2(1.f, 1.f), make_float2(x[b][i], x[b][i + 1]), t);
                    z[i] = x[b][i] = u.x;
                    z[i + 1] = x[b][i + 1] = u.y;
                }
                scale16(z, scal + 64 + 16 * b);
                split16(z, hi, lo);   // where a state's error comes from: 2^-18.4 of each term that a token adds
                tmem_st8(at + kColW + 16 * half + 8 * b, hi);
                tmem_st8(at + kColW + 32 + 16 * half + 8 * b, lo);
            }
            tmem_wait_st();
            tmem_fence_before();
            warp_arrive(&bar.w_ready, lane);
            if (states) continue;
            if (keep && !M::kInStage && c > 0) wait_phase(&bar.u_free, (c - 1) & 1, gave_up);
            // U's upper part where T was, the lower one where the queries were: row 64 in the second half
            const uint32_t tiles = base + M::kTiles + st * M::kStage;
            const uint32_t u_hi = M::kInStage ? tiles + M::kKQ : base + M::kSaveU;
            const uint32_t u_lo = M::kInStage ? tiles + (row < kChunk ? kChunk * 128 : kHalf) : base + M::kSaveU + kHalf;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                split16(x[b], hi, lo);
                tmem_st8(at + kColR + 16 * half + 8 * b, hi);
                tmem_st8(at + kColR + 32 + 16 * half + 8 * b, lo);
                if (keep) keep16(u_hi, u_lo - u_hi, row, 2 * half + b, hi, lo);
            }
            if (keep) fence_async();
            tmem_wait_st();
            tmem_fence_before();
            warp_arrive(&bar.u_ready, lane);
        }
        if (to_state || matrix) {   // the state at the end
            if (chunks > 0) wait_phase(&bar.s_done, (chunks - 1) & 1, gave_up);
            tmem_fence_after();
            unsigned char *m = a.seg_m + (size_t)(chain.slot * a.s.hv + head) * seg_m_bytes(a.s.k);
#pragma unroll 1
            for (int b = 0; b < KP / 32; ++b) {
                const int k0 = half * (KP / 2) + 16 * b;
                tmem_ld16(x[0], at + kColS + k0);
                if (*gave_up)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[0][i] = __int_as_float(0x7fffffff);
                if (matrix) {
                    split16(x[0], hi, lo);   // as the join's products read it
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint32_t to = img(0, row, k0 / 8 + p);
                        *reinterpret_cast<uint4 *>(m + to) = make_uint4(hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
                        *reinterpret_cast<uint4 *>(m + KH * kHalf + to) = make_uint4(lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (k0 + i < a.s.k && v < a.s.v) to_state[(size_t)(k0 + i) * a.s.v + v] = x[0][i];
                }
            }
        }
    } else if (warp >= kFirstOut) {
        const int row = 32 * (warp & 3) + lane;   // this thread's value
        const uint32_t at = (uint32_t)(warp & 3) << 21;
        const size_t ostride = (size_t)a.s.hv * a.s.v;
        const bool rows_out = (a.s.v * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.o) & 15) == 0;
        for (int c = 0; c < chunks && !states; ++c) {
            const int st = c % M::kStages;
            const float *scal = reinterpret_cast<const float *>(smem + M::kScal + st * 3 * kChunk * 4);
            const int n = (int)min((long long)kChunk, sp.len - (long long)c * kChunk);
            T *out = static_cast<T *>(a.o) + ((size_t)(sp.first + (long long)c * kChunk) * a.s.hv + head) * a.s.v + v0;
            float x[4][16];   // scale exp(G) S^T Q^T
            wait_phase(&bar.full[st], (c / M::kStages) & 1, gave_up);
            wait_phase(&bar.x_done, c & 1, gave_up);
            tmem_fence_after();
            tmem_ld16(x[0], at + kColQ, x[1], at + kColQ + 16);
            tmem_ld16(x[2], at + kColQ + 32, x[3], at + kColQ + 48);
            tmem_fence_before();
            warp_arrive(&bar.q_read, lane);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                scale16(x[b], scal + 16 * b);
                scale16(x[b], a.s.scale);
            }
            wait_phase(&bar.o_done, c & 1, gave_up);
            tmem_fence_after();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float y[16];
                tmem_ld16(y, at + kColO + 16 * b);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 o = fma2(make_float2(1.f, 1.f), make_float2(x[b][i], x[b][i + 1]), make_float2(y[i], y[i + 1]));
                    x[b][i] = o.x;
                    x[b][i + 1] = o.y;
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar.o_read);
                mbar_arrive(&bar.empty[st]);
            }
            if (rows_out) {   // by way of shared memory, to store whole rows
                T *stage = reinterpret_cast<T *>(smem + M::kOut);
                asm volatile("bar.sync 1, 128;" ::: "memory");   // the last chunk's rows have been read
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) stage[(16 * b + i) * kBlockV + row] = from_f32<T>(x[b][i]);
                asm volatile("bar.sync 1, 128;" ::: "memory");
                constexpr int PIECES = M::kVRow / 16;
                const int piece = row % PIECES;
                if (piece * 16 < (a.s.v - v0) * (int)sizeof(T))
#pragma unroll 2
                    for (int i = row / PIECES; i < n; i += 128 / PIECES)
                        *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(out + i * ostride) + piece * 16) =
                            *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(stage) + i * M::kVRow + piece * 16);
            } else if (v0 + row < a.s.v) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * b + i < n) out[(16 * b + i) * ostride + row] = from_f32<T>(x[b][i]);
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (*gave_up && a.failed && threadIdx.x == 0) *a.failed = 1;
    if (*gave_up && !states && v0 + (int)threadIdx.x < a.s.v && threadIdx.x < kBlockV)   // the outputs are not what they should be: say so
        for (long long t = 0; t < sp.len; ++t)
            static_cast<T *>(a.o)[((size_t)(sp.first + t) * a.s.hv + head) * a.s.v + v0 + threadIdx.x] =
                from_f32<T>(__int_as_float(0x7fffffff));
    tmem_fence_after();
    if (warp == 0) tmem_free(bar.tmem);
}

namespace {

template <typename T, int KP>
cudaError_t chain(const DeltaArgs &a, cudaStream_t s) {
    using M = ChainSmem<T, KP>;
    const bool states = a.pass == kPassStates;
    const int bytes = a.train && !states ? M::kTrainBytes : M::kBytes;
    cudaError_t e = cudaFuncSetAttribute(delta_chain_kernel<T, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kTrainBytes);
    if (e != cudaSuccess) return e;
    const long long ctas = (a.seg ? a.seg_slots : a.s.seqs) * a.s.hv * (blocks_v(a.s.v) + states);
    delta_chain_kernel<T, KP><<<(unsigned)ctas, kChainThreads, bytes, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t chain_for(const DeltaArgs &a, cudaStream_t s) {
    return a.s.k <= 64 ? chain<T, 64>(a, s) : chain<T, 128>(a, s);
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaArgs &a, int type, cudaStream_t s) {
    switch (type) {
    case PS_REAL_BF16: return chain_for<__nv_bfloat16>(a, s);
    case PS_REAL_F16: return chain_for<__half>(a, s);
    default: return chain_for<float>(a, s);
    }
}

}  // namespace ps
