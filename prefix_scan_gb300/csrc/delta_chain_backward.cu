// delta_chain_backward.cu -- the gradients of the gated delta rule's states,
// chunk before chunk, and of its values (notation in delta_common.cuh).  With
// dS' the gradient of the state at a chunk's end, each chunk takes
//     Y  = diag(exp(G_C - G)) K dS' + P^T dO             (the gradient of U)
//     dU = T^T Y,   dR = diag(beta) dU = dV
//     dS = exp(G_C) dS' + scale (exp(G) Q)^T dO - (exp(G) K)^T dR
// and leaves dS' and dU for the gradients of the other inputs
// (delta_gradients.cu).
//
// Laid out as the forward chain (delta_chain.cu): everything transposed, values
// are the 128 rows of the accumulators, left operands go through registers back
// into tensor memory, right operands are the images in shared memory.  P^T dO
// runs while dS' is on its way through registers, scale (exp(G) Q)^T dO while Y
// is; dO becomes a left operand while the state's product runs.  Segments and their
// two passes are as there, and so is what bounds it: 4 x 4096 tokens, 16 heads of
// 128 x 128, take 246 us; 16384 tokens of 8 heads two passes of 59.
#include "delta_tmem.cuh"

namespace ps {

namespace {

constexpr int kBackThreads = 16 * 32, kFirstConvert = 4, kFirstOut = 12;   // warps
// Tensor-memory columns: dS; its pair, later dU's two accumulators; dO, later K dS'; P^T dO; the
// pair of Y, later of -exp(G) dR; the pair of scale exp(G) dO.  (All 512: K dS' waits until P^T dO has read dO.)
constexpr uint32_t kColS = 0, kColSHi = 128, kColSLo = 192, kColU = 128, kColY = 256, kColO = 256, kColP = 320;
constexpr uint32_t kColR = 384, kColQ = 448;

template <typename T, int KP>
struct BackSmem {
    static constexpr int NP = Planes<T>::NP;
    static constexpr int kKQ = NP * (KP / 64) * kHalf, kTP = 4 * (int)kSquare;
    static constexpr int kStages = NP == 1 || (KP == 64 && sizeof(T) == 2) ? 2 : 1;   // as many as there is room for
    static constexpr int kScal = 256, kTiles = 2048, kStage = kKQ + kTP;   // barriers and two chunks' scalars come first
    static constexpr int kRow = kBlockV * (int)sizeof(T), kTile = kChunk * kRow;
    static constexpr int kDO = kTiles + kStages * kStage, kOut = kDO + kTile, kSave = kOut + kTile;
    // dS' on its way out, and dU, which at K = 128 takes the place of T and of the queries (both used by
    // then) in its stage
    static constexpr int kSaveU = kSave + 2 * (KP / 64) * kHalf;
    static constexpr bool kInStage = KP == 128;
    static constexpr int kBytes = kSaveU + (kInStage ? 0 : 2 * kHalf);
};
struct BackBars {
    uint64_t full[2], empty[2], o_full, o_empty, o_ready, p_done, s_ready[2], y_done, r_ready, u_done, w_ready, s_done, out_ready, out_free;
    uint64_t s_kept, s_free, u_free, drained;
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(BackBars) <= 256, "barriers precede the scalars");

}  // namespace

template <typename T, int KP>
__global__ void __launch_bounds__(kBackThreads, 1) delta_chain_backward_kernel(const DeltaArgs a) {
    using M = BackSmem<T, KP>;
    constexpr int NP = M::NP, KH = KP / 64;
    extern __shared__ __align__(1024) unsigned char smem[];
    BackBars &bar = *reinterpret_cast<BackBars *>(smem);
    volatile int *gave_up = &bar.gave_up;
    const uint32_t base = smem_addr(smem);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // known to be uniform
    const bool states = a.pass == kPassStates;   // of segments, without the gradients of values
    const int blocks = blocks_v(a.s.v), rep = a.s.hv / a.s.hk;
    const int vb = (int)(blockIdx.x % blocks);
    const int head = (int)(blockIdx.x / blocks % a.s.hv);
    Chain chain;
    if (!chain_of(a, blockIdx.x / blocks / a.s.hv, chain)) return;
    if (states && chain.first) return;   // nobody needs it
    const long long seq = chain.seq;
    const Span sp = chain.span;
    const int v0 = vb * kBlockV;
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, true);
    const int chunks = (int)((sp.len + kChunk - 1) / kChunk);
    // the gradient at the end and where it goes at the start
    const size_t one_state = (size_t)a.s.k * a.s.v;
    const float *from = chain.last ? (a.dht ? a.dht + (size_t)(seq * a.s.hv + head) * one_state : nullptr)
                        : states  ? nullptr
                                  : a.seg_state + (size_t)((chain.slot + 1) * a.s.hv + head) * one_state;
    float *to_state = states ? a.seg_state + (size_t)(chain.slot * a.s.hv + head) * one_state
                      : chain.first && a.dh0 ? a.dh0 + (size_t)(seq * a.s.hv + head) * one_state
                                             : nullptr;
    // chunks are taken last to first: i counts them as they come
    auto chunk_ws = [&](int i) { return a.ws + (size_t)((sp.slot + chunks - 1 - i) * a.s.hv + head) * lay.stride; };
    auto first_token = [&](int i) { return (long long)(chunks - 1 - i) * kChunk; };
    auto rows_of = [&](int i) { return (int)min((long long)kChunk, sp.len - first_token(i)); };

    if (threadIdx.x == 0) {
        const int failed = a.failed ? *a.failed : 0;   // what the forward chains kept is not to be used
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1 + (!states && (M::kInStage || M::kStages == 2)));
            mbar_init(&bar.s_ready[i], 8);
        }
        mbar_init(&bar.o_full, 32);
        mbar_init(&bar.o_empty, 8);
        mbar_init(&bar.o_ready, 8);
        mbar_init(&bar.p_done, 1);
        mbar_init(&bar.y_done, 1);
        mbar_init(&bar.r_ready, 8);
        mbar_init(&bar.u_done, 1);
        mbar_init(&bar.w_ready, 8);
        mbar_init(&bar.s_done, 1);
        mbar_init(&bar.out_ready, 8);
        mbar_init(&bar.out_free, 4);
        mbar_init(&bar.s_kept, 8);
        mbar_init(&bar.s_free, 1);
        mbar_init(&bar.u_free, 1);
        mbar_init(&bar.drained, 1);
        bar.gave_up = failed || base & 1023 ? 1 : 0;   // images need their alignment
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
        // operands: keys by rows; keys, queries, T (both of its parts side by side) and P by columns
        const uint64_t kq0 = operand(base + M::kTiles, true, 0), kt0 = operand(base + M::kTiles, false, kHalf);
        const uint64_t tt0 = operand(base + M::kTiles + M::kKQ, false, (uint32_t)kSquare);
#pragma unroll 1
        for (int i = 0; i < chunks && !*gave_up; ++i) {
            const int st = i % M::kStages;
            const uint32_t at_stage = st * M::kStage;
            const uint64_t kq = further(kq0, at_stage), kt = further(kt0, at_stage), tt = further(tt0, at_stage);
            wait_phase(&bar.full[st], (i / M::kStages) & 1, gave_up);
            wait_phase(&bar.o_ready, i & 1, gave_up);
            tmem_fence_after();
            // dO^T P
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int p = 0; p < NP; ++p)   // P's parts, dO's parts
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_tmem(one, tm + kColP, tm + kColO + p * 32 + k * 8,
                                 further(tt, (2 + t) * (uint32_t)kSquare + k * 16 * 128), shape(kChunk, false), t + p + k > 0);
            mma_commit(one, &bar.p_done);
            // dS'^T K^T, by the columns of dS' that are ready together
#pragma unroll
            for (int r = 0; r < KH; ++r) {
                wait_busy(&bar.s_ready[r], i & 1, gave_up);
                if (r == 0) wait_busy(&bar.p_done, i & 1, gave_up);   // dO has been read: K dS' takes its place
                tmem_fence_after();
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = (j >> 1) * (KP / 32) + 2 * r + (j & 1);   // columns 16 k..
                            mma_tmem(one, tm + kColY, tm + (h ? kColSLo : kColSHi) + k * 8,
                                     further(kq, (p * KH + (k >> 2)) * kHalf + (k & 3) * 32), shape(kChunk, true), r + p + h + j > 0);
                        }
            }
            mma_commit(one, &bar.y_done);
            // dS^T += scale (exp(G) dO)^T Q
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_tmem(one, tm + kColS, tm + kColQ + h * 32 + k * 8,
                                 further(kt, p * KH * kHalf + kChunk * 128 + k * 16 * 128), shape(KP, false), true);
            wait_busy(&bar.r_ready, i & 1, gave_up);
            tmem_fence_after();
            // Y^T (T - 1)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_tmem(one, tm + kColU, tm + kColR + k * 8, further(tt, (k & 3) * 16 * 128), shape(2 * kChunk, false), k > 0);
            mma_commit(one, &bar.u_done);
            wait_busy(&bar.w_ready, i & 1, gave_up);
            tmem_fence_after();
            // dS^T -= (exp(G) dR)^T K
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_tmem(one, tm + kColS, tm + kColR + h * 32 + k * 8,
                                 further(kt, p * KH * kHalf + k * 16 * 128), shape(KP, false), true);
            mma_commit(one, &bar.s_done);
            mma_commit(one, &bar.empty[st]);
        }
        mma_commit(one, &bar.drained);
        wait_drained(&bar.drained, 0);
    } else if (warp == 1) {
        if (lane == 0 && !states) {   // dS' and dU for the gradients
            const int rows = min(kBlockV, (a.s.v - v0 + 15) / 16 * 16);
            for (int i = 0; i < chunks; ++i) {
                unsigned char *w = chunk_ws(i);
                wait_phase(&bar.s_kept, i & 1, gave_up);
#pragma unroll
                for (int p = 0; p < 2 * KH; ++p)
                    bulk_store(w + lay.ds + (size_t)(vb * 2 * KH + p) * kHalf, base + M::kSave + p * kHalf, rows * 128);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(&bar.s_free);
                wait_phase(&bar.out_ready, i & 1, gave_up);
                // dV has taken its gates: with two stages the next but one chunk's scalars come in their place
                if (M::kStages == 2 && !M::kInStage) mbar_arrive(&bar.empty[i % M::kStages]);
                unsigned char *u = w + lay.du + (size_t)vb * 2 * kHalf;
                if (M::kInStage) {
                    const uint32_t tiles = base + M::kTiles + i % M::kStages * M::kStage;
                    bulk_store(u, tiles + M::kKQ, rows * 128);
                    bulk_store(u + kHalf, tiles + kChunk * 128, min(rows, kChunk) * 128);
                    if (rows > kChunk) bulk_store(u + kHalf + kChunk * 128, tiles + kHalf + kChunk * 128, (rows - kChunk) * 128);
                } else {
                    for (int p = 0; p < 2; ++p) bulk_store(u + p * kHalf, base + M::kSaveU + p * kHalf, rows * 128);
                }
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(M::kInStage ? &bar.empty[i % M::kStages] : &bar.u_free);
            }
            bulk_wait();
        }
        __syncwarp();
    } else if (warp == 2) {
        if (lane == 0) {
            int i = 0;
            for (; i < chunks; ++i) {
                const int st = i % M::kStages;
                if (i >= M::kStages) wait_phase(&bar.empty[st], (i / M::kStages - 1) & 1, gave_up);
                if (*gave_up) break;
                unsigned char *w = chunk_ws(i), *to = smem + M::kTiles + st * M::kStage;
                mbar_arrive_expect_tx(&bar.full[st], M::kStage + 3 * kChunk * 4);
                bulk_load(to, a.kq + (size_t)((sp.slot + chunks - 1 - i) * a.s.hk + head / rep) * kq_stride(a.s.k, NP), M::kKQ, &bar.full[st]);
                bulk_load(to + M::kKQ, w + lay.t, M::kTP, &bar.full[st]);
                bulk_load(smem + M::kScal + (i & 1) * 3 * kChunk * 4, w + lay.scal, 3 * kChunk * 4, &bar.full[st]);
            }
            for (int j = i < M::kStages ? 0 : i - M::kStages; j < i; ++j)   // copies in flight
                wait_drained(&bar.full[j % M::kStages], (j / M::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 3) {
        const int cols = min(kBlockV, a.s.v - v0);
        for (int i = 0; i < chunks; ++i) {
            const int n = rows_of(i);
            if (i) wait_phase(&bar.o_empty, (i - 1) & 1, gave_up);
            if (*gave_up) break;
            const T *src = row_ptr<T>(a.dout, sp, seq, first_token(i), head) + v0;
            unsigned char *dst = smem + M::kDO;
            if (a.vec_do) {
                constexpr int PIECES = M::kRow / 16;   // 16-byte pieces of a row
                const int piece = lane % PIECES;
                if (piece * 16 < cols * (int)sizeof(T))
                    for (int r = lane / PIECES; r < n; r += 32 / PIECES)
                        cp_async16(smem_addr(dst) + r * M::kRow + piece * 16, reinterpret_cast<const char *>(src + r * a.dout.tok) + piece * 16, true);
                mbar_arrive_after_copies(&bar.o_full);
            } else {
                for (int r = lane; r < n * kBlockV; r += 32)
                    if (r % kBlockV < cols) reinterpret_cast<T *>(dst)[r] = src[(r / kBlockV) * a.dout.tok + r % kBlockV];
                mbar_arrive(&bar.o_full);
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
    } else if (warp < kFirstOut) {
        const int row = 32 * (warp & 3) + lane, half = (warp - kFirstConvert) >> 2, v = v0 + row;   // this thread's value, its half
        const uint32_t at = (uint32_t)(warp & 3) << 21;                                             // lane 32 (warp % 4)
        float x[2][16];
        uint32_t hi[8], lo[8];
        {   // the gradient at the end: all of its loads in flight at once
            float s[KP / 32][16];
            const float *row_from = from + (size_t)half * (KP / 2) * a.s.v + v;
            const int n = from && v < a.s.v ? a.s.k - half * (KP / 2) : 0;
#pragma unroll
            for (int b = 0; b < KP / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[b][i] = 0.f;
                    if (16 * b + i < n) s[b][i] = row_from[(size_t)(16 * b + i) * a.s.v];
                }
#pragma unroll
            for (int b = 0; b < KP / 32; ++b) tmem_st16(at + kColS + half * (KP / 2) + 16 * b, s[b]);
        }
        tmem_wait_st();
        auto scalars = [&](int i) { return reinterpret_cast<const float *>(smem + M::kScal + (i & 1) * 3 * kChunk * 4) + 32 * half; };
        // dO and scale exp(G) dO of a chunk as left operands; rows past the sequence's end and values past V hold
        // anything and count as 0
        auto outputs = [&](int i) {
            const T *op = reinterpret_cast<const T *>(smem + M::kDO) + 32 * half * kBlockV + row;
            const int n = v < a.s.v ? rows_of(i) - 32 * half : 0;
            wait_phase(&bar.o_full, i & 1, gave_up);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j >> 4][j & 15] = to_f32<T>(op[j * kBlockV]);
            if (n < 32)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j >= n) x[j >> 4][j & 15] = 0.f;
            warp_arrive(&bar.o_empty, lane);
            wait_phase(&bar.full[i % M::kStages], (i / M::kStages) & 1, gave_up);
            const float *scal = scalars(i);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                split16(x[b], hi, lo);
                tmem_st8(at + kColO + 16 * half + 8 * b, hi);
                if constexpr (NP == 2) tmem_st8(at + kColO + 32 + 16 * half + 8 * b, lo);
                scale16(x[b], scal + 16 * b);
                scale16(x[b], a.s.scale);
                split16(x[b], hi, lo);
                tmem_st8(at + kColQ + 16 * half + 8 * b, hi);
                tmem_st8(at + kColQ + 32 + 16 * half + 8 * b, lo);
            }
            tmem_wait_st();
            tmem_fence_before();
            warp_arrive(&bar.o_ready, lane);
        };
        if (chunks > 0) outputs(0);
        for (int i = 0; i < chunks; ++i) {
            const float *scal = scalars(i);
            const float eall = scal[kChunk - 1 - 32 * half];
            if (i > 0) {
                if (!states) wait_phase(&bar.s_free, (i - 1) & 1, gave_up);
                wait_phase(&bar.s_done, (i - 1) & 1, gave_up);
                tmem_fence_after();
            }
#pragma unroll 1
            for (int r = 0; r < KH; ++r) {
                const int k16 = half * (KP / 32) + 2 * r;
                tmem_ld16(x[0], at + kColS + 16 * k16, x[1], at + kColS + 16 * k16 + 16);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    split16(x[b], hi, lo);
                    tmem_st8(at + kColSHi + 8 * (k16 + b), hi);
                    tmem_st8(at + kColSLo + 8 * (k16 + b), lo);
                    scale16(x[b], eall);
                    tmem_st16(at + kColS + 16 * (k16 + b), x[b]);
                    if (!states) keep16(base + M::kSave, KH * kHalf, row, k16 + b, hi, lo);
                }
                tmem_wait_st();
                tmem_fence_before();
                warp_arrive(&bar.s_ready[r], lane);
            }
            if (!states) {
                fence_async();
                warp_arrive(&bar.s_kept, lane);
            }

            wait_phase(&bar.y_done, i & 1, gave_up);
            tmem_fence_after();
            {
                float z[2][16];
                tmem_ld16(x[0], at + kColY + 32 * half, z[0], at + kColP + 32 * half);
                tmem_ld16(x[1], at + kColY + 32 * half + 16, z[1], at + kColP + 32 * half + 16);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 el = *reinterpret_cast<const float4 *>(scal + 64 + 16 * b + j);
                        const float2 y0 = fma2(make_float2(el.x, el.y), make_float2(x[b][j], x[b][j + 1]), make_float2(z[b][j], z[b][j + 1]));
                        const float2 y1 = fma2(make_float2(el.z, el.w), make_float2(x[b][j + 2], x[b][j + 3]), make_float2(z[b][j + 2], z[b][j + 3]));
                        x[b][j] = y0.x; x[b][j + 1] = y0.y; x[b][j + 2] = y1.x; x[b][j + 3] = y1.y;
                    }
                    split16(x[b], hi, lo);
                    tmem_st8(at + kColR + 16 * half + 8 * b, hi);
                    tmem_st8(at + kColR + 32 + 16 * half + 8 * b, lo);
                }
            }
            tmem_wait_st();
            tmem_fence_before();
            warp_arrive(&bar.r_ready, lane);

            wait_phase(&bar.u_done, i & 1, gave_up);
            tmem_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {   // dU = Y + (T - 1)^T Y, and -exp(G) beta dU
                float z[16], w[16];
                tmem_ld16(z, at + kColU + 32 * half + 16 * b, w, at + kColU + kChunk + 32 * half + 16 * b);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 eg = *reinterpret_cast<const float4 *>(scal + 16 * b + j);
                    const float4 be = *reinterpret_cast<const float4 *>(scal + 128 + 16 * b + j);
                    const float2 t0 = fma2(make_float2(1.f, 1.f), make_float2(z[j], z[j + 1]), make_float2(w[j], w[j + 1]));
                    const float2 t1 = fma2(make_float2(1.f, 1.f), make_float2(z[j + 2], z[j + 3]), make_float2(w[j + 2], w[j + 3]));
                    const float2 u0 = fma2(make_float2(1.f, 1.f), make_float2(x[b][j], x[b][j + 1]), t0);
                    const float2 u1 = fma2(make_float2(1.f, 1.f), make_float2(x[b][j + 2], x[b][j + 3]), t1);
                    const float2 g0 = mul2(mul2(make_float2(-eg.x, -eg.y), make_float2(be.x, be.y)), u0);
                    const float2 g1 = mul2(mul2(make_float2(-eg.z, -eg.w), make_float2(be.z, be.w)), u1);
                    x[b][j] = u0.x; x[b][j + 1] = u0.y; x[b][j + 2] = u1.x; x[b][j + 3] = u1.y;
                    z[j] = g0.x; z[j + 1] = g0.y; z[j + 2] = g1.x; z[j + 3] = g1.y;
                }
                split16(z, hi, lo);
                tmem_st8(at + kColR + 16 * half + 8 * b, hi);
                tmem_st8(at + kColR + 32 + 16 * half + 8 * b, lo);
            }
            tmem_wait_st();
            tmem_fence_before();
            warp_arrive(&bar.w_ready, lane);
            // dU, and dV = beta dU by rows
            if (states) {
                if (i + 1 < chunks) outputs(i + 1);
                continue;
            }
            if (!M::kInStage && i > 0) wait_phase(&bar.u_free, (i - 1) & 1, gave_up);
            // dU's upper part where T was, the lower one where the queries were: row 64 in the second half
            const uint32_t tiles = base + M::kTiles + i % M::kStages * M::kStage;
            const uint32_t u_hi = M::kInStage ? tiles + M::kKQ : base + M::kSaveU;
            const uint32_t u_lo = M::kInStage ? tiles + (row < kChunk ? kChunk * 128 : kHalf) : base + M::kSaveU + kHalf;
            if (i > 0) wait_phase(&bar.out_free, (i - 1) & 1, gave_up);
            T *stage = reinterpret_cast<T *>(smem + M::kOut) + 32 * half * kBlockV + row;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                split16(x[b], hi, lo);
                keep16(u_hi, u_lo - u_hi, row, 2 * half + b, hi, lo);
                scale16(x[b], scal + 128 + 16 * b);
#pragma unroll
                for (int j = 0; j < 16; ++j) stage[(16 * b + j) * kBlockV] = from_f32<T>(x[b][j]);
            }
            fence_async();
            warp_arrive(&bar.out_ready, lane);
            if (i + 1 < chunks) outputs(i + 1);
        }
        if (to_state) {
            if (chunks > 0) wait_phase(&bar.s_done, (chunks - 1) & 1, gave_up);
            tmem_fence_after();
#pragma unroll 1
            for (int b = 0; b < KP / 32; ++b) {
                const int k0 = half * (KP / 2) + 16 * b;
                tmem_ld16(x[0], at + kColS + k0);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + i < a.s.k && v < a.s.v)
                        to_state[(size_t)(k0 + i) * a.s.v + v] = *gave_up ? __int_as_float(0x7fffffff) : x[0][i];
            }
        }
    } else {
        const int tid = threadIdx.x - 32 * kFirstOut;
        const size_t ostride = (size_t)a.s.hv * a.s.v;
        const int cols = min(kBlockV, a.s.v - v0);
        const bool rows_out = (a.s.v * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.dv) & 15) == 0;
        for (int i = 0; i < chunks && !states; ++i) {
            const int n = rows_of(i);
            T *out = static_cast<T *>(a.dv) + ((size_t)(sp.first + first_token(i)) * a.s.hv + head) * a.s.v + v0;
            const T *stage = reinterpret_cast<const T *>(smem + M::kOut);
            wait_phase(&bar.out_ready, i & 1, gave_up);
            if (rows_out) {
                constexpr int PIECES = M::kRow / 16;
                const int piece = tid % PIECES;
                if (piece * 16 < cols * (int)sizeof(T))
#pragma unroll 4
                    for (int r = tid / PIECES; r < n; r += 128 / PIECES)
                        *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(out + r * ostride) + piece * 16) =
                            *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(stage) + r * M::kRow + piece * 16);
            } else if (tid < cols) {
                for (int r = 0; r < n; ++r) out[r * ostride + tid] = stage[r * kBlockV + tid];
            }
            warp_arrive(&bar.out_free, lane);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (*gave_up && a.failed && threadIdx.x == 0) *a.failed = 1;
    if (*gave_up && !states && v0 + (int)threadIdx.x < a.s.v && threadIdx.x < kBlockV)   // the gradients are not what they should be: say so
        for (long long t = 0; t < sp.len; ++t)
            static_cast<T *>(a.dv)[((size_t)(sp.first + t) * a.s.hv + head) * a.s.v + v0 + threadIdx.x] =
                from_f32<T>(__int_as_float(0x7fffffff));
    tmem_fence_after();
    if (warp == 0) tmem_free(bar.tmem);
}

namespace {

template <typename T, int KP>
cudaError_t chain_back(const DeltaArgs &a, cudaStream_t s) {
    constexpr int bytes = BackSmem<T, KP>::kBytes;
    static_assert(bytes <= 227 * 1024, "too much shared memory");
    cudaError_t e = cudaFuncSetAttribute(delta_chain_backward_kernel<T, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long long ctas = (a.seg ? a.seg_slots : a.s.seqs) * a.s.hv * blocks_v(a.s.v);
    delta_chain_backward_kernel<T, KP><<<(unsigned)ctas, kBackThreads, bytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain_backward(const DeltaArgs &a, int type, cudaStream_t s) {
    const bool small = a.s.k <= 64;
    switch (type) {
    case PS_REAL_BF16: return small ? chain_back<__nv_bfloat16, 64>(a, s) : chain_back<__nv_bfloat16, 128>(a, s);
    case PS_REAL_F16: return small ? chain_back<__half, 64>(a, s) : chain_back<__half, 128>(a, s);
    default: return small ? chain_back<float, 64>(a, s) : chain_back<float, 128>(a, s);
    }
}

}  // namespace ps
