// delta_gradients.cu -- the gradients of the gated delta rule's queries, keys,
// gates and log decays, all chunks at once, from what the two chains left
// (notation in delta_common.cuh and delta_chain_backward.cu).  Per chunk and
// value head, with dP = dO U^T and dN = -dR U^T (j < i only), dR = diag(beta) dU:
//     dQ = scale diag(exp(G)) dO S^T + (scale D dP) K
//     dK = (scale D dP)^T Q + (D dN) K + (D dN)^T K - diag(exp(G)) dR S^T + diag(exp(G_C - G)) U dS'^T
//     dbeta_j = (dU_j . U_j) / beta_j          (U = beta (what was missing))
//     dg_t = sum_{j < t <= i} Z_ij + sum_{i >= t} a_i + sum_{j < t} b_j + exp(G_C) <S, dS'>
// where Z = P dP + N dN (element by element), a_i = exp(G_i) (scale q_i . S dO_i -
// k_i . S dR_i) and b_j = exp(G_C - G_j) k_j . dS' U_j: every term that the decay of
// token t scales, each counted once, so nothing cancels.
//
// One CTA takes a chunk and key head at a time, and goes on to another: gradients of a
// shared key head are sums over its value heads in their order, without atomics.
// The products run on tensor memory with both operands in shared memory, as the images
// lie there, transposed so that keys' columns are the 128 rows:
//     X1 = S dO^T, X2 = S dU^T, X3 = dS' U^T           (columns: tokens)
// and, U's two parts one above the other as 128 rows, U dO^T and U dU^T.  One warp
// issues them, two load (64 values at a time, 32 where inputs are pairs; on into the
// next item while the last one is being finished), sixteen take them apart: a lane per
// column of the keys, or per token j, a quarter of the tokens i each.
//
// Bounded by shared memory: products read both operands there, and so do the sixteen
// warps, whose steps follow one another.  So F is stored by whole 16-byte pieces (eight
// tokens i of a row j; number by number it took a sixth of the kernel), and gradients
// leave four columns at a time.  4 x 4096 tokens, 16 heads of 128 x 128: 282 us for
// 1.1 GB read and written, 3.9 TB/s.
#include <type_traits>

#include "delta_tmem.cuh"

namespace ps {

namespace {

constexpr int kGradWarps = 16, kGradThreads = 32 * (kGradWarps + 3);
constexpr int kZStride = kChunk + 8;   // eight columns of four rows in different banks
// Tensor-memory columns: X1, X2, X3, U dO^T, U dU^T (dU's two parts side by side), the products of
// F that go to dQ and to dK (and before them [K; Q] [K; Q]^T)
constexpr uint32_t kColX = 0, kColP = 192, kColN = 256, kColF = 384;

template <int NP, int KP>
struct GradSmem {
    static constexpr int kV = NP == 1 ? 64 : 32, kSlice = kV * 128;   // values taken at a time, bytes of 64 columns of them
    static constexpr int kKQ = (KP / 64) * kHalf, kSP = (KP / 64) * kSlice, kOP = kChunk * 128;   // planes
    // of a slice: U, dU (pairs), dO; S, dS' (pairs)
    static constexpr int kU = NP * kKQ, kDU = kU + 2 * kSlice, kO = kDU + 2 * kSlice, kS = kO + NP * kOP, kDS = kS + 2 * kSP;
    static constexpr int kF1 = kDS + 2 * kSP, kF2 = kF1 + 2 * (int)kSquare;   // pairs; before them what lanes j and 64 + j exchange
    static constexpr int kZ = kF2 + 2 * (int)kSquare, kKK = kZ + kChunk * kZStride * 4;
    static constexpr int kScal = (kKK + 2 * kChunk * kChunk * 4 + 15) / 16 * 16, kMore = kScal + 2 * 6 * kChunk * 4;   // scalars of two heads
    static constexpr int kBars = kMore + (4 * kChunk + 4 * kChunk + 4 * kChunk + kChunk + 16) * 4;
    static constexpr int kBytes = kBars + 512;
    static_assert(kBytes <= 227 * 1024, "too much shared memory");
};
struct GradItem {          // a chunk and key head
    long long token;         // its first token, among all of them
    int head_k, rows;        // rows 0: there are no more items
};
struct GradBars {
    uint64_t item_full[2], item_empty[2], u_full, u_empty, s_full, s_empty, kq_full, kq_empty, scal_full[2], scal_empty[2];
    uint64_t x_done, acc_free, f_ready, f_done, drained;
    GradItem item[2];
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(GradBars) <= 512, "room for the barriers");
// Whether any of the sixteen warps' threads says so; they wait for one another.
__device__ __forceinline__ bool meet_any(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"((uint32_t)x), "n"(32 * kGradWarps) : "memory");
    return r != 0;
}
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" :: "n"(32 * kGradWarps) : "memory"); }   // the sixteen warps

// Sums of 16 numbers each over the warp: lane l ends up with the l / 2-th.
__device__ __forceinline__ float sum16(float (&x)[16], int lane) {
#pragma unroll
    for (int step = 8, m = 16; step >= 1; step >>= 1, m >>= 1) {
        const bool high = lane & m;
#pragma unroll
        for (int i = 0; i < step; ++i) {
            const float send = high ? x[i] : x[i + step], keep = high ? x[i + step] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

// Lane l holds column l of 16 tokens and stores four columns (from `to` on) of tokens l % 4, l % 4 + 4, ... below `rows`.
template <typename T>
__device__ __forceinline__ void store_quads(const float (&x)[16], T *to, size_t stride, int lane, int rows, bool take) {
    const bool b0 = lane & 1, b1 = lane & 2;
    uint32_t w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const float got = __shfl_xor_sync(0xffffffffu, b0 ? x[2 * p] : x[2 * p + 1], 1);
        w[p] = b0 ? pack2<T>(got, x[2 * p + 1]) : pack2<T>(x[2 * p], got);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? w[2 * m] : w[2 * m + 1], 2);
        const int token = 4 * m + (lane & 3);
        if (take && token < rows)
            *reinterpret_cast<uint2 *>(to + token * stride) = b1 ? make_uint2(got, w[2 * m + 1]) : make_uint2(w[2 * m], got);
    }
}

}  // namespace

template <typename T, int KP>
__global__ void __launch_bounds__(kGradThreads, 1) delta_gradients_kernel(const DeltaArgs a) {
    constexpr int NP = Planes<T>::NP, KH = KP / 64;
    using M = GradSmem<NP, KP>;
    constexpr int kGradV = M::kV, kSlice = M::kSlice;
    extern __shared__ __align__(1024) unsigned char smem[];
    GradBars &bar = *reinterpret_cast<GradBars *>(smem + M::kBars);
    volatile int *gave_up = &bar.gave_up;
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // known to be uniform
    const int rep = a.s.hv / a.s.hk;
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, true);
    const int vpad = (a.s.v + 15) / 16 * 16;
    const bool quads = a.s.k % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.dq) | reinterpret_cast<uintptr_t>(a.dk)) & 7) == 0;

    if (tid == 0) {
        const int failed = *a.failed;   // what the chains kept is not to be used
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.item_full[i], 1);
            mbar_init(&bar.item_empty[i], kGradWarps + 1);
            mbar_init(&bar.scal_full[i], 1);
            mbar_init(&bar.scal_empty[i], kGradWarps);
        }
        mbar_init(&bar.u_full, 1 + 32);
        mbar_init(&bar.u_empty, 1);
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.s_empty, 1 + kGradWarps);
        mbar_init(&bar.kq_full, 1);
        mbar_init(&bar.kq_empty, kGradWarps);
        mbar_init(&bar.x_done, 1);
        mbar_init(&bar.acc_free, kGradWarps);
        mbar_init(&bar.f_ready, kGradWarps);
        mbar_init(&bar.f_done, 1);
        mbar_init(&bar.drained, 1);
        bar.gave_up = failed || base & 1023 ? 1 : 0;   // images need their alignment
        mbar_init_done();
    }
    if (warp == 0) tmem_alloc(smem_addr(&bar.tmem));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    constexpr uint32_t tm = 0;   // all columns are this CTA's
    if (tid == 0 && bar.tmem != tm) bar.gave_up = 1;

    if (warp == kGradWarps) {   // loads: items, scalars, U, dU, dO
        uint32_t n = 0, items = 0, heads = 0;   // slices, items and value heads so far
        const long long all = a.slots * a.s.hk;
        auto announce_item = [&](const GradItem &item) {
            if (items >= 2) wait_phase(&bar.item_empty[items & 1], (items / 2 - 1) & 1, gave_up);
            if (lane == 0) {
                bar.item[items & 1] = item;
                mbar_arrive(&bar.item_full[items & 1]);
            }
            ++items;
        };
        for (long long i = blockIdx.x; i < all && !*gave_up; i += gridDim.x) {
            const long long slot = i / a.s.hk, seq = seq_of_slot(a.s, slot);
            if (seq < 0) continue;
            const int head_k = (int)(i % a.s.hk);
            const Span sp = span_of(a.s, seq);
            const long long t0 = (slot - sp.slot) * kChunk;
            const int rows = (int)min((long long)kChunk, sp.len - t0);
            announce_item(GradItem{sp.first + t0, head_k, rows});
            for (int hr = 0; hr < rep; ++hr, ++heads) {
                const int head = head_k * rep + hr;
                const unsigned char *w = a.ws + (size_t)(slot * a.s.hv + head) * lay.stride;
                if (heads >= 2) wait_phase(&bar.scal_empty[heads & 1], (heads / 2 - 1) & 1, gave_up);
                if (lane == 0 && !*gave_up) {
                    mbar_arrive_expect_tx(&bar.scal_full[heads & 1], 6 * kChunk * 4);
                    bulk_load(smem + M::kScal + (heads & 1) * 6 * kChunk * 4, w + lay.scal, 6 * kChunk * 4, &bar.scal_full[heads & 1]);
                }
                const T *out = row_ptr<T>(a.dout, sp, seq, t0, head);
                for (int v0 = 0; v0 < vpad && !*gave_up; v0 += kGradV, ++n) {
                    const int bytes = min(kGradV, vpad - v0) * 128, vb = v0 / kBlockV, vi = v0 % kBlockV;
                    if (n) wait_phase(&bar.u_empty, (n - 1) & 1, gave_up);
                    if (*gave_up) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.u_full, 4 * bytes);
                        for (int p = 0; p < 2; ++p) {
                            const size_t from = (size_t)(vb * 2 + p) * kHalf + vi * 128;
                            bulk_load(smem + M::kU + p * kSlice, w + lay.u + from, bytes, &bar.u_full);
                            bulk_load(smem + M::kDU + p * kSlice, w + lay.du + from, bytes, &bar.u_full);
                        }
                    }
                    load_tile<T, kGradV>(base + M::kO, M::kOP, out + v0, a.dout.tok, rows, a.s.v - v0, a.vec_do != 0, lane, 32);
                    cp_async_commit();
                    cp_async_wait<0>();   // dO
                    fence_async();
                    mbar_arrive(&bar.u_full);
                }
            }
        }
        announce_item(GradItem{0, 0, 0});
        if (*gave_up && lane == 0 && n) wait_drained(&bar.u_full, (n - 1) & 1);   // copies in flight; without it the others have waited for every one
        __syncwarp();
    } else if (warp == kGradWarps + 2) {   // loads: S, dS', keys and queries
        if (lane == 0) {
            uint32_t n = 0, items = 0;
            const long long all = a.slots * a.s.hk;
            for (long long i = blockIdx.x; i < all && !*gave_up; i += gridDim.x) {
                const long long slot = i / a.s.hk;
                if (seq_of_slot(a.s, slot) < 0) continue;
                const int head_k = (int)(i % a.s.hk);
                // after the slices that go ahead while the last item's keys and queries are still in use
                int kq_after = vpad > kGradV ? 2 : 1;
                for (int hr = 0; hr < rep; ++hr) {
                    const unsigned char *w = a.ws + (size_t)(slot * a.s.hv + head_k * rep + hr) * lay.stride;
                    for (int v0 = 0; v0 < vpad && !*gave_up; v0 += kGradV, ++n) {
                        const int bytes = min(kGradV, vpad - v0) * 128, vb = v0 / kBlockV, vi = v0 % kBlockV;
                        if (n) wait_phase(&bar.s_empty, (n - 1) & 1, gave_up);
                        if (*gave_up) break;
                        mbar_arrive_expect_tx(&bar.s_full, 4 * KH * bytes);
                        for (int p = 0; p < 2 * KH; ++p) {   // parts and halves
                            const size_t from = (size_t)(vb * 2 * KH + p) * kHalf + vi * 128;
                            bulk_load(smem + M::kS + p * kSlice, w + lay.s + from, bytes, &bar.s_full);
                            bulk_load(smem + M::kDS + p * kSlice, w + lay.ds + from, bytes, &bar.s_full);
                        }
                        if (--kq_after == 0) {
                            if (items) wait_phase(&bar.kq_empty, (items - 1) & 1, gave_up);
                            if (*gave_up) { ++n; break; }
                            mbar_arrive_expect_tx(&bar.kq_full, NP * M::kKQ);
                            bulk_load(smem, a.kq + (size_t)(slot * a.s.hk + head_k) * kq_stride(a.s.k, NP), NP * M::kKQ, &bar.kq_full);
                            ++items;
                        }
                    }
                }
            }
            if (*gave_up && n) {   // copies in flight
                wait_drained(&bar.s_full, (n - 1) & 1);
                if (items) wait_drained(&bar.kq_full, (items - 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == kGradWarps + 1) {   // products
        const uint32_t one = elect_lane();
        constexpr uint32_t kSplit = KH == 2 ? kSlice : 0, kKSplit = KH == 2 ? kHalf : 0;   // 64 columns of keys only: twice the same rows
        const uint64_t u_left = operand(base + M::kU, false, kSlice), u_right = operand(base + M::kU, false, kSlice);
        const uint64_t du = operand(base + M::kDU, false, kSlice), o = operand(base + M::kO, true, 0);
        const uint64_t sl = operand(base + M::kS, false, kSplit), dsl = operand(base + M::kDS, false, kSplit);
        const uint64_t kq_rows = operand(base, true, 0), k_left = operand(base, false, kKSplit);
        const uint64_t f_rows = operand(base + M::kF1, true, 0), f_cols = operand(base + M::kF1, false, M::kF2 - M::kF1);
        uint32_t n = 0, heads = 0;
        for (uint32_t items = 0;; ++items) {
            wait_phase(&bar.item_full[items & 1], (items / 2) & 1, gave_up);
            const int rows = bar.item[items & 1].rows;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.item_empty[items & 1]);
            if (rows == 0 || *gave_up) break;
            for (int hr = 0; hr < rep; ++hr, ++heads) {
                if (heads) wait_phase(&bar.acc_free, (heads - 1) & 1, gave_up);
                for (int v0 = 0; v0 < vpad; v0 += kGradV, ++n) {
                    const int steps = min(kGradV, vpad - v0) / 16;
                    wait_phase(&bar.u_full, n & 1, gave_up);
                    tmem_fence_after();
#pragma unroll 1
                    for (int k = 0; k < steps; ++k) {
                        const bool add = v0 + k > 0;
#pragma unroll
                        for (int p = 0; p < NP; ++p)
                            mma_smem(one, tm + kColP, further(u_left, k * 2048), further(o, p * M::kOP + k * 32),
                                     shape(kChunk, true) | kLeftByColumns, add || p);
                        mma_smem(one, tm + kColN, further(u_left, k * 2048), further(du, k * 2048),
                                 shape(2 * kChunk, false) | kLeftByColumns, add);
                    }
                    wait_phase(&bar.s_full, n & 1, gave_up);
                    tmem_fence_after();
#pragma unroll 1
                    for (int k = 0; k < steps; ++k) {
                        const bool add = v0 + k > 0;
                        const uint64_t s0 = further(sl, k * 2048), d0 = further(dsl, k * 2048);
#pragma unroll
                        for (int p = 0; p < 2 * NP; ++p)   // S's parts, dO's parts
                            mma_smem(one, tm + kColX, further(s0, (p & 1) * M::kSP), further(o, (p >> 1) * M::kOP + k * 32),
                                     shape(kChunk, true) | kLeftByColumns, add || p);
#pragma unroll
                        for (int t = 0; t < 2 + NP; ++t) {   // hi hi, lo hi, hi lo, and lo lo for f16 and f32 (delta_common.cuh says why)
                            const uint32_t l = t & 1 ? M::kSP : 0, r = t & 2 ? kSlice : 0;
                            mma_smem(one, tm + kColX + 64, further(s0, l), further(du, r + k * 2048), shape(kChunk, false) | kLeftByColumns, add || t);
                            mma_smem(one, tm + kColX + 128, further(d0, l), further(u_right, r + k * 2048), shape(kChunk, false) | kLeftByColumns, add || t);
                        }
                    }
                    mma_commit(one, &bar.u_empty);
                    mma_commit(one, &bar.s_empty);
                }
                if (hr == 0) {   // [K; Q] [K; Q]^T
                    wait_phase(&bar.kq_full, items & 1, gave_up);
                    tmem_fence_after();
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int q = 0; q < NP; ++q)
#pragma unroll 1
                            for (int k = 0; k < KP / 16; ++k) {
                                const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
                                mma_smem(one, tm + kColF, further(kq_rows, p * M::kKQ + at), further(kq_rows, q * M::kKQ + at),
                                         shape(2 * kChunk, true), p + q + k > 0);
                            }
                }
                mma_commit(one, &bar.x_done);
                wait_phase(&bar.f_ready, heads & 1, gave_up);
                tmem_fence_after();
                // F1 K to dQ; F2 K, F1^T Q and F2^T K to dK, all transposed.  (F1 and F2 side by side would make one
                // product of the first two, but of another shape than those that add to half of its columns.)
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            const bool add = hr + p + h + k > 0;
                            const uint64_t kl = further(k_left, p * M::kKQ + k * 2048), ql = further(kl, kChunk * 128);
                            const uint64_t fr = further(f_rows, h * (uint32_t)kSquare + k * 32), fc = further(f_cols, h * (uint32_t)kSquare + k * 2048);
                            mma_smem(one, tm + kColF, kl, fc, shape(kChunk, false) | kLeftByColumns, add);
                            mma_smem(one, tm + kColF + 64, kl, further(fc, M::kF2 - M::kF1), shape(kChunk, false) | kLeftByColumns, add);
                            mma_smem(one, tm + kColF + 64, ql, fr, shape(kChunk, true) | kLeftByColumns, true);
                            mma_smem(one, tm + kColF + 64, kl, further(fr, M::kF2 - M::kF1), shape(kChunk, true) | kLeftByColumns, true);
                        }
                mma_commit(one, &bar.f_done);
            }
        }
        mma_commit(one, &bar.drained);
        wait_drained(&bar.drained, 0);
    } else {
        const int quadrant = warp & 3, part = warp >> 2, tok = 16 * part;   // this thread's tokens i: tok ..
        const uint32_t at = (uint32_t)quadrant << 21;                       // lane 32 quadrant
        const int col = 32 * quadrant + lane;                               // this thread's column of the keys
        const int j = col & 63, role = quadrant >> 1;                       // and its token j, with U's upper or lower part
        float *exch = reinterpret_cast<float *>(smem + M::kF1), *Z = reinterpret_cast<float *>(smem + M::kZ);
        float *kk = reinterpret_cast<float *>(smem + M::kKK), *qk = kk + kChunk * kChunk;   // [i][j]
        float *dots = reinterpret_cast<float *>(smem + M::kMore);   // [4 quadrants][64] of a_i
        float *dotb = dots + 4 * kChunk;                            // the same of b_j
        float *run = dotb + 4 * kChunk;                             // [4 quarters of the rows][64] column sums of Z
        float *diag = run + 4 * kChunk;                             // [64] dU_j . U_j
        float *inner = diag + kChunk;                               // <S, dS'> by warps
        uint32_t n = 0, heads = 0, items = 0;
        GradItem item;
        float prod = 0.f;   // this thread's part of <S, dS'>
        auto products = [&](int v0) {   // of a slice
            const int vr = min(kGradV, vpad - v0);
            wait_phase(&bar.s_full, n & 1, gave_up);
#pragma unroll 1
            for (int i = tid; i < kGradV * KP / 8; i += 32 * kGradWarps) {   // the same place in all four images
                if (i % (kGradV * 8) >= vr * 8) continue;                    // not loaded
                const uint4 *sv = reinterpret_cast<const uint4 *>(smem + M::kS) + i;
                const uint4 *dv = reinterpret_cast<const uint4 *>(smem + M::kDS) + i;
                const uint4 sh = sv[0], sl = sv[M::kSP / 16], dh = dv[0], dl = dv[M::kSP / 16];
                const uint32_t *shp = &sh.x, *slp = &sl.x, *dhp = &dh.x, *dlp = &dl.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    prod += (bf16_low(shp[e]) + bf16_low(slp[e])) * (bf16_low(dhp[e]) + bf16_low(dlp[e]));
                    prod += (bf16_high(shp[e]) + bf16_high(slp[e])) * (bf16_high(dhp[e]) + bf16_high(dlp[e]));
                }
            }
            warp_arrive(&bar.s_empty, lane);
            ++n;
        };
        auto next_item = [&]() -> bool {   // one decision for all; then the first slice, so that the second is loaded early
            wait_phase(&bar.item_full[items & 1], (items / 2) & 1, gave_up);
            item = bar.item[items & 1];
            const bool stop = meet_any(item.rows == 0 || *gave_up);
            warp_arrive(&bar.item_empty[items & 1], lane);
            ++items;
            if (!stop) products(0);
            return !stop;
        };
        for (bool more = next_item(); more;) {
            float dq[16], dk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) dq[i] = dk[i] = 0.f;

            for (int hr = 0; hr < rep; ++hr, ++heads) {
                const int head = item.head_k * rep + hr;
                const float *scal = reinterpret_cast<const float *>(smem + M::kScal + (heads & 1) * 6 * kChunk * 4);
                for (int v0 = kGradV; v0 < vpad; v0 += kGradV) products(v0);
#pragma unroll
                for (int m = 16; m; m >>= 1) prod += __shfl_xor_sync(0xffffffffu, prod, m);
                if (lane == 0) inner[warp] = prod;
                prod = 0.f;
                wait_phase(&bar.scal_full[heads & 1], (heads / 2) & 1, gave_up);
                if (hr == 0) wait_phase(&bar.kq_full, (items - 1) & 1, gave_up);
                if (heads) wait_phase(&bar.f_done, (heads - 1) & 1, gave_up);   // F has been used
                wait_phase(&bar.x_done, heads & 1, gave_up);
                tmem_fence_after();

                // U dO^T and U dU^T: lanes j and 64 + j hold what U's two parts give; each of the two
                // threads takes eight of the sixteen tokens i and sends the other eight
                float dp[8], dn[8];
                {
                    float p[16], u[16], w[16];
                    tmem_ld16(p, at + kColP + tok);
                    tmem_ld16(u, at + kColN + tok, w, at + kColN + kChunk + tok);
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[i] += w[i];
                    float *to = exch + (1 - role) * (kChunk * kChunk);   // [16 of P and N, 4 parts][64 j]
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        to[(part * 16 + i) * kChunk + j] = role ? p[i] : p[8 + i];
                        to[(part * 16 + 8 + i) * kChunk + j] = role ? u[i] : u[8 + i];
                        dp[i] = role ? p[8 + i] : p[i];
                        dn[i] = role ? u[8 + i] : u[i];
                    }
                    if (hr == 0 && role == 0) {   // k_j . k_i and k_j . q_i
                        tmem_ld16(u, at + kColF + tok, w, at + kColF + kChunk + tok);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            kk[(tok + i) * kChunk + j] = u[i];
                            qk[(tok + i) * kChunk + j] = w[i];
                        }
                    }
                }
                meet();
                float *from = exch + role * (kChunk * kChunk);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dp[i] += from[(part * 16 + i) * kChunk + j];
                    dn[i] += from[(part * 16 + 8 + i) * kChunk + j];
                }
                meet();   // the images of F take the place of what was exchanged

                // F1 = scale D dP and F2 = D dN, transposed, as pairs, and Z
                {
                    const float ghj = scal[192 + j], glj = scal[256 + j], rj = scal[320 + j];
                    const int i0 = tok + 8 * role;
                    float f1[8], f2[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 be = *reinterpret_cast<const float4 *>(scal + 128 + i0 + e), gh = *reinterpret_cast<const float4 *>(scal + 192 + i0 + e);
                        const float4 gl = *reinterpret_cast<const float4 *>(scal + 256 + i0 + e), rr = *reinterpret_cast<const float4 *>(scal + 320 + i0 + e);
                        auto one = [&](int m, float beta, float high, float low, float count) {
                            const int i = i0 + m;
                            const float D = i >= j && count == rj ? expf((high - ghj) + (low - glj)) : 0.f;
                            if (i == j) diag[j] = dn[m];
                            f1[m] = i >= j ? a.s.scale * D * dp[m] : 0.f;
                            f2[m] = i > j ? -beta * D * dn[m] : 0.f;
                            Z[i * kZStride + j] = i > j ? f1[m] * qk[i * kChunk + j] + f2[m] * kk[i * kChunk + j] : 0.f;
                        };
                        one(e, be.x, gh.x, gl.x, rr.x);
                        one(e + 1, be.y, gh.y, gl.y, rr.y);
                        one(e + 2, be.z, gh.z, gl.z, rr.z);
                        one(e + 3, be.w, gh.w, gl.w, rr.w);
                    }
                    const uint32_t ji = img(base + M::kF1, j, i0 >> 3);   // eight tokens i of row j
                    uint4 h, l;   // 16 bits, as of all that these products read
                    split2(f1[0], f1[1], h.x, l.x); split2(f1[2], f1[3], h.y, l.y); split2(f1[4], f1[5], h.z, l.z); split2(f1[6], f1[7], h.w, l.w);
                    st_shared16(ji, h);
                    st_shared16(ji + (uint32_t)kSquare, l);
                    split2(f2[0], f2[1], h.x, l.x); split2(f2[2], f2[3], h.y, l.y); split2(f2[4], f2[5], h.z, l.z); split2(f2[6], f2[7], h.w, l.w);
                    st_shared16(ji + (M::kF2 - M::kF1), h);
                    st_shared16(ji + (M::kF2 - M::kF1) + (uint32_t)kSquare, l);
                }
                fence_async();
                tmem_fence_before();
                warp_arrive(&bar.f_ready, lane);

                // through the states: a lane is a column of the keys
                {
                    float x[16], y[16], z[16];
                    tmem_ld16(x, at + kColX + tok, y, at + kColX + 64 + tok);
                    tmem_ld16(z, at + kColX + 128 + tok);
                    tmem_fence_before();
                    warp_arrive(&bar.acc_free, lane);
                    const uint32_t piece = (uint32_t)(col >> 3), in = (uint32_t)(col & 7) * 2;
#pragma unroll
                    for (int i4 = 0; i4 < 16; i4 += 4) {
                        const float4 eg4 = *reinterpret_cast<const float4 *>(scal + tok + i4), el4 = *reinterpret_cast<const float4 *>(scal + 64 + tok + i4);
                        const float4 be4 = *reinterpret_cast<const float4 *>(scal + 128 + tok + i4);
                        auto one = [&](int i, float eg, float el, float be) {
                            float kv = 0.f, qv = 0.f;
                            if (col < KP) {
                                const uint32_t k0 = img(0, tok + i, piece) + in, q0 = k0 + kChunk * 128;
                                kv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(smem + k0));
                                qv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(smem + q0));
                                if constexpr (NP == 2) {
                                    kv += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(smem + M::kKQ + k0));
                                    qv += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(smem + M::kKQ + q0));
                                }
                            }
                            const float x1 = a.s.scale * eg * x[i], x2 = eg * be * y[i], x3 = el * z[i];
                            dq[i] += x1;
                            dk[i] += x3 - x2;
                            x[i] = qv * x1 - kv * x2;   // to a_i
                            y[i] = kv * x3;             // to b_j
                        };
                        one(i4, eg4.x, el4.x, be4.x);
                        one(i4 + 1, eg4.y, el4.y, be4.y);
                        one(i4 + 2, eg4.z, el4.z, be4.z);
                        one(i4 + 3, eg4.w, el4.w, be4.w);
                    }
                    const float sa = sum16(x, lane), sb = sum16(y, lane);
                    if ((lane & 1) == 0) {
                        dots[quadrant * kChunk + tok + (lane >> 1)] = sa;
                        dotb[quadrant * kChunk + tok + (lane >> 1)] = sb;
                    }
                }
                meet();   // Z, the dots

                // sum over i >= t of Z_ij within quarters of 16 rows, then with the quarters below
                if (tid < 256) {
                    const int jj = tid & 63, q = tid >> 6;
                    float s = 0.f;
#pragma unroll
                    for (int t = 15; t >= 0; --t) {
                        s += Z[(16 * q + t) * kZStride + jj];
                        Z[(16 * q + t) * kZStride + jj] = s;
                    }
                    run[q * kChunk + jj] = s;
                } else if (tid < 256 + 2 * kChunk) {   // the quadrants' dots
                    float *d = (tid & kChunk ? dotb : dots) + (tid & 63);
                    d[0] = (d[0] + d[kChunk]) + (d[2 * kChunk] + d[3 * kChunk]);
                }
                meet();
                {   // row t: sum over j < t (eight threads a row), and all else for token t
                    const int t = tid >> 3, sub = tid & 7;
                    float s = 0.f;
#pragma unroll
                    for (int m = 0; m < kChunk; m += 8) {
                        const int jj = sub + m;
                        float z = Z[t * kZStride + jj];
#pragma unroll
                        for (int q = 1; q < 4; ++q) z += q > t >> 4 ? run[q * kChunk + jj] : 0.f;
                        // a_i of i >= t, b_j of j < t, <S, dS'>
                        s += jj < t ? z + dotb[jj] : dots[jj];
                    }
                    s += scal[kChunk - 1] * (inner[sub] + inner[8 + sub]);
#pragma unroll
                    for (int m = 1; m < 8; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                    if (sub == 0 && t < item.rows) {
                        // the decay of a token that forgets the state scales nothing
                        const bool forgets = scal[320 + t] != (t ? scal[319 + t] : 0.f);
                        const size_t out = (size_t)(item.token + t) * a.s.hv + head;
                        a.dg[out] = forgets ? 0.f : s;
                        const float d = diag[t] / scal[128 + t];
                        if (a.beta_f32) static_cast<float *>(a.dbeta)[out] = d;
                        else static_cast<T *>(a.dbeta)[out] = from_f32<T>(d);
                    }
                }
                meet();
                warp_arrive(&bar.scal_empty[heads & 1], lane);
                if (hr + 1 < rep) products(0);   // of the next head
            }
            const GradItem was = item;
            more = next_item();
            wait_phase(&bar.f_done, (heads - 1) & 1, gave_up);
            tmem_fence_after();
            {
                float x[16], y[16];
                tmem_ld16(x, at + kColF + tok, y, at + kColF + 64 + tok);
                tmem_fence_before();
                warp_arrive(&bar.kq_empty, lane);
                const size_t ostride = (size_t)a.s.hk * a.s.k, first = ((size_t)(was.token + tok) * a.s.hk + was.head_k) * a.s.k + col;
                T *oq = static_cast<T *>(a.dq) + first, *ok = static_cast<T *>(a.dk) + first;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    dq[i] += x[i];
                    dk[i] += y[i];
                }
                if constexpr (sizeof(T) == 2)
                    if (quads) {   // four lanes exchange, so that each has four columns of every fourth token
                        store_quads<T>(dq, oq - (lane & 3), ostride, lane, was.rows - tok, col < a.s.k);
                        store_quads<T>(dk, ok - (lane & 3), ostride, lane, was.rows - tok, col < a.s.k);
                    }
                if ((sizeof(T) > 2 || !quads) && col < a.s.k) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (tok + i < was.rows) {
                            oq[i * ostride] = from_f32<T>(dq[i]);
                            ok[i * ostride] = from_f32<T>(dk[i]);
                        }
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (a.s.cu) {   // tokens of no sequence: before the first one and after the last, or between them where offsets fall
        int falls = 0;
        for (long long i = tid; i < a.s.seqs; i += kGradThreads) falls |= a.s.cu[i + 1] < a.s.cu[i];
        falls = __syncthreads_or(falls);
        const Span last = span_of(a.s, a.s.seqs - 1);
        const long long before = span_of(a.s, 0).first, from = last.first + last.len;
        const long long n = falls ? a.s.tokens : before + a.s.tokens - from;
        for (long long i = blockIdx.x; i < n; i += gridDim.x) {
            const long long t = falls || i < before ? i : i - before + from;
            if (falls) {
                int held = 0;
                for (long long q = tid; q < a.s.seqs; q += kGradThreads) {
                    const Span sp = span_of(a.s, q);
                    held |= t >= sp.first && t < sp.first + sp.len;
                }
                if (__syncthreads_or(held)) continue;
            }
            auto clear = [&](auto *p, int width) {
                for (int x = tid; x < width; x += kGradThreads) p[t * width + x] = from_f32<std::remove_reference_t<decltype(*p)>>(0.f);
            };
            clear(static_cast<T *>(a.dq), a.s.hk * a.s.k);
            clear(static_cast<T *>(a.dk), a.s.hk * a.s.k);
            clear(static_cast<T *>(a.dv), a.s.hv * a.s.v);
            clear(a.dg, a.s.hv);
            if (a.beta_f32) clear(static_cast<float *>(a.dbeta), a.s.hv);
            else clear(static_cast<T *>(a.dbeta), a.s.hv);
        }
    }
    if (*gave_up) {   // this CTA's items are not what they should be: say so
        const float bad = __int_as_float(0x7fffffff);
        for (long long i = blockIdx.x; i < a.slots * a.s.hk; i += gridDim.x) {
            const long long slot = i / a.s.hk, seq = seq_of_slot(a.s, slot);
            if (seq < 0) continue;
            const Span sp = span_of(a.s, seq);
            const long long t0 = (slot - sp.slot) * kChunk;
            const int rows = (int)min((long long)kChunk, sp.len - t0), head_k = (int)(i % a.s.hk);
            for (int x = tid; x < rows * a.s.k; x += kGradThreads) {
                const size_t at = ((size_t)(sp.first + t0 + x / a.s.k) * a.s.hk + head_k) * a.s.k + x % a.s.k;
                static_cast<T *>(a.dq)[at] = static_cast<T *>(a.dk)[at] = from_f32<T>(bad);
            }
            for (int x = tid; x < rows * rep; x += kGradThreads) {
                const size_t at = (size_t)(sp.first + t0 + x / rep) * a.s.hv + head_k * rep + x % rep;
                a.dg[at] = bad;
                if (a.beta_f32) static_cast<float *>(a.dbeta)[at] = bad;
                else static_cast<T *>(a.dbeta)[at] = from_f32<T>(bad);
            }
        }
    }
    if (warp == 0) tmem_free(bar.tmem);
}

namespace {

template <typename T, int KP>
cudaError_t gradients(const DeltaArgs &a, cudaStream_t s) {
    constexpr int bytes = GradSmem<Planes<T>::NP, KP>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(delta_gradients_kernel<T, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long long items = a.slots * a.s.hk;
    delta_gradients_kernel<T, KP><<<(unsigned)(items < 152 ? items : 152), kGradThreads, bytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_gradients(const DeltaArgs &a, int type, cudaStream_t s) {
    const bool small = a.s.k <= 64;
    switch (type) {
    case PS_REAL_BF16: return small ? gradients<__nv_bfloat16, 64>(a, s) : gradients<__nv_bfloat16, 128>(a, s);
    case PS_REAL_F16: return small ? gradients<__half, 64>(a, s) : gradients<__half, 128>(a, s);
    default: return small ? gradients<float, 64>(a, s) : gradients<float, 128>(a, s);
    }
}

}  // namespace ps
