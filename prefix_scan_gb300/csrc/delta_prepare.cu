// delta_prepare.cu -- what the chunks of the gated delta rule need before
// their states are known: decays, the masked products P and N, the triangular
// inverse T (notation in delta_common.cuh), and the chunk's keys and queries as
// images.  One CTA per chunk and key head, all chunks at once; the products
// k k^T and q k^T stay in registers for all value heads that share the key head.
//
// T comes in blocks of 16: the four diagonal blocks by forward substitution in
// f32 (one column per thread), the blocks below them a block column per warp,
//     T_ij = -T_ii diag(beta) sum_{j <= l < i} N_il T_lj,
// transposed, so that each product's left operand is the result before it in
// the warp's registers.
//
// Bounded by the waits between these steps (a third of the issue slots busy), so
// CTAs are small and four share an SM: P passes through the place that T takes,
// and T's diagonal blocks through N's.  12345 tokens in 48 sequences, 16 key heads
// and 32 value heads of 128: 114 us, 4.0 TB/s written and read (three CTAs an SM,
// with a place for each: 137; five, at 96 registers: 119).
#include "delta_common.cuh"

namespace ps {

namespace {

constexpr int kPrepThreads = 128;   // four warps: 16 rows of a 64 x 64 product each
// Scalars of a value head: the six arrays of ChunkLayout; exp(G_i - G_m) with m the last token before i's
// block of 16 (1 in the first block); exp(G_m - G_j) for the m of each of blocks 1, 2, 3.  Both are at most
// 1, and their product is D below the diagonal blocks, at one exponential a row and column.
constexpr int kRow = 6 * kChunk, kCol = 7 * kChunk, kScalars = 10 * kChunk;
constexpr int kDiag = 264;          // floats from one diagonal block to the next: 16 x 16, and 8 against bank conflicts

template <int NP, int KP>
struct PrepSmem {
    static constexpr int kPlane = 2 * kChunk * KP * 2;                           // keys, then queries
    static constexpr int kK = 0, kQ = kChunk * 128;
    // in the place of K and Q: P, later T; N below its diagonal blocks, and T's diagonal blocks in theirs
    static constexpr int kT = 0, kN = 2 * (int)kSquare;
    static constexpr int kScal = NP * kPlane > 4 * (int)kSquare ? NP * kPlane : 4 * (int)kSquare;
    static constexpr int kL = kScal + 4 * kScalars * 4;                          // f32 diagonal blocks of diag(beta) N
    static constexpr int kBytes = kL + 4 * kDiag * 4;
};

// exp(x) leaves f32's normal range below this: the state is forgotten.
constexpr float kForget = -87.f;
// In the place of smaller gates: the backward pass divides by beta.  No result changes by more than that.
constexpr float kLeastBeta = 0x1p-60f;

}  // namespace

template <typename T, int KP>
__global__ void __launch_bounds__(kPrepThreads, Planes<T>::NP == 1 ? 4 : KP == 64 ? 3 : 2) delta_prepare_kernel(const DeltaArgs a) {
    constexpr int NP = Planes<T>::NP;
    using M = PrepSmem<NP, KP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    float *L = reinterpret_cast<float *>(smem + M::kL);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long slot = blockIdx.x;
    const int head_k = blockIdx.y, rep = a.s.hv / a.s.hk;

    if (a.failed && slot == 0 && head_k == 0 && tid == 0) *a.failed = 0;
    if (a.order && slot == 0 && head_k == 0) {
        int *len = reinterpret_cast<int *>(smem);
        for (int i = tid; i < a.s.seqs; i += kPrepThreads) len[i] = (int)span_of(a.s, i).len;
        __syncthreads();
        for (int i = tid; i < a.s.seqs; i += kPrepThreads) {
            int rank = 0;
            for (int j = 0; j < a.s.seqs; ++j) rank += len[j] > len[i] || (len[j] == len[i] && j < i);
            a.order[rank] = i;
        }
        __syncthreads();
    }
    const long long seq = seq_of_slot(a.s, slot);
    if (seq < 0) return;
    const Span sp = span_of(a.s, seq);
    const long long t0 = (slot - sp.slot) * kChunk;
    const int rows = (int)min((long long)kChunk, sp.len - t0);

    load_tile<T, KP>(base + M::kK, M::kPlane, row_ptr<T>(a.k, sp, seq, t0, head_k), a.k.tok, rows, a.s.k, a.vec_qk != 0,
                     tid, kPrepThreads);
    load_tile<T, KP>(base + M::kQ, M::kPlane, row_ptr<T>(a.q, sp, seq, t0, head_k), a.q.tok, rows, a.s.k, a.vec_qk != 0,
                     tid, kPrepThreads);
    cp_async_commit();
    // the scalars of four value heads from the hr-th on, one per warp: tokens 2 lane, 2 lane + 1
    auto scalars = [&](int hr) {
        if (hr + warp < rep) {
            float *sc = reinterpret_cast<float *>(smem + M::kScal) + warp * kScalars;
            const int head = head_k * rep + hr + warp;
            const float *gp = row_ptr<float>(a.g, sp, seq, t0, head);
            float g[2], b[2] = {0.f, 0.f};
            bool f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                g[e] = i < rows ? gp[i * a.g.tok] : 0.f;
                if (i < rows)
                    b[e] = a.beta_f32 ? row_ptr<float>(a.beta, sp, seq, t0, head)[i * a.beta.tok]
                                      : to_f32<T>(row_ptr<T>(a.beta, sp, seq, t0, head)[i * a.beta.tok]);
                if (fabsf(b[e]) < kLeastBeta) b[e] = kLeastBeta;
                f[e] = g[e] <= kForget;
                if (f[e]) g[e] = 0.f;
            }
            // running sums of g in 64 bits, kept as two floats: differences of far sums stay exact to
            // f32.  Tokens that forget the state start a new count r; sums go on without them.
            double sum = (double)g[0] + (double)g[1];
            int cnt = (int)f[0] + (int)f[1];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double s2 = __shfl_up_sync(0xffffffffu, sum, d);
                const int c2 = __shfl_up_sync(0xffffffffu, cnt, d);
                if (lane >= d) { sum += s2; cnt += c2; }
            }
            const double last = __shfl_sync(0xffffffffu, sum, 31);
            const int rlast = __shfl_sync(0xffffffffu, cnt, 31);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                const double G = e ? sum : sum - (double)g[1];
                const int r = e ? cnt : cnt - (int)f[1];
                const float hi = (float)G;
                sc[i] = r == 0 ? exp_rounded((float)G) : 0.f;   // the 63rd multiplies the state
                sc[64 + i] = i < rows && r == rlast ? expf((float)(last - G)) : 0.f;
                sc[128 + i] = b[e];
                sc[192 + i] = hi;
                sc[256 + i] = (float)(G - (double)hi);
                sc[320 + i] = (float)r;
            }
#pragma unroll
            for (int blk = 0; blk < 4; ++blk) {   // m = 16 blk - 1, in lane 8 blk - 1
                const double Gm = __shfl_sync(0xffffffffu, sum, blk ? 8 * blk - 1 : 0);
                const int rm = __shfl_sync(0xffffffffu, cnt, blk ? 8 * blk - 1 : 0);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    const double G = e ? sum : sum - (double)g[1];
                    const int r = e ? cnt : cnt - (int)f[1];
                    if (i >> 4 == blk) sc[kRow + i] = blk == 0 ? 1.f : r == rm ? expf((float)(G - Gm)) : 0.f;
                    if (blk && i < 16 * blk) sc[kCol + (blk - 1) * kChunk + i] = r == rm ? expf((float)(Gm - G)) : 0.f;
                }
            }
        }
    };
    scalars(0);   // while keys and queries are on their way
    cp_async_wait<0>();
    __syncthreads();

    // k k^T and q k^T: a warp's diagonal block, and one or two of the six below them
    int bi[3], bj[3];
    bi[0] = bj[0] = warp;
    bi[1] = warp < 2 ? 3 : warp == 2 ? 2 : 1;
    bj[1] = warp == 1 ? 2 : warp == 2 ? 1 : 0;
    bi[2] = 3 - warp;
    bj[2] = 1 - warp;
    const int blocks = warp < 2 ? 3 : 2;
    float kk[3][2][4], qk[3][2][4];
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[n][0][e] = kk[n][1][e] = qk[n][0][e] = qk[n][1][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            if (n >= blocks) continue;
            uint32_t ak[NP][4], aq[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                load_a(ak[p], base + M::kK + p * M::kPlane, 16 * bi[n], 16 * kt, lane);
                load_a(aq[p], base + M::kQ + p * M::kPlane, 16 * bi[n], 16 * kt, lane);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                uint32_t b[4];
                load_b(b, base + M::kK + p * M::kPlane, 16 * bj[n], 16 * kt, lane);
#pragma unroll
                for (int f = 0; f < NP; ++f) {
                    mma_bf16(kk[n][0], ak[f], b[0], b[1]);
                    mma_bf16(kk[n][1], ak[f], b[2], b[3]);
                    mma_bf16(qk[n][0], aq[f], b[0], b[1]);
                    mma_bf16(qk[n][1], aq[f], b[2], b[3]);
                }
            }
        }
    }
    {
        uint4 *kq = reinterpret_cast<uint4 *>(a.kq + (size_t)(slot * a.s.hk + head_k) * kq_stride(a.s.k, NP));
#pragma unroll
        for (int i = 0; i < NP * M::kPlane / (16 * kPrepThreads); ++i)
            kq[i * kPrepThreads + tid] = reinterpret_cast<const uint4 *>(smem + M::kK)[i * kPrepThreads + tid];
    }
    __syncthreads();

#pragma unroll
    for (int np = 1; np < 4; ++np)   // above the diagonal blocks P and T are 0, for all heads
        if (np > warp) {
            const uint32_t at = img(base + M::kT, 16 * warp + (lane & 15), 2 * np + (lane >> 4));
            stsm4(at, 0, 0, 0, 0);
            stsm4(at + (uint32_t)kSquare, 0, 0, 0, 0);
        }
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, a.train != 0);
    for (int hr = 0; hr < rep; ++hr) {
        const int head = head_k * rep + hr;
        float *scal = reinterpret_cast<float *>(smem + M::kScal) + (hr & 3) * kScalars;
        unsigned char *out = a.ws + (size_t)(slot * a.s.hv + head) * lay.stride;
        if (hr > 0 && (hr & 3) == 0) {
            scalars(hr);
            __syncthreads();
        }

        // P and N as pairs, the diagonal blocks of diag(beta) N in f32
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            if (n >= blocks) continue;
            const int r8 = lane >> 2, i0 = 16 * bi[n] + r8, c2 = 2 * (lane & 3);
            const uint32_t at = img(base + M::kT, 16 * bi[n] + (lane & 15), 2 * bj[n] + (lane >> 4));
            float nv[2][4], pv[2][4];   // tiles of the block
            uint32_t f[2][4];
            if (n > 0) {
                const float row0 = scal[kRow + i0], row1 = scal[kRow + i0 + 8];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float2 col = *reinterpret_cast<const float2 *>(scal + kCol + (bi[n] - 1) * kChunk + 16 * bj[n] + 8 * t + c2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float D = (e < 2 ? row0 : row1) * (e & 1 ? col.y : col.x);
                        nv[t][e] = D * kk[n][t][e];
                        pv[t][e] = a.s.scale * D * qk[n][t][e];
                    }
                }
                split_tiles(nv[0], nv[1], f);   // 16 bits: T's blocks and P are read as pairs by the chains anyway
                stsm4(at + M::kN, f[0][0], f[0][1], f[0][2], f[0][3]);
                stsm4(at + M::kN + (uint32_t)kSquare, f[1][0], f[1][1], f[1][2], f[1][3]);
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = i0 + 8 * (e >> 1), c = 16 * warp + 8 * t + c2 + (e & 1);
                        const float dx = (scal[192 + i] - scal[192 + c]) + (scal[256 + i] - scal[256 + c]);
                        const float D = i >= c && scal[320 + i] == scal[320 + c] ? expf(dx) : 0.f;
                        nv[t][e] = i > c ? D * kk[n][t][e] : 0.f;
                        pv[t][e] = i >= c ? a.s.scale * D * qk[n][t][e] : 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float be = scal[128 + i0 + 8 * e];
                        *reinterpret_cast<float2 *>(L + warp * kDiag + (r8 + 8 * e) * 16 + 8 * t + c2) =
                            make_float2(be * nv[t][2 * e], be * nv[t][2 * e + 1]);
                    }
                }
            }
            split_tiles(pv[0], pv[1], f);
            stsm4(at, f[0][0], f[0][1], f[0][2], f[0][3]);
            stsm4(at + (uint32_t)kSquare, f[1][0], f[1][1], f[1][2], f[1][3]);
        }
        __syncthreads();

        if (tid < kChunk) {
            // column c of a diagonal block by forward substitution: x_i = delta_ic - sum_{l < i} L_il x_l
            const int c = tid & 15;
            const float *D = L + (tid >> 4) * kDiag;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s[4] = {i == c ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int l = 0; l < i; l += 4) {
                    const float4 d = *reinterpret_cast<const float4 *>(D + i * 16 + l);
                    s[0] -= d.x * x[l];
                    if (l + 1 < i) s[1] -= d.y * x[l + 1];
                    if (l + 2 < i) s[2] -= d.z * x[l + 2];
                    if (l + 3 < i) s[3] -= d.w * x[l + 3];
                }
                x[i] = (s[0] + s[1]) + (s[2] + s[3]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {   // solved in f32, 16 bits of it for the products below and for the chains
                const __nv_bfloat16 h = __float2bfloat16_rn(x[i]);
                const __nv_bfloat16 l = __float2bfloat16_rn(x[i] - __bfloat162float(h));
                const int at = (int)img(0, (tid & ~15) + i, tid >> 3) + (tid & 7) * 2;
                *reinterpret_cast<__nv_bfloat16 *>(smem + M::kN + at) = h;
                *reinterpret_cast<__nv_bfloat16 *>(smem + M::kN + kSquare + at) = l;
            }
        } else {   // the other warps take P out meanwhile
#pragma unroll 4
            for (int i = tid - kChunk; i < 2 * (int)kSquare / 16; i += kPrepThreads - kChunk)
                reinterpret_cast<uint4 *>(out + lay.p)[i] = reinterpret_cast<const uint4 *>(smem + M::kT)[i];
        }
        __syncthreads();

        if (warp == 3) {   // which has no blocks below its diagonal one: T's diagonal blocks
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = img(p * (uint32_t)kSquare, 16 * i + (lane & 15), 2 * i + (lane >> 4));
                    *reinterpret_cast<uint4 *>(smem + M::kT + at) = *reinterpret_cast<const uint4 *>(smem + M::kN + at);
                }
        } else {   // block column `warp` below its diagonal block
            uint32_t x[4][2][4];   // T_lj^T as left operands
#pragma unroll
            for (int p = 0; p < 2; ++p)
                load_a_t(x[0][p], base + M::kN + p * (uint32_t)kSquare, 16 * warp, 16 * warp, lane);
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int i = warp + d;
                if (i > 3) continue;
                float y[2][4], z[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[0][e] = y[1][e] = z[0][e] = z[1][e] = 0.f;
#pragma unroll
                for (int l = 0; l < d; ++l) {
                    uint32_t bh[4], bl[4];
                    load_b(bh, base + M::kN, 16 * i, 16 * (warp + l), lane);
                    load_b(bl, base + M::kN + (uint32_t)kSquare, 16 * i, 16 * (warp + l), lane);
                    mma_bf16(y[0], x[l][0], bh[0], bh[1]);
                    mma_bf16(y[1], x[l][0], bh[2], bh[3]);
                    mma_bf16(y[0], x[l][1], bh[0], bh[1]);
                    mma_bf16(y[1], x[l][1], bh[2], bh[3]);
                    mma_bf16(y[0], x[l][0], bl[0], bl[1]);
                    mma_bf16(y[1], x[l][0], bl[2], bl[3]);
                    mma_bf16(y[0], x[l][1], bl[0], bl[1]);
                    mma_bf16(y[1], x[l][1], bl[2], bl[3]);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float2 be = *reinterpret_cast<const float2 *>(scal + 128 + 16 * i + 8 * t + 2 * (lane & 3));
                    y[t][0] *= -be.x; y[t][1] *= -be.y; y[t][2] *= -be.x; y[t][3] *= -be.y;
                }
                uint32_t f[2][4], bh[4], bl[4];
                split_tiles(y[0], y[1], f);
                load_b(bh, base + M::kN, 16 * i, 16 * i, lane);
                load_b(bl, base + M::kN + (uint32_t)kSquare, 16 * i, 16 * i, lane);
                mma_bf16(z[0], f[0], bh[0], bh[1]);
                mma_bf16(z[1], f[0], bh[2], bh[3]);
                mma_bf16(z[0], f[1], bh[0], bh[1]);
                mma_bf16(z[1], f[1], bh[2], bh[3]);
                mma_bf16(z[0], f[0], bl[0], bl[1]);
                mma_bf16(z[1], f[0], bl[2], bl[3]);
                mma_bf16(z[0], f[1], bl[0], bl[1]);
                mma_bf16(z[1], f[1], bl[2], bl[3]);
                split_tiles(z[0], z[1], x[d]);
                const uint32_t at = img(base + M::kT, 16 * i + (lane & 7) + ((lane >> 4) << 3), 2 * warp + ((lane >> 3) & 1));
                stsm4_t(at, x[d][0][0], x[d][0][1], x[d][0][2], x[d][0][3]);
                stsm4_t(at + (uint32_t)kSquare, x[d][1][0], x[d][1][1], x[d][1][2], x[d][1][3]);
            }
        }
        __syncthreads();

#pragma unroll 4
        for (int i = tid; i < 2 * (int)kSquare / 16; i += kPrepThreads) {
            uint4 x = reinterpret_cast<const uint4 *>(smem + M::kT)[i];
            const int row = i >> 3 & 63;
            if (((i ^ row) & 7) == row >> 3) {   // the image is T - 1
                const uint32_t keep = row & 1 ? 0xffffu : 0xffff0000u;
                (row & 4 ? row & 2 ? x.w : x.z : row & 2 ? x.y : x.x) &= keep;
            }
            reinterpret_cast<uint4 *>(out + lay.t)[i] = x;
        }
        for (int i = tid; i < 6 * kChunk; i += kPrepThreads) reinterpret_cast<float *>(out + lay.scal)[i] = scal[i];
        __syncthreads();
    }
}

namespace {

template <typename T, int KP>
cudaError_t prepare(const DeltaArgs &a, cudaStream_t s) {
    constexpr int bytes = PrepSmem<Planes<T>::NP, KP>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel<T, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    delta_prepare_kernel<T, KP><<<dim3((unsigned)a.slots, (unsigned)a.s.hk), kPrepThreads, bytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prepare(const DeltaArgs &a, int type, cudaStream_t s) {
    const bool small = a.s.k <= 64;
    switch (type) {
    case PS_REAL_BF16: return small ? prepare<__nv_bfloat16, 64>(a, s) : prepare<__nv_bfloat16, 128>(a, s);
    case PS_REAL_F16: return small ? prepare<__half, 64>(a, s) : prepare<__half, 128>(a, s);
    default: return small ? prepare<float, 64>(a, s) : prepare<float, 128>(a, s);
    }
}

}  // namespace ps
