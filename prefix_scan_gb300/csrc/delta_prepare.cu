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
    static constexpr int kT = 0, kP = 2 * (int)kSquare, kN = 4 * (int)kSquare;   // in the place of K and Q
    static constexpr int kScal = NP * kPlane > 6 * (int)kSquare ? NP * kPlane : 6 * (int)kSquare;
    static constexpr int kL = kScal + 4 * kScalars * 4;                          // f32 diagonal blocks of diag(beta) N
    static constexpr int kBytes = kL + 4 * kDiag * 4;
};

// exp(x) leaves f32's normal range below this: the state is forgotten.
constexpr float kForget = -87.f;
// In the place of smaller gates: the backward pass divides by beta.  No result changes by more than that.
constexpr float kLeastBeta = 0x1p-60f;

}  // namespace

template <typename T, int KP>
__global__ void __launch_bounds__(kPrepThreads, 3) delta_prepare_kernel(const DeltaArgs a) {
    constexpr int NP = Planes<T>::NP;
    using M = PrepSmem<NP, KP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    float *L = reinterpret_cast<float *>(smem + M::kL);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long slot = blockIdx.x;
    const int head_k = blockIdx.y, rep = a.s.hv / a.s.hk;

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
                sc[i] = r == 0 ? expf((float)G) : 0.f;
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

    // rows 16 warp .. of k k^T and q k^T, columns j <= i only
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
        uint32_t ak[NP][4], aq[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            load_a(ak[p], base + M::kK + p * M::kPlane, 16 * warp, 16 * kt, lane);
            load_a(aq[p], base + M::kQ + p * M::kPlane, 16 * warp, 16 * kt, lane);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np <= warp) {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    uint32_t b[4];
                    load_b(b, base + M::kK + p * M::kPlane, 16 * np, 16 * kt, lane);
#pragma unroll
                    for (int f = 0; f < NP; ++f) {
                        mma_bf16(kk[2 * np], ak[f], b[0], b[1]);
                        mma_bf16(kk[2 * np + 1], ak[f], b[2], b[3]);
                        mma_bf16(qk[2 * np], aq[f], b[0], b[1]);
                        mma_bf16(qk[2 * np + 1], aq[f], b[2], b[3]);
                    }
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

    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, a.train != 0);
    for (int hr = 0; hr < rep; ++hr) {
        const int head = head_k * rep + hr;
        float *scal = reinterpret_cast<float *>(smem + M::kScal) + (hr & 3) * kScalars;
        if (hr > 0 && (hr & 3) == 0) {
            scalars(hr);
            __syncthreads();
        }

        {   // P and N as pairs, the diagonal blocks of diag(beta) N in f32
            const int r8 = lane >> 2, i0 = 16 * warp + r8, c2 = 2 * (lane & 3);
            const float row0 = scal[kRow + i0], row1 = scal[kRow + i0 + 8];
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                const uint32_t at = img(0, 16 * warp + (lane & 15), 2 * np + (lane >> 4));
                if (np > warp) {   // above the diagonal: T and P are 0, N is not read
#pragma unroll
                    for (int m = 0; m < 4; ++m) stsm4(base + M::kT + at + m * (uint32_t)kSquare, 0, 0, 0, 0);
                    continue;
                }
                float nv[2][4], pv[2][4];   // tiles of the block
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int n = 2 * np + t, j = 8 * n + c2;
                    if (np < warp) {
                        const float2 col = *reinterpret_cast<const float2 *>(scal + kCol + (warp - 1) * kChunk + j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float D = (e < 2 ? row0 : row1) * (e & 1 ? col.y : col.x);
                            nv[t][e] = D * kk[n][e];
                            pv[t][e] = a.s.scale * D * qk[n][e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = i0 + 8 * (e >> 1), c = j + (e & 1);
                            const float dx = (scal[192 + i] - scal[192 + c]) + (scal[256 + i] - scal[256 + c]);
                            const float D = i >= c && scal[320 + i] == scal[320 + c] ? expf(dx) : 0.f;
                            nv[t][e] = i > c ? D * kk[n][e] : 0.f;
                            pv[t][e] = i >= c ? a.s.scale * D * qk[n][e] : 0.f;
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float be = scal[128 + i0 + 8 * r];
                            *reinterpret_cast<float2 *>(L + warp * kDiag + (r8 + 8 * r) * 16 + 8 * t + c2) =
                                make_float2(be * nv[t][2 * r], be * nv[t][2 * r + 1]);
                        }
                    }
                }
                uint32_t f[2][4];
                split_tiles(pv[0], pv[1], f);
                stsm4(base + M::kP + at, f[0][0], f[0][1], f[0][2], f[0][3]);
                stsm4(base + M::kP + (uint32_t)kSquare + at, f[1][0], f[1][1], f[1][2], f[1][3]);
                split_tiles(nv[0], nv[1], f);
                stsm4(base + M::kN + at, f[0][0], f[0][1], f[0][2], f[0][3]);
                stsm4(base + M::kN + (uint32_t)kSquare + at, f[1][0], f[1][1], f[1][2], f[1][3]);
            }
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
            for (int i = 0; i < 16; ++i) {
                const __nv_bfloat16 h = __float2bfloat16_rn(x[i]);
                const __nv_bfloat16 l = __float2bfloat16_rn(x[i] - __bfloat162float(h));
                const int at = (int)img(0, (tid & ~15) + i, tid >> 3) + (tid & 7) * 2;
                *reinterpret_cast<__nv_bfloat16 *>(smem + M::kT + at) = h;
                *reinterpret_cast<__nv_bfloat16 *>(smem + M::kT + kSquare + at) = l;
            }
        }
        __syncthreads();

        {   // block column `warp` below its diagonal block
            uint32_t x[4][2][4];   // T_lj^T as left operands
#pragma unroll
            for (int p = 0; p < 2; ++p)
                load_a_t(x[0][p], base + M::kT + p * (uint32_t)kSquare, 16 * warp, 16 * warp, lane);
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
                load_b(bh, base + M::kT, 16 * i, 16 * i, lane);
                load_b(bl, base + M::kT + (uint32_t)kSquare, 16 * i, 16 * i, lane);
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

        if (tid < kChunk) {   // the image is T - 1
            const uint32_t at = img(0, tid, tid >> 3) + (tid & 7) * 2;
            *reinterpret_cast<uint16_t *>(smem + M::kT + at) = 0;
            *reinterpret_cast<uint16_t *>(smem + M::kT + kSquare + at) = 0;
        }
        __syncthreads();
        unsigned char *out = a.ws + (size_t)(slot * a.s.hv + head) * lay.stride;
        constexpr int imgs = 4 * (int)kSquare / 16;   // T and P follow one another on both sides
#pragma unroll 4
        for (int i = tid; i < imgs; i += kPrepThreads)
            reinterpret_cast<uint4 *>(out + lay.t)[i] = reinterpret_cast<const uint4 *>(smem + M::kT)[i];
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
