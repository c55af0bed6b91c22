// delta_chain.cu -- the gated delta rule's states, chunk after chunk, and its
// outputs (notation in delta_common.cuh).
//
// A warp owns 16 of the V columns of one head's state, transposed: S^T is a
// 16 x K accumulator in registers, and every product of a chunk,
//     X^T = S^T K^T,  U^T = (beta R)^T T^T,  S'^T = exp(G_C) S^T + (exp(G_C - G) U)^T K,
// has its left operand in this warp's registers (the result of the one before
// it: an accumulator's registers are a left operand's) and its right operand
// in shared memory, the same for all warps.  So the chain of dependent
// products, which bounds the kernel, crosses no barrier and no memory.
//
// Each such warp has a partner on the same 16 columns that does what the chain
// does not wait for: the loads of the next chunk, the outputs
//     O^T = scale exp(G) S^T Q^T + U^T P^T
// from the S and U that the chain left in shared memory, and in training their
// way to memory for the backward pass.
#include "delta_common.cuh"

namespace ps {

namespace {

template <typename T, int KP, int NW>
struct ChainSmem {
    static constexpr int NP = Planes<T>::NP;
    static constexpr int VB = 16 * NW;
    static constexpr int kKP = kChunk * KP * 2, kVP = kChunk * VB * 2;
    // one stage
    static constexpr int kK = 0, kQ = NP * kKP, kV = 2 * NP * kKP, kT = kV + NP * kVP;
    static constexpr int kP = kT + 2 * (int)kSquare, kScal = kP + 2 * (int)kSquare;
    static constexpr int kStage = kScal + 1024;   // exp(G), exp(G_C - G), beta; stages 1024 bytes apart
    static constexpr int kStages = NP == 1 ? 2 : 1;
    // for each pair of warps: images of S and U, rows of outputs
    static constexpr int kS = 0, kU = 2 * 16 * KP * 2, kOut = kU + 2 * 16 * kChunk * 2;
    static constexpr int kWarp = kOut + (sizeof(T) == 2 ? kChunk * 16 * 2 : 0);
    static constexpr int kBytes = kStages * kStage + NW * kWarp;
    static_assert(kStage % 1024 == 0 && kWarp % 128 == 0 && kBytes <= 227 * 1024, "images are aligned and fit");
};

}  // namespace

template <typename T, int KP, int NW>
__global__ void __launch_bounds__(NW * 64) delta_chain_kernel(const DeltaArgs a) {
    using M = ChainSmem<T, KP, NW>;
    constexpr int NP = M::NP, VB = M::VB, NT = NW * 32, KT = KP / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % NW;
    const bool helper = threadIdx.x >= NT;
    const int blocks = (a.s.v + VB - 1) / VB, rep = a.s.hv / a.s.hk;
    const int vb = (int)(blockIdx.x % blocks);
    const int head = (int)(blockIdx.x / blocks % a.s.hv);
    const long long seq = blockIdx.x / blocks / a.s.hv;
    const Span sp = span_of(a.s, seq);
    const int v0 = vb * VB, vw = v0 + 16 * warp;   // this CTA's and this pair's first column
    const bool idle = vw >= a.s.v;                 // no column of this pair exists
    const int r8 = lane >> 2, c2 = 2 * (lane & 3);
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, a.train != 0);
    const long long chunks = (sp.len + kChunk - 1) / kChunk;
    const uint32_t own = base + M::kStages * M::kStage + warp * M::kWarp;
    const int s_ready = 1 + warp, u_ready = 1 + NW + warp;

    if (helper) {
        const unsigned char *ownp = smem + M::kStages * M::kStage + warp * M::kWarp;
        const int tid = threadIdx.x - NT;
        auto load = [&](long long c, int stage) {
            const uint32_t st = base + stage * M::kStage;
            const int rows = (int)min((long long)kChunk, sp.len - c * kChunk);
            const unsigned char *w = a.ws + (size_t)((sp.slot + c) * a.s.hv + head) * lay.stride;
            const unsigned char *kq = a.kq + (size_t)((sp.slot + c) * a.s.hk + head / rep) * kq_stride(a.s.k, NP);
            load_image<2 * NP * M::kKP, NT>(st + M::kK, kq, tid);
            load_image<4 * (int)kSquare, NT>(st + M::kT, w + lay.t, tid);
            load_image<3 * kChunk * 4, NT>(st + M::kScal, w + lay.scal, tid);
            load_tile<T, VB>(st + M::kV, M::kVP, row_ptr<T>(a.v, sp, seq, c * kChunk, head) + v0, a.v.tok, rows,
                             a.s.v - v0, a.vec_v != 0, tid, NT);
            cp_async_commit();
        };
        if (chunks > 0) load(0, 0);
        for (long long c = 0; c < chunks; ++c) {
            const int stage = M::kStages == 2 ? (int)(c & 1) : 0;
            cp_async_wait<0>();
            __syncthreads();
            if (M::kStages == 2 && c + 1 < chunks) load(c + 1, stage ^ 1);
            const uint32_t st = base + stage * M::kStage;
            const float *scal = reinterpret_cast<const float *>(smem + stage * M::kStage + M::kScal);
            if (!idle) {
                unsigned char *w = a.ws + (size_t)((sp.slot + c) * a.s.hv + head) * lay.stride;
                const int rows = (int)min((long long)kChunk, sp.len - c * kChunk);
                float o[8][4];
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
                await(s_ready);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) load_a<KP * 2>(f[h], own + M::kS + h * 16 * KP * 2, 0, 16 * kt, lane);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        uint32_t b[4][4];
#pragma unroll
                        for (int np = 0; np < 4; ++np) load_b<KP * 2>(b[np], st + M::kQ + p * M::kKP, 16 * np, 16 * kt, lane);
#pragma unroll
                        for (int h = 0; h + p < 2; ++h)
#pragma unroll
                            for (int np = 0; np < 4; ++np) {
                                mma_bf16(o[2 * np], f[h], b[np][0], b[np][1]);
                                mma_bf16(o[2 * np + 1], f[h], b[np][2], b[np][3]);
                            }
                    }
                }
                const size_t srow = (size_t)pad_v(a.s.v) * KP * 2, urow = (size_t)pad_v(a.s.v) * kChunk * 2;
                if (a.train)   // the state at the chunk's start
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        store_image<16 * KP * 2>(w + lay.s + p * srow + (size_t)vw * KP * 2, ownp + M::kS + p * 16 * KP * 2, lane);
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float2 eg = *reinterpret_cast<const float2 *>(scal + 8 * n + c2);
                    o[n][0] *= a.s.scale * eg.x; o[n][1] *= a.s.scale * eg.y;
                    o[n][2] *= a.s.scale * eg.x; o[n][3] *= a.s.scale * eg.y;
                }
                await(u_ready);
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {   // P is lower triangular
                    uint32_t f[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) load_a<128>(f[h], own + M::kU + h * 16 * kChunk * 2, 0, 16 * kt, lane);
#pragma unroll
                    for (int np = kt; np < 4; ++np) {
                        uint32_t ph[4], pl[4];
                        load_b<128>(ph, st + M::kP, 16 * np, 16 * kt, lane);
                        load_b<128>(pl, st + M::kP + (uint32_t)kSquare, 16 * np, 16 * kt, lane);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            mma_bf16(o[2 * np], f[h], ph[0], ph[1]);
                            mma_bf16(o[2 * np + 1], f[h], ph[2], ph[3]);
                        }
                        mma_bf16(o[2 * np], f[0], pl[0], pl[1]);
                        mma_bf16(o[2 * np + 1], f[0], pl[2], pl[3]);
                    }
                }
                if (a.train)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        store_image<16 * kChunk * 2>(w + lay.u + p * urow + (size_t)vw * kChunk * 2,
                                                     ownp + M::kU + p * 16 * kChunk * 2, lane);
                // O^T in registers, rows of 16 columns in memory
                T *out = static_cast<T *>(a.o) + ((size_t)(sp.first + c * kChunk) * a.s.hv + head) * a.s.v + vw;
                const size_t ostride = (size_t)a.s.hv * a.s.v;
                const bool whole = vw + 16 <= a.s.v && (a.s.v & 7) == 0 && (reinterpret_cast<uintptr_t>(a.o) & 15) == 0;
                if (sizeof(T) == 2 && whole) {
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int np = 0; np < 4; ++np) {
                            const int row = 16 * np + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
                            stsm4_t(own + M::kOut + row * 32 + half * 16, pack2<T>(o[2 * np][0], o[2 * np][1]),
                                    pack2<T>(o[2 * np][2], o[2 * np][3]), pack2<T>(o[2 * np + 1][0], o[2 * np + 1][1]),
                                    pack2<T>(o[2 * np + 1][2], o[2 * np + 1][3]));
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = i * 16 + (lane >> 1);
                            if (row < rows)
                                *reinterpret_cast<uint4 *>(out + row * ostride + (lane & 1) * 8) =
                                    *reinterpret_cast<const uint4 *>(ownp + M::kOut + row * 32 + (lane & 1) * 16);
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = 8 * n + c2 + (e & 1), v = r8 + 8 * (e >> 1);
                            if (tok < rows && vw + v < a.s.v) out[tok * ostride + v] = from_f32<T>(o[n][e]);
                        }
                }
                __syncwarp();
            }
            if (M::kStages == 1) {
                __syncthreads();
                if (c + 1 < chunks) load(c + 1, 0);
            }
        }
        return;
    }

    float s[2 * KT][4];   // S^T: rows vw + r8 (+8), columns 8 n + c2 (+1)
    const size_t state = (size_t)(seq * a.s.hv + head) * a.s.k * a.s.v;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 8 * n + c2 + (e & 1), v = vw + r8 + 8 * (e >> 1);
            s[n][e] = a.h0 != nullptr && k < a.s.k && v < a.s.v ? a.h0[state + (size_t)k * a.s.v + v] : 0.f;
        }
    for (long long c = 0; c < chunks; ++c) {
        const int stage = M::kStages == 2 ? (int)(c & 1) : 0;
        __syncthreads();
        if (!idle) {
            const uint32_t st = base + stage * M::kStage;
            const float *scal = reinterpret_cast<const float *>(smem + stage * M::kStage + M::kScal);
            // X^T = S^T K^T: tile n is tokens 8 n..
            float x[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                uint32_t f[2][4];
                split_tiles(s[2 * kt], s[2 * kt + 1], f);
                const uint32_t at = img<KP * 2>(own + M::kS, lane & 15, 2 * kt + (lane >> 4));
                stsm4(at, f[0][0], f[0][1], f[0][2], f[0][3]);
                stsm4(at + 16 * KP * 2, f[1][0], f[1][1], f[1][2], f[1][3]);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    uint32_t b[4][4];
#pragma unroll
                    for (int np = 0; np < 4; ++np) load_b<KP * 2>(b[np], st + M::kK + p * M::kKP, 16 * np, 16 * kt, lane);
#pragma unroll
                    for (int h = 0; h + p < 2; ++h)
#pragma unroll
                        for (int np = 0; np < 4; ++np) {
                            mma_bf16(x[2 * np], f[h], b[np][0], b[np][1]);
                            mma_bf16(x[2 * np + 1], f[h], b[np][2], b[np][3]);
                        }
                }
            }
            announce(s_ready);

            // beta R as left operands, and U^T = (beta R)^T T^T; T is lower triangular
            float u[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) u[n][e] = 0.f;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t f[NP][4], r[2][4];
#pragma unroll
                for (int p = 0; p < NP; ++p) load_a_t<VB * 2>(f[p], st + M::kV + p * M::kVP, 16 * kt, 16 * warp, lane);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = 2 * kt + (q >> 1), tok = 8 * n + c2;
                    const float2 eg = *reinterpret_cast<const float2 *>(scal + tok);
                    const float2 be = *reinterpret_cast<const float2 *>(scal + 128 + tok);
                    float y0 = bf16_low(f[0][q]), y1 = bf16_high(f[0][q]);
                    if constexpr (NP == 2) { y0 += bf16_low(f[1][q]); y1 += bf16_high(f[1][q]); }
                    y0 = be.x * (y0 - eg.x * x[n][2 * (q & 1)]);
                    y1 = be.y * (y1 - eg.y * x[n][2 * (q & 1) + 1]);
                    split2(y0, y1, r[0][q], r[1][q]);
                }
                uint32_t th[4][4], tl[4][4];
#pragma unroll
                for (int np = kt; np < 4; ++np) {
                    load_b<128>(th[np], st + M::kT, 16 * np, 16 * kt, lane);
                    load_b<128>(tl[np], st + M::kT + (uint32_t)kSquare, 16 * np, 16 * kt, lane);
                }
#pragma unroll
                for (int h = 0; h < 3; ++h)
#pragma unroll
                    for (int np = kt; np < 4; ++np) {
                        const uint32_t(&b)[4] = h == 2 ? tl[np] : th[np];
                        mma_bf16(u[2 * np], r[h & 1], b[0], b[1]);
                        mma_bf16(u[2 * np + 1], r[h & 1], b[2], b[3]);
                    }
            }

            // the state: S^T = exp(G_C) S^T + (exp(G_C - G) U)^T K; exp(G_C) is the last token's
            const float eall = scal[kChunk - 1];
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] *= eall;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t f[2][4];
                split_tiles(u[2 * kt], u[2 * kt + 1], f);
                const uint32_t at = img<128>(own + M::kU, lane & 15, 2 * kt + (lane >> 4));
                stsm4(at, f[0][0], f[0][1], f[0][2], f[0][3]);
                stsm4(at + 16 * kChunk * 2, f[1][0], f[1][1], f[1][2], f[1][3]);
            }
            announce(u_ready);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t f[2][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = 2 * kt + (q >> 1);
                    const float2 el = *reinterpret_cast<const float2 *>(scal + 64 + 8 * n + c2);
                    split2(el.x * u[n][2 * (q & 1)], el.y * u[n][2 * (q & 1) + 1], f[0][q], f[1][q]);
                }
#pragma unroll
                for (int nb = 0; nb < KT; nb += 4)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        uint32_t b[4][4];
#pragma unroll
                        for (int np = 0; np < 4; ++np)
                            load_b_t<KP * 2>(b[np], st + M::kK + p * M::kKP, 16 * kt, 16 * (nb + np), lane);
#pragma unroll
                        for (int h = 0; h + p < 2; ++h)
#pragma unroll
                            for (int np = 0; np < 4; ++np) {
                                mma_bf16(s[2 * (nb + np)], f[h], b[np][0], b[np][1]);
                                mma_bf16(s[2 * (nb + np) + 1], f[h], b[np][2], b[np][3]);
                            }
                    }
            }
        }
        if (M::kStages == 1) __syncthreads();
    }

    if (a.ht != nullptr) {
#pragma unroll
        for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 8 * n + c2 + (e & 1), v = vw + r8 + 8 * (e >> 1);
                if (k < a.s.k && v < a.s.v) a.ht[state + (size_t)k * a.s.v + v] = s[n][e];
            }
    }
}

namespace {

template <typename T, int KP, int NW>
cudaError_t chain(const DeltaArgs &a, cudaStream_t s) {
    using M = ChainSmem<T, KP, NW>;
    cudaError_t e = cudaFuncSetAttribute(delta_chain_kernel<T, KP, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kBytes);
    if (e != cudaSuccess) return e;
    const long long ctas = a.s.seqs * a.s.hv * ((a.s.v + M::VB - 1) / M::VB);
    delta_chain_kernel<T, KP, NW><<<(unsigned)ctas, NW * 64, M::kBytes, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t chain_for(const DeltaArgs &a, cudaStream_t s) {
    return a.s.k <= 64 ? chain<T, 64, 4>(a, s) : chain<T, 128, 4>(a, s);
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
