// delta_chain_backward.cu -- the gradients of the gated delta rule's states,
// chunk before chunk, and of its values (notation in delta_common.cuh).  With
// dS' the gradient of the state at a chunk's end, each chunk takes
//     Y  = diag(exp(G_C - G)) K dS' + P^T dO             (the gradient of U)
//     dU = T^T Y,   dR = diag(beta) dU = dV
//     dS = exp(G_C) dS' + scale (exp(G) Q)^T dO - (exp(G) K)^T dR
// and leaves dS' and dU for the gradients of the other inputs
// (delta_gradients.cu).
//
// As in the forward chain, a warp owns 16 columns and keeps dS'^T and every
// left operand of the dependent products in registers.  Its partner works one
// chunk ahead on what does not depend on the states, P^T dO and scale (exp(G)
// Q)^T dO, holds both in registers until the chain has taken the last ones from
// shared memory, loads the next chunk, and takes dS', dU and dV to memory.
#include "delta_common.cuh"

namespace ps {

namespace {

template <typename T, int KP, int NW>
struct BackSmem {
    static constexpr int NP = Planes<T>::NP;
    static constexpr int VB = 16 * NW;
    static constexpr int kKP = kChunk * KP * 2, kVP = kChunk * VB * 2;
    // a stage of what the chain reads; the partners' tiles; exp(G), exp(G_C - G), beta of two chunks
    static constexpr int kK = 0, kT = NP * kKP, kStage = kT + 2 * (int)kSquare;
    static constexpr int kStages = NP == 1 ? 2 : 1;
    static constexpr int kQ = kStages * kStage, kP = kQ + NP * kKP, kO = kP + 2 * (int)kSquare;
    static constexpr int kScal = kO + NP * kVP, kPairs = kScal + 2 * 1024;
    // for each pair of warps: P^T dO and (exp(G) Q)^T dO as accumulators, images of dS' and dU, rows of dV
    static constexpr int kA1 = 0, kA2 = kA1 + 16 * kChunk * 4, kDS = kA2 + 16 * KP * 4, kDU = kDS + 2 * 16 * KP * 2;
    static constexpr int kOut = kDU + 2 * 16 * kChunk * 2;
    static constexpr int kWarp = kOut + (sizeof(T) == 2 ? kChunk * 16 * 2 : 0);
    static constexpr int kBytes = kPairs + NW * kWarp;
    static_assert(kStage % 1024 == 0 && kWarp % 128 == 0 && kBytes <= 227 * 1024, "images are aligned and fit");
};

}  // namespace

template <typename T, int KP, int NW>
__global__ void __launch_bounds__(NW * 64) delta_chain_backward_kernel(const DeltaArgs a) {
    using M = BackSmem<T, KP, NW>;
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
    const int v0 = vb * VB, vw = v0 + 16 * warp;
    const bool idle = vw >= a.s.v;
    const int r8 = lane >> 2, c2 = 2 * (lane & 3);
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, true);
    const long long chunks = (sp.len + kChunk - 1) / kChunk;
    const uint32_t own = base + M::kPairs + warp * M::kWarp;
    unsigned char *ownp = smem + M::kPairs + warp * M::kWarp;
    float4 *a1p = reinterpret_cast<float4 *>(ownp + M::kA1) + lane, *a2p = reinterpret_cast<float4 *>(ownp + M::kA2) + lane;
    const int s_ready = 1 + warp, r_ready = 1 + NW + warp, a_ready = 1 + 2 * NW + warp;

    if (helper) {
        const int tid = threadIdx.x - NT;
        auto chunk_ws = [&](long long c) { return a.ws + (size_t)((sp.slot + c) * a.s.hv + head) * lay.stride; };
        auto chunk_kq = [&](long long c) {
            return a.kq + (size_t)((sp.slot + c) * a.s.hk + head / rep) * kq_stride(a.s.k, NP);
        };
        auto load_chain = [&](long long c, int stage) {
            load_image<NP * M::kKP, NT>(base + stage * M::kStage + M::kK, chunk_kq(c), tid);
            load_image<2 * (int)kSquare, NT>(base + stage * M::kStage + M::kT, chunk_ws(c) + lay.t, tid);
        };
        auto load_own = [&](long long c) {
            const int rows = (int)min((long long)kChunk, sp.len - c * kChunk);
            load_image<NP * M::kKP, NT>(base + M::kQ, chunk_kq(c) + NP * M::kKP, tid);
            load_image<2 * (int)kSquare, NT>(base + M::kP, chunk_ws(c) + lay.p, tid);
            load_image<3 * kChunk * 4, NT>(base + M::kScal + (uint32_t)(c & 1) * 1024, chunk_ws(c) + lay.scal, tid);
            load_tile<T, VB>(base + M::kO, M::kVP, row_ptr<T>(a.dout, sp, seq, c * kChunk, head) + v0, a.dout.tok, rows,
                             a.s.v - v0, a.vec_do != 0, tid, NT);
        };
        float a1[8][4], a2[2 * KT][4];
        // the tiles of chunk c have been loaded by all partners: P^T dO and scale (exp(G) Q)^T dO, transposed
        auto ahead = [&](long long c) {
            const float *scal = reinterpret_cast<const float *>(smem + M::kScal + (c & 1) * 1024);
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) a1[n][e] = 0.f;
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) a2[n][e] = 0.f;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t f[NP][4], g[2][4];
#pragma unroll
                for (int p = 0; p < NP; ++p) load_a_t<VB * 2>(f[p], base + M::kO + p * M::kVP, 16 * kt, 16 * warp, lane);
#pragma unroll
                for (int np = 0; np <= kt; ++np) {   // token kt at or after token np
                    uint32_t ph[4], pl[4];
                    load_b_t<128>(ph, base + M::kP, 16 * kt, 16 * np, lane);
                    load_b_t<128>(pl, base + M::kP + (uint32_t)kSquare, 16 * kt, 16 * np, lane);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        mma_bf16(a1[2 * np], f[p], ph[0], ph[1]);
                        mma_bf16(a1[2 * np + 1], f[p], ph[2], ph[3]);
                    }
                    mma_bf16(a1[2 * np], f[0], pl[0], pl[1]);
                    mma_bf16(a1[2 * np + 1], f[0], pl[2], pl[3]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 eg = *reinterpret_cast<const float2 *>(scal + 8 * (2 * kt + (q >> 1)) + c2);
                    float x0 = bf16_low(f[0][q]), x1 = bf16_high(f[0][q]);
                    if constexpr (NP == 2) { x0 += bf16_low(f[1][q]); x1 += bf16_high(f[1][q]); }
                    split2(a.s.scale * eg.x * x0, a.s.scale * eg.y * x1, g[0][q], g[1][q]);
                }
#pragma unroll
                for (int np = 0; np < KT; ++np)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        uint32_t b[4];
                        load_b_t<KP * 2>(b, base + M::kQ + p * M::kKP, 16 * kt, 16 * np, lane);
#pragma unroll
                        for (int h = 0; h + p < 2; ++h) {
                            mma_bf16(a2[2 * np], g[h], b[0], b[1]);
                            mma_bf16(a2[2 * np + 1], g[h], b[2], b[3]);
                        }
                    }
            }
        };
        auto partners = [&] { asm volatile("bar.sync %0, %1;" :: "r"(1 + 3 * NW), "n"(NT) : "memory"); };

        if (chunks > 0) {
            load_chain(chunks - 1, 0);
            load_own(chunks - 1);
            cp_async_commit();
            cp_async_wait<0>();
            partners();
            ahead(chunks - 1);
        }
        for (long long c = chunks - 1; c >= 0; --c) {
            const int stage = M::kStages == 2 ? (int)((chunks - 1 - c) & 1) : 0;
            __syncthreads();   // the chain is done with chunk c + 1; this chunk's stage is loaded; all partners are done with theirs
            if (!idle) {
#pragma unroll
                for (int n = 0; n < 8; ++n) a1p[n * 32] = make_float4(a1[n][0], a1[n][1], a1[n][2], a1[n][3]);
#pragma unroll
                for (int n = 0; n < 2 * KT; ++n) a2p[n * 32] = make_float4(a2[n][0], a2[n][1], a2[n][2], a2[n][3]);
                announce(a_ready);
            }
            if (c > 0) {
                if (M::kStages == 2) load_chain(c - 1, stage ^ 1);
                load_own(c - 1);
                cp_async_commit();
            }
            unsigned char *w = chunk_ws(c);
            const int rows = (int)min((long long)kChunk, sp.len - c * kChunk), vpad = pad_v(a.s.v);
            if (!idle) {
                await(s_ready);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    store_image<16 * KP * 2>(w + lay.ds + ((size_t)p * vpad + vw) * KP * 2, ownp + M::kDS + p * 16 * KP * 2, lane);
            }
            if (c > 0) {
                cp_async_wait<0>();
                partners();
                ahead(c - 1);
            }
            if (!idle) {
                await(r_ready);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    store_image<16 * kChunk * 2>(w + lay.du + ((size_t)p * vpad + vw) * kChunk * 2,
                                                 ownp + M::kDU + p * 16 * kChunk * 2, lane);
                // dV = dR: rows of 16 columns (f32 rows go out from the chain)
                T *out = static_cast<T *>(a.dv) + ((size_t)(sp.first + c * kChunk) * a.s.hv + head) * a.s.v + vw;
                const size_t ostride = (size_t)a.s.hv * a.s.v;
                if constexpr (sizeof(T) == 2) {
                    if (vw + 16 <= a.s.v && (a.s.v & 7) == 0 && (reinterpret_cast<uintptr_t>(a.dv) & 15) == 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = i * 16 + (lane >> 1);
                            if (row < rows)
                                *reinterpret_cast<uint4 *>(out + row * ostride + (lane & 1) * 8) =
                                    *reinterpret_cast<const uint4 *>(ownp + M::kOut + row * 32 + (lane & 1) * 16);
                        }
                    } else {
                        for (int i = lane; i < rows * 16; i += 32)
                            if (vw + (i & 15) < a.s.v)
                                out[(i >> 4) * ostride + (i & 15)] = reinterpret_cast<const T *>(ownp + M::kOut)[i];
                    }
                }
            }
            if (M::kStages == 1) {
                __syncthreads();
                if (c > 0) {
                    load_chain(c - 1, 0);
                    cp_async_commit();
                    cp_async_wait<0>();
                }
            }
        }
        return;
    }

    float ds[2 * KT][4];   // dS'^T: rows vw + r8 (+8), columns 8 n + c2 (+1)
    const size_t state = (size_t)(seq * a.s.hv + head) * a.s.k * a.s.v;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 8 * n + c2 + (e & 1), v = vw + r8 + 8 * (e >> 1);
            ds[n][e] = a.dht != nullptr && k < a.s.k && v < a.s.v ? a.dht[state + (size_t)k * a.s.v + v] : 0.f;
        }
    for (long long c = chunks - 1; c >= 0; --c) {
        const int stage = M::kStages == 2 ? (int)((chunks - 1 - c) & 1) : 0;
        __syncthreads();
        if (!idle) {
            const uint32_t st = base + stage * M::kStage;
            const float *scal = reinterpret_cast<const float *>(smem + M::kScal + (c & 1) * 1024);
            // Y^T: first dS'^T K^T
            float y[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[n][e] = 0.f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                uint32_t f[2][4];
                split_tiles(ds[2 * kt], ds[2 * kt + 1], f);
                const uint32_t at = img<KP * 2>(own + M::kDS, lane & 15, 2 * kt + (lane >> 4));
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
                            mma_bf16(y[2 * np], f[h], b[np][0], b[np][1]);
                            mma_bf16(y[2 * np + 1], f[h], b[np][2], b[np][3]);
                        }
                }
            }
            announce(s_ready);
            await(a_ready);
            float du[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const float2 el = *reinterpret_cast<const float2 *>(scal + 64 + 8 * n + c2);
                const float4 p = a1p[n * 32];
                y[n][0] = el.x * y[n][0] + p.x; y[n][1] = el.y * y[n][1] + p.y;
                y[n][2] = el.x * y[n][2] + p.z; y[n][3] = el.y * y[n][3] + p.w;
#pragma unroll
                for (int e = 0; e < 4; ++e) du[n][e] = 0.f;
            }
            // dU^T = Y^T T: row kt at or after column np
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t f[2][4], th[4][4], tl[4][4];
                split_tiles(y[2 * kt], y[2 * kt + 1], f);
#pragma unroll
                for (int np = 0; np <= kt; ++np) {
                    load_b_t<128>(th[np], st + M::kT, 16 * kt, 16 * np, lane);
                    load_b_t<128>(tl[np], st + M::kT + (uint32_t)kSquare, 16 * kt, 16 * np, lane);
                }
#pragma unroll
                for (int h = 0; h < 3; ++h)
#pragma unroll
                    for (int np = 0; np <= kt; ++np) {
                        const uint32_t(&b)[4] = h == 2 ? tl[np] : th[np];
                        mma_bf16(du[2 * np], f[h & 1], b[0], b[1]);
                        mma_bf16(du[2 * np + 1], f[h & 1], b[2], b[3]);
                    }
            }
            // dU and dV = dR leave; the state's gradient at the chunk's start
            const float eall = scal[kChunk - 1];
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n) {
                const float4 p = a2p[n * 32];
                ds[n][0] = eall * ds[n][0] + p.x; ds[n][1] = eall * ds[n][1] + p.y;
                ds[n][2] = eall * ds[n][2] + p.z; ds[n][3] = eall * ds[n][3] + p.w;
            }
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t r[2][4];
                split_tiles(du[2 * kt], du[2 * kt + 1], r);
#pragma unroll
                for (int t = 0; t < 2; ++t) {   // dU is now dR
                    const int n = 2 * kt + t;
                    const float2 be = *reinterpret_cast<const float2 *>(scal + 128 + 8 * n + c2);
                    du[n][0] *= be.x; du[n][1] *= be.y; du[n][2] *= be.x; du[n][3] *= be.y;
                }
                const uint32_t at = img<128>(own + M::kDU, lane & 15, 2 * kt + (lane >> 4));
                stsm4(at, r[0][0], r[0][1], r[0][2], r[0][3]);
                stsm4(at + 16 * kChunk * 2, r[1][0], r[1][1], r[1][2], r[1][3]);
                if constexpr (sizeof(T) == 2) {
                    const int row = 16 * kt + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
                    stsm4_t(own + M::kOut + row * 32 + half * 16, pack2<T>(du[2 * kt][0], du[2 * kt][1]),
                            pack2<T>(du[2 * kt][2], du[2 * kt][3]), pack2<T>(du[2 * kt + 1][0], du[2 * kt + 1][1]),
                            pack2<T>(du[2 * kt + 1][2], du[2 * kt + 1][3]));
                }
            }
            announce(r_ready);
            if constexpr (sizeof(T) == 4) {
                const int rows = (int)min((long long)kChunk, sp.len - c * kChunk);
                T *out = static_cast<T *>(a.dv) + ((size_t)(sp.first + c * kChunk) * a.s.hv + head) * a.s.v + vw;
                const size_t ostride = (size_t)a.s.hv * a.s.v;
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = 8 * n + c2 + (e & 1), v = r8 + 8 * (e >> 1);
                        if (tok < rows && vw + v < a.s.v) out[tok * ostride + v] = du[n][e];
                    }
            }
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t g[2][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = 2 * kt + (q >> 1);
                    const float2 eg = *reinterpret_cast<const float2 *>(scal + 8 * n + c2);
                    split2(-eg.x * du[n][2 * (q & 1)], -eg.y * du[n][2 * (q & 1) + 1], g[0][q], g[1][q]);
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
                                mma_bf16(ds[2 * (nb + np)], g[h], b[np][0], b[np][1]);
                                mma_bf16(ds[2 * (nb + np) + 1], g[h], b[np][2], b[np][3]);
                            }
                    }
            }
        }
        if (M::kStages == 1) __syncthreads();
    }

    if (a.dh0 != nullptr) {
#pragma unroll
        for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 8 * n + c2 + (e & 1), v = vw + r8 + 8 * (e >> 1);
                if (k < a.s.k && v < a.s.v) a.dh0[state + (size_t)k * a.s.v + v] = ds[n][e];
            }
    }
}

namespace {

template <typename T, int KP>
cudaError_t chain_back(const DeltaArgs &a, cudaStream_t s) {
    using M = BackSmem<T, KP, 4>;
    cudaError_t e = cudaFuncSetAttribute(delta_chain_backward_kernel<T, KP, 4>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, M::kBytes);
    if (e != cudaSuccess) return e;
    const long long ctas = a.s.seqs * a.s.hv * ((a.s.v + M::VB - 1) / M::VB);
    delta_chain_backward_kernel<T, KP, 4><<<(unsigned)ctas, 256, M::kBytes, s>>>(a);
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
