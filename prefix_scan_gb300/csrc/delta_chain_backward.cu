// delta_chain_backward.cu -- the gradients of the gated delta rule's states,
// chunk before chunk, and of its values (notation in delta_common.cuh).  With
// dS' the gradient of the state at a chunk's end, each chunk takes
//     Y  = diag(exp(G_C - G)) K dS'                      (what U did to the state)
//     dU = T^T (Y + P^T dO)
//     dR = diag(beta) dU = dV
//     dS = exp(G_C) dS' + scale (exp(G) Q)^T dO - (exp(G) K)^T dR
// and leaves dS' and dR for the gradients of q, k and g (delta_gradients.cu),
// and the sums over this warp's columns of U dU and of U Y.
//
// As in the forward chain, a warp owns 16 columns and keeps dS'^T and every
// left operand in registers.
#include "delta_common.cuh"

namespace ps {

namespace {

template <typename T, int KP, int NW>
struct BackSmem {
    static constexpr int NP = Planes<T>::NP;
    static constexpr int VB = 16 * NW;
    static constexpr int kKP = kChunk * KP * 2, kVP = kChunk * VB * 2, kUP = VB * kChunk * 2;
    static constexpr int kK = 0, kQ = NP * kKP, kO = 2 * NP * kKP, kT = kO + NP * kVP;
    static constexpr int kP = kT + 2 * (int)kSquare, kU = kP + 2 * (int)kSquare, kScal = kU + 2 * kUP;
    static constexpr int kStage = kScal + 3 * kChunk * 4 + 256;
    static constexpr int kStages = NP == 1 ? 2 : 1;
    // per warp: dS' as it leaves, later dR and after it the rows of dV
    static constexpr int kOut = 2 * 16 * kChunk * 2;
    static constexpr int kWarp = 2 * 16 * KP * 2 > kOut + 2048 ? 2 * 16 * KP * 2 : kOut + 2048;
    static constexpr int kBytes = kStages * kStage + NW * kWarp;
    static_assert(kStage % 1024 == 0 && kWarp % 128 == 0 && kBytes <= 227 * 1024, "images are aligned and fit");
};

}  // namespace

template <typename T, int KP, int NW>
__global__ void __launch_bounds__(NW * 32) delta_chain_backward_kernel(const DeltaArgs a) {
    using M = BackSmem<T, KP, NW>;
    constexpr int NP = M::NP, VB = M::VB, NT = NW * 32, KT = KP / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (a.s.v + VB - 1) / VB, rep = a.s.hv / a.s.hk;
    const int vb = (int)(blockIdx.x % blocks);
    const int head = (int)(blockIdx.x / blocks % a.s.hv);
    const long long seq = blockIdx.x / blocks / a.s.hv;
    const Span sp = span_of(a.s, seq);
    const int v0 = vb * VB, vw = v0 + 16 * warp;
    const int r8 = lane >> 2, c2 = 2 * (lane & 3);
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, true);
    const long long chunks = (sp.len + kChunk - 1) / kChunk;
    const int vpad = pad_v(a.s.v);
    const uint32_t own = base + M::kStages * M::kStage + warp * M::kWarp;
    const unsigned char *ownp = smem + M::kStages * M::kStage + warp * M::kWarp;

    float ds[2 * KT][4];   // dS'^T: rows vw + r8 (+8), columns 8 n + c2 (+1)
    const size_t state = (size_t)(seq * a.s.hv + head) * a.s.k * a.s.v;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 8 * n + c2 + (e & 1), v = vw + r8 + 8 * (e >> 1);
            ds[n][e] = a.dht != nullptr && k < a.s.k && v < a.s.v ? a.dht[state + (size_t)k * a.s.v + v] : 0.f;
        }

    auto load = [&](long long c, int stage) {
        const uint32_t st = base + stage * M::kStage;
        const long long t0 = c * kChunk;
        const int rows = (int)min((long long)kChunk, sp.len - t0);
        const unsigned char *w = a.ws + (size_t)((sp.slot + c) * a.s.hv + head) * lay.stride;
        const int urows = min(VB, vpad - v0);
        load_image(st + M::kT, w + lay.t, 4 * (int)kSquare, tid, NT);
        load_image(st + M::kScal, w + lay.scal, 3 * kChunk * 4, tid, NT);
#pragma unroll
        for (int p = 0; p < 2; ++p)
            load_image(st + M::kU + p * M::kUP, w + lay.u + (size_t)p * vpad * kChunk * 2 + (size_t)v0 * kChunk * 2,
                       urows * kChunk * 2, tid, NT);
        load_tile<T, KP>(st + M::kK, M::kKP, row_ptr<T>(a.k, sp, seq, t0, head / rep), a.k.tok, rows, a.s.k,
                         a.vec_qk != 0, tid, NT);
        load_tile<T, VB>(st + M::kO, M::kVP, row_ptr<T>(a.dout, sp, seq, t0, head) + v0, a.dout.tok, rows, a.s.v - v0,
                         a.vec_do != 0, tid, NT);
        load_tile<T, KP>(st + M::kQ, M::kKP, row_ptr<T>(a.q, sp, seq, t0, head / rep), a.q.tok, rows, a.s.k,
                         a.vec_qk != 0, tid, NT);
        cp_async_commit();
    };
    if (chunks > 0) load(chunks - 1, 0);

    for (long long c = chunks - 1; c >= 0; --c) {
        const int stage = M::kStages == 2 ? (int)((chunks - 1 - c) & 1) : 0;
        cp_async_wait<0>();
        __syncthreads();
        if (M::kStages == 2 && c > 0) load(c - 1, stage ^ 1);
        const uint32_t st = base + stage * M::kStage;
        const float *scal = reinterpret_cast<const float *>(smem + stage * M::kStage + M::kScal);
        unsigned char *w = a.ws + (size_t)((sp.slot + c) * a.s.hv + head) * lay.stride;
        const int rows = (int)min((long long)kChunk, sp.len - c * kChunk);

        // Y^T = dS'^T K^T, not yet times exp(G_C - G)
        float y[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[n][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            uint32_t f[2][4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                split2(ds[2 * kt + (q >> 1)][2 * (q & 1)], ds[2 * kt + (q >> 1)][2 * (q & 1) + 1], f[0][q], f[1][q]);
            const uint32_t at = img<KP * 2>(own, lane & 15, 2 * kt + (lane >> 4));
            stsm4(at, f[0][0], f[0][1], f[0][2], f[0][3]);
            stsm4(at + 16 * KP * 2, f[1][0], f[1][1], f[1][2], f[1][3]);
#pragma unroll
            for (int np = 0; np < 4; ++np)
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    uint32_t b[4];
                    load_b<KP * 2>(b, st + M::kK + p * M::kKP, 16 * np, 16 * kt, lane);
#pragma unroll
                    for (int h = 0; h + p < 2; ++h) {
                        mma_bf16(y[2 * np], f[h], b[0], b[1]);
                        mma_bf16(y[2 * np + 1], f[h], b[2], b[3]);
                    }
                }
        }
        __syncwarp();
        if (vw < a.s.v) {
            const size_t plane = (size_t)vpad * KP * 2;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < 16 * KP * 2 / 512; ++i)
                    *reinterpret_cast<uint4 *>(w + lay.ds + p * plane + (size_t)vw * KP * 2 + i * 512 + lane * 16) =
                        *reinterpret_cast<const uint4 *>(ownp + p * 16 * KP * 2 + i * 512 + lane * 16);
        }
        __syncwarp();

        // Y, and the sums of U Y over the columns
        float sum_b[8][2], sum_y[8][2];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t uh[4], ul[4];
            load_a<128>(uh, st + M::kU, 16 * warp, 16 * np, lane);
            load_a<128>(ul, st + M::kU + M::kUP, 16 * warp, 16 * np, lane);
            if (vw >= a.s.v)   // rows past the values: nothing was loaded
#pragma unroll
                for (int q = 0; q < 4; ++q) uh[q] = ul[q] = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * np + h;
                const float2 el = *reinterpret_cast<const float2 *>(scal + 64 + 8 * n + c2);
                y[n][0] *= el.x; y[n][1] *= el.y; y[n][2] *= el.x; y[n][3] *= el.y;
                sum_y[n][0] = (bf16_low(uh[2 * h]) + bf16_low(ul[2 * h])) * y[n][0] +
                              (bf16_low(uh[2 * h + 1]) + bf16_low(ul[2 * h + 1])) * y[n][2];
                sum_y[n][1] = (bf16_high(uh[2 * h]) + bf16_high(ul[2 * h])) * y[n][1] +
                              (bf16_high(uh[2 * h + 1]) + bf16_high(ul[2 * h + 1])) * y[n][3];
            }
        }
        // + (P^T dO)^T = dO^T P: token i at or after token j
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t f[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) load_a_t<VB * 2>(f[p], st + M::kO + p * M::kVP, 16 * kt, 16 * warp, lane);
#pragma unroll
            for (int np = 0; np <= kt; ++np) {
                uint32_t ph[4], pl[4];
                load_b_t<128>(ph, st + M::kP, 16 * kt, 16 * np, lane);
                load_b_t<128>(pl, st + M::kP + (uint32_t)kSquare, 16 * kt, 16 * np, lane);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    mma_bf16(y[2 * np], f[p], ph[0], ph[1]);
                    mma_bf16(y[2 * np + 1], f[p], ph[2], ph[3]);
                }
                mma_bf16(y[2 * np], f[0], pl[0], pl[1]);
                mma_bf16(y[2 * np + 1], f[0], pl[2], pl[3]);
            }
        }
        // dU^T = (..)^T T
        float du[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) du[n][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t f[2][4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                split2(y[2 * kt + (q >> 1)][2 * (q & 1)], y[2 * kt + (q >> 1)][2 * (q & 1) + 1], f[0][q], f[1][q]);
#pragma unroll
            for (int np = 0; np <= kt; ++np) {
                uint32_t th[4], tl[4];
                load_b_t<128>(th, st + M::kT, 16 * kt, 16 * np, lane);
                load_b_t<128>(tl, st + M::kT + (uint32_t)kSquare, 16 * kt, 16 * np, lane);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma_bf16(du[2 * np], f[h], th[0], th[1]);
                    mma_bf16(du[2 * np + 1], f[h], th[2], th[3]);
                }
                mma_bf16(du[2 * np], f[0], tl[0], tl[1]);
                mma_bf16(du[2 * np + 1], f[0], tl[2], tl[3]);
            }
        }
        // the sums of U dU, and dR = beta dU
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t uh[4], ul[4];
            load_a<128>(uh, st + M::kU, 16 * warp, 16 * np, lane);
            load_a<128>(ul, st + M::kU + M::kUP, 16 * warp, 16 * np, lane);
            if (vw >= a.s.v)
#pragma unroll
                for (int q = 0; q < 4; ++q) uh[q] = ul[q] = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * np + h;
                const float2 be = *reinterpret_cast<const float2 *>(scal + 128 + 8 * n + c2);
                sum_b[n][0] = (bf16_low(uh[2 * h]) + bf16_low(ul[2 * h])) * du[n][0] +
                              (bf16_low(uh[2 * h + 1]) + bf16_low(ul[2 * h + 1])) * du[n][2];
                sum_b[n][1] = (bf16_high(uh[2 * h]) + bf16_high(ul[2 * h])) * du[n][1] +
                              (bf16_high(uh[2 * h + 1]) + bf16_high(ul[2 * h + 1])) * du[n][3];
                du[n][0] *= be.x; du[n][1] *= be.y; du[n][2] *= be.x; du[n][3] *= be.y;
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) {
                    sum_b[n][e] += __shfl_xor_sync(0xffffffffu, sum_b[n][e], m);
                    sum_y[n][e] += __shfl_xor_sync(0xffffffffu, sum_y[n][e], m);
                }
        if (lane < 4 && vw < a.s.v) {
            float *part = a.part + ((size_t)((sp.slot + c) * a.s.hv + head) * ((a.s.v + 15) / 16) + vw / 16) * 2 * kChunk;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                *reinterpret_cast<float2 *>(part + 8 * n + c2) = make_float2(sum_b[n][0], sum_b[n][1]);
                *reinterpret_cast<float2 *>(part + kChunk + 8 * n + c2) = make_float2(sum_y[n][0], sum_y[n][1]);
            }
        }

        // the state's gradient at the chunk's start
        const float eall = scal[kChunk - 1];
#pragma unroll
        for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) ds[n][e] *= eall;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t fo[NP][4], f[2][4], g[2][4], r[2][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) load_a_t<VB * 2>(fo[p], st + M::kO + p * M::kVP, 16 * kt, 16 * warp, lane);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = 2 * kt + (q >> 1);
                const float2 eg = *reinterpret_cast<const float2 *>(scal + 8 * n + c2);
                float x0 = bf16_low(fo[0][q]), x1 = bf16_high(fo[0][q]);
                if constexpr (NP == 2) { x0 += bf16_low(fo[1][q]); x1 += bf16_high(fo[1][q]); }
                split2(a.s.scale * eg.x * x0, a.s.scale * eg.y * x1, f[0][q], f[1][q]);
                const float d0 = du[n][2 * (q & 1)], d1 = du[n][2 * (q & 1) + 1];
                split2(d0, d1, r[0][q], r[1][q]);
                split2(-eg.x * d0, -eg.y * d1, g[0][q], g[1][q]);
            }
            const uint32_t at = img<128>(own, lane & 15, 2 * kt + (lane >> 4));
            stsm4(at, r[0][0], r[0][1], r[0][2], r[0][3]);
            stsm4(at + 16 * 128, r[1][0], r[1][1], r[1][2], r[1][3]);
#pragma unroll
            for (int np = 0; np < KT; ++np)
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    uint32_t bq[4], bk[4];
                    load_b_t<KP * 2>(bq, st + M::kQ + p * M::kKP, 16 * kt, 16 * np, lane);
                    load_b_t<KP * 2>(bk, st + M::kK + p * M::kKP, 16 * kt, 16 * np, lane);
#pragma unroll
                    for (int h = 0; h + p < 2; ++h) {
                        mma_bf16(ds[2 * np], f[h], bq[0], bq[1]);
                        mma_bf16(ds[2 * np + 1], f[h], bq[2], bq[3]);
                        mma_bf16(ds[2 * np], g[h], bk[0], bk[1]);
                        mma_bf16(ds[2 * np + 1], g[h], bk[2], bk[3]);
                    }
                }
        }
        __syncwarp();
        if (vw < a.s.v) {
            const size_t plane = (size_t)vpad * kChunk * 2;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(w + lay.dr + p * plane + (size_t)vw * 128 + i * 512 + lane * 16) =
                        *reinterpret_cast<const uint4 *>(ownp + p * 16 * 128 + i * 512 + lane * 16);
        }

        // dV = dR
        T *out = static_cast<T *>(a.dv) + ((size_t)(sp.first + c * kChunk) * a.s.hv + head) * a.s.v + vw;
        const size_t ostride = (size_t)a.s.hv * a.s.v;
        const bool whole = vw + 16 <= a.s.v && (a.s.v & 7) == 0 && (reinterpret_cast<uintptr_t>(a.dv) & 15) == 0;
        if (sizeof(T) == 2 && whole) {
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    const int row = 16 * np + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
                    stsm4_t(own + M::kOut + row * 32 + half * 16, pack2<T>(du[2 * np][0], du[2 * np][1]),
                            pack2<T>(du[2 * np][2], du[2 * np][3]), pack2<T>(du[2 * np + 1][0], du[2 * np + 1][1]),
                            pack2<T>(du[2 * np + 1][2], du[2 * np + 1][3]));
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
                    if (tok < rows && vw + v < a.s.v) out[tok * ostride + v] = from_f32<T>(du[n][e]);
                }
        }
        __syncwarp();
        if (M::kStages == 1) {
            __syncthreads();
            if (c > 0) load(c - 1, 0);
        }
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
    delta_chain_backward_kernel<T, KP, 4><<<(unsigned)ctas, 128, M::kBytes, s>>>(a);
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
