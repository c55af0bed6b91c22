// delta_gradients.cu -- the gradients of the gated delta rule's queries, keys,
// gates and log decays, all chunks at once, from what the two chains left
// (notation in delta_common.cuh and delta_chain_backward.cu).  Per chunk and
// value head, with dP = dO U^T and dN = -dR U^T (j < i only):
//     dQ = scale diag(exp(G)) dO S^T + (scale D dP) K
//     dK = (scale D dP)^T Q + (D dN) K + (D dN)^T K - diag(exp(G)) dR S^T + diag(exp(G_C - G)) U dS'^T
//     dbeta_j = (dU_j . U_j) / beta_j          (U = beta (what was missing))
//     dg_t = sum_{j < t <= i} Z_ij + sum_{i >= t} a_i + sum_{j < t} b_j + exp(G_C) <S, dS'>
// where Z = P dP + N dN (element by element), a_i = exp(G_i) (scale q_i . S dO_i -
// k_i . S dR_i) and b_j = exp(G_C - G_j) k_j . dS' U_j: every term that the decay of token t scales,
// each counted once, so nothing cancels.
//
// One CTA per chunk and key head: gradients of a shared key head are sums over its
// value heads in their order, in registers, without atomics.
#include "delta_common.cuh"

namespace ps {

namespace {

constexpr int kGradThreads = 512;   // sixteen warps: 16 rows and a quarter of the columns each
constexpr int kGradV = 32;          // values taken at a time
constexpr int kSlice = kGradV * 128;   // bytes of 64 columns of a block of the state
constexpr int kZStride = kChunk + 1;

template <int NP, int KP>
struct GradSmem {
    static constexpr int kKQ = (KP / 64) * kHalf, kSP = kGradV * KP * 2, kUP = kGradV * kChunk * 2, kOP = kChunk * 128;   // planes
    static constexpr int kK = 0, kQ = kChunk * 128;
    // a stage: S, dS', U, dU, dO of the values taken at a time
    static constexpr int kS = 0, kDS = kS + 2 * kSP, kU = kDS + 2 * kSP, kDU = kU + 2 * kUP, kO = kDU + 2 * kUP, kStage = kO + NP * kOP;
    static constexpr int kStages = NP == 1 ? 2 : 1, kFirst = NP * kKQ;
    static constexpr int kF1 = kFirst + kStages * kStage, kF2 = kF1 + 2 * (int)kSquare, kZ = kF2 + 2 * (int)kSquare;
    static constexpr int kScal = kZ + kChunk * kZStride * 4, kMore = kScal + 2 * 6 * kChunk * 4;   // scalars of two heads
    static constexpr int kBytes = kMore + (4 * kChunk + 4 * kChunk + 4 * kChunk + kChunk + 16) * 4;
    static_assert(kBytes <= 227 * 1024, "too much shared memory");
};

}  // namespace

template <typename T, int KP>
__global__ void __launch_bounds__(kGradThreads, 1) delta_gradients_kernel(const DeltaArgs a) {
    constexpr int NP = Planes<T>::NP, NQ = KP / 32, KH = KP / 64;   // NQ: column tiles of a quarter of a row
    using M = GradSmem<NP, KP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    float *Z = reinterpret_cast<float *>(smem + M::kZ);
    float *dots = reinterpret_cast<float *>(smem + M::kMore);   // [4 quarters of the columns][64] of a_i
    float *dotb = dots + 4 * kChunk;                            // the same of b_j
    float *run = dotb + 4 * kChunk;                             // [4 quarters of the rows][64] column sums of Z
    float *diag = run + 4 * kChunk;                             // [64] dU_j . U_j
    float *inner = diag + kChunk;                               // <S, dS'> by warps
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int strip = warp & 3, quarter = warp >> 2;   // rows 16 strip.., this quarter of the columns
    const int r8 = lane >> 2, c2 = 2 * (lane & 3), i0 = 16 * strip + r8;
    const long long slot = blockIdx.x;
    const int head_k = blockIdx.y, rep = a.s.hv / a.s.hk;

    const long long seq = seq_of_slot(a.s, slot);
    if (seq < 0) return;
    const Span sp = span_of(a.s, seq);
    const long long t0 = (slot - sp.slot) * kChunk;
    const int rows = (int)min((long long)kChunk, sp.len - t0);
    const ChunkLayout lay = chunk_layout(a.s.k, a.s.v, true);
    const int vpad = (a.s.v + 15) / 16 * 16;

    load_image<NP * M::kKQ, kGradThreads>(base + M::kK, a.kq + (size_t)(slot * a.s.hk + head_k) * kq_stride(a.s.k, NP), tid);

    // all value heads' values, kGradV at a time, in one sequence of stages
    const int slices = (vpad + kGradV - 1) / kGradV;
    auto load = [&](int it) {
        const int head = head_k * rep + it / slices, v0 = it % slices * kGradV, vr = min(kGradV, vpad - v0);
        const int vb = v0 / kBlockV, vi = v0 % kBlockV;
        const uint32_t st = base + M::kFirst + it % M::kStages * M::kStage;
        const unsigned char *w = a.ws + (size_t)(slot * a.s.hv + head) * lay.stride;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int h = 0; h < KH; ++h) {
                const size_t from = ((size_t)(vb * 2 + p) * KH + h) * kHalf + vi * 128;
                load_part<kSlice, kGradThreads>(st + M::kS + p * M::kSP + h * kSlice, w + lay.s + from, vr * 128, tid);
                load_part<kSlice, kGradThreads>(st + M::kDS + p * M::kSP + h * kSlice, w + lay.ds + from, vr * 128, tid);
            }
            const size_t from = (size_t)(vb * 2 + p) * kHalf + vi * 128;
            load_part<M::kUP, kGradThreads>(st + M::kU + p * M::kUP, w + lay.u + from, vr * 128, tid);
            load_part<M::kUP, kGradThreads>(st + M::kDU + p * M::kUP, w + lay.du + from, vr * 128, tid);
        }
        load_tile<T, kGradV>(st + M::kO, M::kOP, row_ptr<T>(a.dout, sp, seq, t0, head) + v0, a.dout.tok, rows, a.s.v - v0,
                             a.vec_do != 0, tid, kGradThreads);
        if (v0 == 0) load_image<6 * kChunk * 4, kGradThreads>(base + M::kScal + (it / slices & 1) * 6 * kChunk * 4, w + lay.scal, tid);
        cp_async_commit();
    };
    load(0);

    float dq[NQ][4], dk[NQ][4];   // rows i0 (+8), columns 8 (quarter NQ + n) + c2 (+1)
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[n][e] = dk[n][e] = 0.f;

    for (int hr = 0; hr < rep; ++hr) {
        const int head = head_k * rep + hr;
        const unsigned char *w = a.ws + (size_t)(slot * a.s.hv + head) * lay.stride;
        const float *scal = reinterpret_cast<const float *>(smem + M::kScal + (hr & 1) * 6 * kChunk * 4);
        float pa[2][4], na[2][4];                     // dP and dU U^T: columns 16 quarter + 8 n..
        float x1[NQ][4], x2[NQ][4], x3[NQ][4];        // dO S^T, dU S^T, U dS'^T
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) pa[n][e] = na[n][e] = 0.f;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x1[n][e] = x2[n][e] = x3[n][e] = 0.f;
        float prod = 0.f;   // this thread's part of <S, dS'>

        for (int s = 0; s < slices; ++s) {
            const int it = hr * slices + s, vr = min(kGradV, vpad - s * kGradV);
            const uint32_t st = base + M::kFirst + it % M::kStages * M::kStage;
            cp_async_wait<0>();
            __syncthreads();
            if (M::kStages == 2 && it + 1 < rep * slices) load(it + 1);

            const unsigned char *sp8 = smem + (st - base);
            for (int i = tid; i < kGradV * KP / 8; i += kGradThreads) {   // the same place in all four images
                if (i % (kGradV * 8) >= vr * 8) continue;   // not loaded
                const uint4 *sv = reinterpret_cast<const uint4 *>(sp8 + M::kS) + i;
                const uint4 *dv = reinterpret_cast<const uint4 *>(sp8 + M::kDS) + i;
                const uint4 sh = sv[0], sl = sv[M::kSP / 16], dh = dv[0], dl = dv[M::kSP / 16];
                const uint32_t *shp = &sh.x, *slp = &sl.x, *dhp = &dh.x, *dlp = &dl.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    prod += (bf16_low(shp[j]) + bf16_low(slp[j])) * (bf16_low(dhp[j]) + bf16_low(dlp[j]));
                    prod += (bf16_high(shp[j]) + bf16_high(slp[j])) * (bf16_high(dhp[j]) + bf16_high(dlp[j]));
                }
            }
            for (int kt = 0; kt < vr / 16; ++kt) {
                {   // dO: dP and dO S^T
                    uint32_t f[NP][4];
#pragma unroll
                    for (int p = 0; p < NP; ++p) load_a(f[p], st + M::kO + p * M::kOP, 16 * strip, 16 * kt, lane);
                    if (quarter <= strip)   // columns at or before the rows
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            uint32_t b[4];
                            load_b_t(b, st + M::kU + p * M::kUP, 16 * kt, 16 * quarter, lane);
#pragma unroll
                            for (int h = 0; h < NP && h + p < 2; ++h) {
                                mma_bf16(pa[0], f[h], b[0], b[1]);
                                mma_bf16(pa[1], f[h], b[2], b[3]);
                            }
                        }
#pragma unroll
                    for (int np = 0; np < NQ / 2; ++np)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            uint32_t b[4];
                            load_b_t<kSlice>(b, st + M::kS + p * M::kSP, 16 * kt, 8 * quarter * NQ + 16 * np, lane);
#pragma unroll
                            for (int h = 0; h < NP && h + p < 2; ++h) {
                                mma_bf16(x1[2 * np], f[h], b[0], b[1]);
                                mma_bf16(x1[2 * np + 1], f[h], b[2], b[3]);
                            }
                        }
                }
                {   // dU: dU U^T and dU S^T
                    uint32_t f[2][4];
#pragma unroll
                    for (int p = 0; p < 2; ++p) load_a_t(f[p], st + M::kDU + p * M::kUP, 16 * kt, 16 * strip, lane);
                    if (quarter <= strip)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            uint32_t b[4];
                            load_b_t(b, st + M::kU + p * M::kUP, 16 * kt, 16 * quarter, lane);
#pragma unroll
                            for (int h = 0; h + p < 2; ++h) {
                                mma_bf16(na[0], f[h], b[0], b[1]);
                                mma_bf16(na[1], f[h], b[2], b[3]);
                            }
                        }
#pragma unroll
                    for (int np = 0; np < NQ / 2; ++np)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            uint32_t b[4];
                            load_b_t<kSlice>(b, st + M::kS + p * M::kSP, 16 * kt, 8 * quarter * NQ + 16 * np, lane);
#pragma unroll
                            for (int h = 0; h + p < 2; ++h) {
                                mma_bf16(x2[2 * np], f[h], b[0], b[1]);
                                mma_bf16(x2[2 * np + 1], f[h], b[2], b[3]);
                            }
                        }
                }
                {   // U: U dS'^T
                    uint32_t f[2][4];
#pragma unroll
                    for (int p = 0; p < 2; ++p) load_a_t(f[p], st + M::kU + p * M::kUP, 16 * kt, 16 * strip, lane);
#pragma unroll
                    for (int np = 0; np < NQ / 2; ++np)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            uint32_t b[4];
                            load_b_t<kSlice>(b, st + M::kDS + p * M::kSP, 16 * kt, 8 * quarter * NQ + 16 * np, lane);
#pragma unroll
                            for (int h = 0; h + p < 2; ++h) {
                                mma_bf16(x3[2 * np], f[h], b[0], b[1]);
                                mma_bf16(x3[2 * np + 1], f[h], b[2], b[3]);
                            }
                        }
                }
            }
            if (M::kStages == 1) {
                __syncthreads();
                if (it + 1 < rep * slices) load(it + 1);
            }
        }

        // <S, dS'>, the parts of dQ and dK that go through the states, a_i and b_j
#pragma unroll
        for (int m = 16; m; m >>= 1) prod += __shfl_xor_sync(0xffffffffu, prod, m);
        if (lane == 0) inner[warp] = prod;
        float dot[2] = {0.f, 0.f}, dob[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int col = 8 * (quarter * NQ + n) + c2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // rows i0, i0 + 8
                const int i = i0 + 8 * e;
                const uint32_t at = img(0, i, col >> 3) + (col & 7) * 2;
                uint32_t kw = *reinterpret_cast<const uint32_t *>(smem + M::kK + at);
                uint32_t qw = *reinterpret_cast<const uint32_t *>(smem + M::kQ + at);
                float k0 = bf16_low(kw), k1 = bf16_high(kw), q0 = bf16_low(qw), q1 = bf16_high(qw);
                if constexpr (NP == 2) {
                    kw = *reinterpret_cast<const uint32_t *>(smem + M::kK + M::kKQ + at);
                    qw = *reinterpret_cast<const uint32_t *>(smem + M::kQ + M::kKQ + at);
                    k0 += bf16_low(kw); k1 += bf16_high(kw); q0 += bf16_low(qw); q1 += bf16_high(qw);
                }
                const float eg = scal[i], el = scal[64 + i], sc = a.s.scale * eg, eb = eg * scal[128 + i];
                const float y0 = sc * x1[n][2 * e], y1 = sc * x1[n][2 * e + 1];
                const float z0 = eb * x2[n][2 * e], z1 = eb * x2[n][2 * e + 1];
                dot[e] += q0 * y0 + q1 * y1 - (k0 * z0 + k1 * z1);
                const float u0 = el * x3[n][2 * e], u1 = el * x3[n][2 * e + 1];
                dob[e] += k0 * u0 + k1 * u1;
                dq[n][2 * e] += y0;
                dq[n][2 * e + 1] += y1;
                dk[n][2 * e] += u0 - z0;
                dk[n][2 * e + 1] += u1 - z1;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            dot[e] += __shfl_xor_sync(0xffffffffu, dot[e], 1);
            dot[e] += __shfl_xor_sync(0xffffffffu, dot[e], 2);
            dob[e] += __shfl_xor_sync(0xffffffffu, dob[e], 1);
            dob[e] += __shfl_xor_sync(0xffffffffu, dob[e], 2);
            if ((lane & 3) == 0) {
                dots[quarter * kChunk + i0 + 8 * e] = dot[e];
                dotb[quarter * kChunk + i0 + 8 * e] = dob[e];
            }
        }
        // F1 = scale D dP, F2 = D dN as pairs, and Z
        {
            const int cb = 16 * quarter;   // first column of the block
            uint32_t f1h[4] = {0, 0, 0, 0}, f1l[4] = {0, 0, 0, 0}, f2h[4] = {0, 0, 0, 0}, f2l[4] = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = q >> 1, row = q & 1, i = i0 + 8 * row, j = cb + 8 * n + c2;
                float z0 = 0.f, z1 = 0.f;
                if (cb <= 16 * strip) {
                    const uint32_t at = img(0, i, j >> 3) + (j & 7) * 2;
                    const uint32_t ph = *reinterpret_cast<const uint32_t *>(w + lay.p + at);
                    const uint32_t pl = *reinterpret_cast<const uint32_t *>(w + lay.p + kSquare + at);
                    const uint32_t nh = *reinterpret_cast<const uint32_t *>(w + lay.n + at);
                    const uint32_t nl = *reinterpret_cast<const uint32_t *>(w + lay.n + kSquare + at);
                    float f1[2], f2[2], z[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = j + e;
                        const float dx = (scal[192 + i] - scal[192 + c]) + (scal[256 + i] - scal[256 + c]);
                        const float D = i >= c && scal[320 + i] == scal[320 + c] ? expf(dx) : 0.f;
                        const float dp = pa[n][2 * row + e], dn = -scal[128 + i] * na[n][2 * row + e];
                        if (i == c) diag[i] = na[n][2 * row + e];
                        const float pv = e ? bf16_high(ph) + bf16_high(pl) : bf16_low(ph) + bf16_low(pl);
                        const float nv = e ? bf16_high(nh) + bf16_high(nl) : bf16_low(nh) + bf16_low(nl);
                        f1[e] = i >= c ? a.s.scale * D * dp : 0.f;
                        f2[e] = i > c ? D * dn : 0.f;
                        z[e] = i > c ? pv * dp + nv * dn : 0.f;
                    }
                    split2(f1[0], f1[1], f1h[q], f1l[q]);
                    split2(f2[0], f2[1], f2h[q], f2l[q]);
                    z0 = z[0];
                    z1 = z[1];
                }
                Z[i * kZStride + j] = z0;
                Z[i * kZStride + j + 1] = z1;
            }
            const uint32_t at = img(0, 16 * strip + (lane & 15), (cb >> 3) + (lane >> 4));
            stsm4(base + M::kF1 + at, f1h[0], f1h[1], f1h[2], f1h[3]);
            stsm4(base + M::kF1 + (uint32_t)kSquare + at, f1l[0], f1l[1], f1l[2], f1l[3]);
            stsm4(base + M::kF2 + at, f2h[0], f2h[1], f2h[2], f2h[3]);
            stsm4(base + M::kF2 + (uint32_t)kSquare + at, f2l[0], f2l[1], f2l[2], f2l[3]);
        }
        __syncthreads();

        // dQ += F1 K; dK += F1^T Q + F2 K + F2^T K
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t f1[2][4], f1t[2][4], f2[2][4];
            const bool down = kt <= strip, up = kt >= strip;   // tokens kt at or before / at or after the rows
            if (down)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    load_a(f1[p], base + M::kF1 + p * (uint32_t)kSquare, 16 * strip, 16 * kt, lane);
                    load_a(f2[p], base + M::kF2 + p * (uint32_t)kSquare, 16 * strip, 16 * kt, lane);
                }
            if (up)
#pragma unroll
                for (int p = 0; p < 2; ++p) load_a_t(f1t[p], base + M::kF1 + p * (uint32_t)kSquare, 16 * kt, 16 * strip, lane);
#pragma unroll
            for (int np = 0; np < NQ / 2; ++np)
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    uint32_t bk[4], bq[4];
                    load_b_t(bk, base + M::kK + p * M::kKQ, 16 * kt, 8 * quarter * NQ + 16 * np, lane);
                    load_b_t(bq, base + M::kQ + p * M::kKQ, 16 * kt, 8 * quarter * NQ + 16 * np, lane);
#pragma unroll
                    for (int h = 0; h + p < 2; ++h) {
                        if (down) {
                            mma_bf16(dq[2 * np], f1[h], bk[0], bk[1]);
                            mma_bf16(dq[2 * np + 1], f1[h], bk[2], bk[3]);
                            mma_bf16(dk[2 * np], f2[h], bk[0], bk[1]);
                            mma_bf16(dk[2 * np + 1], f2[h], bk[2], bk[3]);
                        }
                        if (up) {
                            mma_bf16(dk[2 * np], f1t[h], bq[0], bq[1]);
                            mma_bf16(dk[2 * np + 1], f1t[h], bq[2], bq[3]);
                        }
                    }
                }
            if (up) {
#pragma unroll
                for (int p = 0; p < 2; ++p) load_a_t(f1t[p], base + M::kF2 + p * (uint32_t)kSquare, 16 * kt, 16 * strip, lane);
#pragma unroll
                for (int np = 0; np < NQ / 2; ++np)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        uint32_t bk[4];
                        load_b_t(bk, base + M::kK + p * M::kKQ, 16 * kt, 8 * quarter * NQ + 16 * np, lane);
#pragma unroll
                        for (int h = 0; h + p < 2; ++h) {
                            mma_bf16(dk[2 * np], f1t[h], bk[0], bk[1]);
                            mma_bf16(dk[2 * np + 1], f1t[h], bk[2], bk[3]);
                        }
                    }
            }
        }

        // sum over i >= t of Z_ij within quarters of 16 rows, then with the quarters below
        if (tid < 256) {
            const int j = tid & 63, q = tid >> 6;
            float s = 0.f;
#pragma unroll
            for (int t = 15; t >= 0; --t) {
                s += Z[(16 * q + t) * kZStride + j];
                Z[(16 * q + t) * kZStride + j] = s;
            }
            run[q * kChunk + j] = s;
        }
        __syncthreads();
        {   // row t: sum over j < t (eight threads a row)
            const int t = tid >> 3, part = tid & 7;
            float s = 0.f;
            for (int j = part; j < t; j += 8) {
                s += Z[t * kZStride + j];
                for (int q = (t >> 4) + 1; q < 4; ++q) s += run[q * kChunk + j];
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            __syncthreads();
            if (part == 0) run[t] = s;
        }
        __syncthreads();
        if (warp == 0) {   // tokens 2 lane, 2 lane + 1
            float av[2], b[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                av[e] = (dots[t] + dots[kChunk + t]) + (dots[2 * kChunk + t] + dots[3 * kChunk + t]);
                b[e] = (dotb[t] + dotb[kChunk + t]) + (dotb[2 * kChunk + t] + dotb[3 * kChunk + t]);
            }
            float below = av[0] + av[1], above = b[0] + b[1];   // sums over i >= 2 lane, over j <= 2 lane + 1
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float x = __shfl_down_sync(0xffffffffu, below, d), y = __shfl_up_sync(0xffffffffu, above, d);
                if (lane + d < 32) below += x;
                if (lane >= d) above += y;
            }
            const float upto = __shfl_up_sync(0xffffffffu, above, 1);   // over j < 2 lane
            const float next = __shfl_down_sync(0xffffffffu, below, 1); // over i >= 2 lane + 2
            float c = 0.f;
#pragma unroll
            for (int i = 0; i < kGradThreads / 32; ++i) c += inner[i];
            c *= scal[kChunk - 1];
            const size_t at = ((size_t)sp.first + t0) * a.s.hv + head;
            const float before = lane ? upto : 0.f, after = lane < 31 ? next : 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                if (t < rows) {
                    // the decay of a token that forgets the state scales nothing
                    const bool forgets = scal[320 + t] != (t ? scal[319 + t] : 0.f);
                    const float s = run[t] + (e ? after + av[1] : below) + (e ? before + b[0] : before) + c;
                    a.dg[at + (size_t)t * a.s.hv] = forgets ? 0.f : s;
                    const float d = diag[t] / scal[128 + t];
                    if (a.beta_f32) static_cast<float *>(a.dbeta)[at + (size_t)t * a.s.hv] = d;
                    else static_cast<T *>(a.dbeta)[at + (size_t)t * a.s.hv] = from_f32<T>(d);
                }
            }
        }
        __syncthreads();
    }

    T *oq = static_cast<T *>(a.dq) + ((size_t)(sp.first + t0) * a.s.hk + head_k) * a.s.k;
    T *ok = static_cast<T *>(a.dk) + ((size_t)(sp.first + t0) * a.s.hk + head_k) * a.s.k;
    const size_t ostride = (size_t)a.s.hk * a.s.k;
    const bool pairs = sizeof(T) == 2 && (a.s.k & 1) == 0 &&
                       ((reinterpret_cast<uintptr_t>(a.dq) | reinterpret_cast<uintptr_t>(a.dk)) & 3) == 0;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + 8 * e, col = 8 * (quarter * NQ + n) + c2;
            if (i >= rows) continue;
            if (pairs) {
                if constexpr (sizeof(T) == 2) {
                    if (col < a.s.k) {
                        *reinterpret_cast<uint32_t *>(oq + i * ostride + col) = pack2<T>(dq[n][2 * e], dq[n][2 * e + 1]);
                        *reinterpret_cast<uint32_t *>(ok + i * ostride + col) = pack2<T>(dk[n][2 * e], dk[n][2 * e + 1]);
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (col + x < a.s.k) {
                        oq[i * ostride + col + x] = from_f32<T>(dq[n][2 * e + x]);
                        ok[i * ostride + col + x] = from_f32<T>(dk[n][2 * e + x]);
                    }
            }
        }
}

namespace {

template <typename T, int KP>
cudaError_t gradients(const DeltaArgs &a, cudaStream_t s) {
    constexpr int bytes = GradSmem<Planes<T>::NP, KP>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(delta_gradients_kernel<T, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    delta_gradients_kernel<T, KP><<<dim3((unsigned)a.slots, (unsigned)a.s.hk), kGradThreads, bytes, s>>>(a);
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
