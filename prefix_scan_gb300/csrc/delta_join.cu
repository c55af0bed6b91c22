// delta_join.cu -- the states at the starts of a long sequence's segments from
// the first pass's parts (DeltaArgs::seg): one segment after the other,
//     S_{s+1} = M_s S_s + B_s,       backward   dS_s = M_s^T dS_{s+1} + C_s.
// A CTA takes 16 values of one head.  Each step is a product of 16 x K by K x K
// numbers: the state in shared memory, M's images streamed in ahead, a quarter
// of the columns per warp.  It reads a segment's M (64 KiB at K = 128) per
// step and is bound by that latency, about as long as one chunk of the chain:
// 36 us for a 32768-token prompt in 19 segments, 8 heads.
#include "delta_common.cuh"

namespace ps {

namespace {

constexpr int kJoinThreads = 128, kJoinV = 16;

}  // namespace

template <int KP, bool BACK>
__global__ void __launch_bounds__(kJoinThreads) delta_join_kernel(const DeltaArgs a) {
    constexpr int KH = KP / 64, NQ = KP / 32, kM = 2 * KH * kHalf, kRow = KP + 4;   // NQ: column tiles of a warp
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    float *S = reinterpret_cast<float *>(smem + 2 * kM);   // [16 values][K], rows padded against bank conflicts
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r8 = lane >> 2, c2 = 2 * (lane & 3);
    const int blocks = (a.s.v + kJoinV - 1) / kJoinV, v0 = (int)(blockIdx.x % blocks) * kJoinV;
    const int head = (int)(blockIdx.x / blocks % a.s.hv);
    const long long seq = blockIdx.x / blocks / a.s.hv;
    const Span sp = span_of(a.s, seq);
    const long long seg0 = first_segment(a, seq), tokens = (long long)a.seg * kChunk;
    const int parts = (int)((sp.len + tokens - 1) / tokens);
    const size_t one_state = (size_t)a.s.k * a.s.v;
    if (parts < 3) return;
    // segments 1 .. parts - 2 have an M; forward in order, backward in the other
    const int steps = parts - 2;
    auto segment = [&](int i) { return BACK ? parts - 2 - i : 1 + i; };
    // the state that step i reads, and the part that it completes
    auto reads = [&](int i) { return a.seg_state + (size_t)((seg0 + segment(i) + (BACK ? 1 : 0)) * a.s.hv + head) * one_state; };
    auto completes = [&](int i) { return a.seg_state + (size_t)((seg0 + segment(i) + (BACK ? 0 : 1)) * a.s.hv + head) * one_state; };
    auto load = [&](int i) {
        load_image<kM, kJoinThreads>(base + (i & 1) * kM, a.seg_m + (size_t)((seg0 + segment(i)) * a.s.hv + head) * seg_m_bytes(a.s.k), tid);
        cp_async_commit();
    };
    load(0);
    {
        const float *s = reads(0);
        for (int i = tid; i < kJoinV * KP; i += kJoinThreads) {
            const int v = i % kJoinV, k = i / kJoinV;
            S[v * kRow + k] = k < a.s.k && v0 + v < a.s.v ? s[(size_t)k * a.s.v + v0 + v] : 0.f;
        }
    }
    for (int i = 0; i < steps; ++i) {
        float *to = completes(i);
        float acc[NQ][4];   // rows r8 (+8), columns 8 (warp NQ + n) + c2 (+1)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 8 * (warp * NQ + n) + c2 + (e & 1), v = v0 + r8 + 8 * (e >> 1);
                acc[n][e] = k < a.s.k && v < a.s.v ? to[(size_t)k * a.s.v + v] : 0.f;
            }
        if (i + 1 < steps) {
            load(i + 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        const uint32_t m = base + (i & 1) * kM;
#pragma unroll
        for (int kt = 0; kt < KP / 16; ++kt) {
            uint32_t f[2][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 x = *reinterpret_cast<const float2 *>(S + (r8 + 8 * (q & 1)) * kRow + 16 * kt + 8 * (q >> 1) + c2);
                split2(x.x, x.y, f[0][q], f[1][q]);   // for the product alone: what is added to and kept is f32
            }
#pragma unroll
            for (int np = 0; np < NQ / 2; ++np)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t b[4];
                    // M's image has row j, column k: forward the sum runs over j, backward over k
                    if constexpr (BACK) load_b(b, m + p * KH * kHalf, 8 * warp * NQ + 16 * np, 16 * kt, lane);
                    else load_b_t(b, m + p * KH * kHalf, 16 * kt, 8 * warp * NQ + 16 * np, lane);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma_bf16(acc[2 * np], f[h], b[0], b[1]);
                        mma_bf16(acc[2 * np + 1], f[h], b[2], b[3]);
                    }
                }
        }
        __syncthreads();   // S has been read, and M
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 8 * (warp * NQ + n) + c2 + (e & 1), v = v0 + r8 + 8 * (e >> 1);
                S[(r8 + 8 * (e >> 1)) * kRow + k] = acc[n][e];
                if (k < a.s.k && v < a.s.v) to[(size_t)k * a.s.v + v] = acc[n][e];
            }
    }
}

namespace {

template <int KP, bool BACK>
cudaError_t join(const DeltaArgs &a, cudaStream_t s) {
    constexpr int bytes = 2 * 2 * (KP / 64) * kHalf + kJoinV * (KP + 4) * 4;
    cudaError_t e = cudaFuncSetAttribute(delta_join_kernel<KP, BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long long ctas = a.s.seqs * a.s.hv * ((a.s.v + kJoinV - 1) / kJoinV);
    delta_join_kernel<KP, BACK><<<(unsigned)ctas, kJoinThreads, bytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_join(const DeltaArgs &a, bool backward, cudaStream_t s) {
    if (a.s.k <= 64) return backward ? join<64, true>(a, s) : join<64, false>(a, s);
    return backward ? join<128, true>(a, s) : join<128, false>(a, s);
}

}  // namespace ps
