// delta_step.cu -- the gated delta rule for the next token or few, on states
// in a pool of pages (notation in delta_common.cuh).
//
// Bound by memory: a token reads and writes its K x V f32 state once (128 KiB
// at 128 x 128) and does 7 K V operations on it.  A CTA holds one head's state,
// or a block of its columns, in registers: all loads are in flight at once, and
// all tokens of the call run before the state goes back.  k^T S and q^T S are
// summed in one pass over the decayed state, because
//     q^T (S + k u^T) = q^T S + (q.k) u,
// so a token costs one exchange between the warps.
#include "delta_common.cuh"

namespace ps {

namespace {

constexpr int kStepThreads = 256, kStepWarps = kStepThreads / 32;
constexpr int kStepTokens = 8;   // tokens whose q and k are kept in shared memory at a time

__device__ __forceinline__ float4 shfl_add(float4 x, int d) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, d);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, d);
    x.z += __shfl_xor_sync(0xffffffffu, x.z, d);
    x.w += __shfl_xor_sync(0xffffffffu, x.w, d);
    return x;
}
__device__ __forceinline__ void fma4(float4 &d, float a, const float4 &b) {
    d.x += a * b.x; d.y += a * b.y; d.z += a * b.z; d.w += a * b.w;
}

}  // namespace

// VT columns of the state per CTA: VT / 4 lanes hold a row's columns, four each.
template <typename T, int KP, int VT>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaStepArgs a, const int vec4) {
    constexpr int LPR = VT / 4, GROUPS = kStepThreads / LPR, ROWS = KP / GROUPS;
    __shared__ float sk[kStepTokens][KP], sq[kStepTokens][KP];
    __shared__ float sa[kStepTokens], sb[kStepTokens], sqk[kStepTokens];
    __shared__ float4 sum_k[2][kStepWarps][LPR], sum_q[2][kStepWarps][LPR];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (a.v + VT - 1) / VT;
    const int vb = (int)(blockIdx.x % blocks), head = (int)(blockIdx.x / blocks % a.hv);
    const long long seq = blockIdx.x / blocks / a.hv;
    const int col = tid % LPR, group = tid / LPR, c0 = vb * VT + 4 * col, head_k = head / (a.hv / a.hk);

    const long long page = a.slots ? a.slots[seq] : seq;
    int count = a.lengths ? a.lengths[seq] : a.t;
    count = count < 0 ? 0 : count > a.t ? a.t : count;
    if (page < 0 || page >= a.pages) count = 0;
    T *out = static_cast<T *>(a.o) + ((size_t)seq * a.t * a.hv + head) * a.v;
    const size_t ostride = (size_t)a.hv * a.v;
    if (count < a.t)   // outputs of tokens that do not count
        for (int i = tid; i < (a.t - count) * VT; i += kStepThreads)
            if (vb * VT + i % VT < a.v) out[(count + i / VT) * ostride + vb * VT + i % VT] = from_f32<T>(0.f);
    if (count == 0) return;

    float4 S[ROWS];
    float *state = a.state + ((size_t)page * a.hv + head) * a.k * a.v;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int k = group + r * GROUPS;
        S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < a.k) {
            const float *p = state + (size_t)k * a.v + c0;
            if (vec4) {
                if (c0 < a.v) S[r] = __ldcs(reinterpret_cast<const float4 *>(p));
            } else {
                if (c0 < a.v) S[r].x = p[0];
                if (c0 + 1 < a.v) S[r].y = p[1];
                if (c0 + 2 < a.v) S[r].z = p[2];
                if (c0 + 3 < a.v) S[r].w = p[3];
            }
        }
    }

    const Span none{};
    for (int t0 = 0; t0 < count; t0 += kStepTokens) {
        const int nt = min(kStepTokens, count - t0);
        if (t0) __syncthreads();
        for (int i = tid; i < nt * KP; i += kStepThreads) {
            const int t = i / KP, k = i % KP;
            sk[t][k] = k < a.k ? to_f32<T>(row_ptr<T>(a.kk, none, seq, t0 + t, head_k)[k]) : 0.f;
            sq[t][k] = k < a.k ? to_f32<T>(row_ptr<T>(a.q, none, seq, t0 + t, head_k)[k]) : 0.f;
        }
        if (tid < nt) {
            const float g = row_ptr<float>(a.g, none, seq, t0 + tid, head)[0];
            sa[tid] = g <= -87.f ? 0.f : expf(g);
            sb[tid] = a.beta_f32 ? row_ptr<float>(a.beta, none, seq, t0 + tid, head)[0]
                                 : to_f32<T>(row_ptr<T>(a.beta, none, seq, t0 + tid, head)[0]);
        }
        __syncthreads();
        if (warp < nt) {   // q.k of token `warp` (at most eight tokens, eight warps); read after the next barrier
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < KP / 32; ++i) d += sk[warp][lane + 32 * i] * sq[warp][lane + 32 * i];
#pragma unroll
            for (int m = 16; m; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
            if (lane == 0) sqk[warp] = d;
        }
        for (int t = 0; t < nt; ++t) {
            const T *vp = row_ptr<T>(a.vv, none, seq, t0 + t, head);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c0 < a.v) v.x = to_f32<T>(vp[c0]);
            if (c0 + 1 < a.v) v.y = to_f32<T>(vp[c0 + 1]);
            if (c0 + 2 < a.v) v.z = to_f32<T>(vp[c0 + 2]);
            if (c0 + 3 < a.v) v.w = to_f32<T>(vp[c0 + 3]);
            const float decay = sa[t], beta = sb[t];
            float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                // a forgotten state is 0 even where it held an infinity or a NaN
                if (decay == 0.f) S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                S[r].x *= decay; S[r].y *= decay; S[r].z *= decay; S[r].w *= decay;
                fma4(pk, sk[t][group + r * GROUPS], S[r]);
                fma4(pq, sq[t][group + r * GROUPS], S[r]);
            }
#pragma unroll
            for (int d = LPR; d < 32; d <<= 1) { pk = shfl_add(pk, d); pq = shfl_add(pq, d); }
            if (lane < LPR) { sum_k[t & 1][warp][lane] = pk; sum_q[t & 1][warp][lane] = pq; }
            __syncthreads();
            pk = sum_k[t & 1][0][col];
            pq = sum_q[t & 1][0][col];
#pragma unroll
            for (int w = 1; w < kStepWarps; ++w) {
                fma4(pk, 1.f, sum_k[t & 1][w][col]);
                fma4(pq, 1.f, sum_q[t & 1][w][col]);
            }
            const float4 u = make_float4(beta * (v.x - pk.x), beta * (v.y - pk.y), beta * (v.z - pk.z), beta * (v.w - pk.w));
#pragma unroll
            for (int r = 0; r < ROWS; ++r) fma4(S[r], sk[t][group + r * GROUPS], u);
            if (group == 0) {
                fma4(pq, sqk[t], u);
                T *op = out + (t0 + t) * ostride + c0;
                if (c0 < a.v) op[0] = from_f32<T>(a.scale * pq.x);
                if (c0 + 1 < a.v) op[1] = from_f32<T>(a.scale * pq.y);
                if (c0 + 2 < a.v) op[2] = from_f32<T>(a.scale * pq.z);
                if (c0 + 3 < a.v) op[3] = from_f32<T>(a.scale * pq.w);
            }
        }
    }

#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int k = group + r * GROUPS;
        if (k < a.k) {
            float *p = state + (size_t)k * a.v + c0;
            if (vec4) {
                if (c0 < a.v) __stcs(reinterpret_cast<float4 *>(p), S[r]);
            } else {
                if (c0 < a.v) p[0] = S[r].x;
                if (c0 + 1 < a.v) p[1] = S[r].y;
                if (c0 + 2 < a.v) p[2] = S[r].z;
                if (c0 + 3 < a.v) p[3] = S[r].w;
            }
        }
    }
}

namespace {

template <typename T, int KP, int VT>
cudaError_t step(const DeltaStepArgs &a, cudaStream_t s) {
    const int vec4 = a.v % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
    const long long ctas = a.seqs * a.hv * ((a.v + VT - 1) / VT);
    delta_step_kernel<T, KP, VT><<<(unsigned)ctas, kStepThreads, 0, s>>>(a, vec4);
    return cudaGetLastError();
}
template <typename T, int KP>
cudaError_t step_for(const DeltaStepArgs &a, cudaStream_t s) {
    // Whole rows of up to 128 columns where there are CTAs enough for the machine, narrower blocks
    // where there are not: more of the state's bytes are then in flight at once.
    const long long heads = a.seqs * a.hv;
    if (a.v <= 32 || heads * ((a.v + 63) / 64) < 2 * 152) return step<T, KP, 32>(a, s);
    if (a.v <= 64 || heads * ((a.v + 127) / 128) < 2 * 152) return step<T, KP, 64>(a, s);
    return step<T, KP, 128>(a, s);
}
template <typename T>
cudaError_t step_type(const DeltaStepArgs &a, cudaStream_t s) {
    return a.k <= 64 ? step_for<T, 64>(a, s) : step_for<T, 128>(a, s);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepArgs &a, int type, cudaStream_t s) {
    switch (type) {
    case PS_REAL_BF16: return step_type<__nv_bfloat16>(a, s);
    case PS_REAL_F16: return step_type<__half>(a, s);
    default: return step_type<float>(a, s);
    }
}

}  // namespace ps
