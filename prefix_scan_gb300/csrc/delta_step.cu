// delta_step.cu -- the gated delta rule for the next token or few, on states
// in a pool of pages (notation in delta_common.cuh).
//
// Bound by memory: a token reads and writes its K x V f32 state once (128 KiB
// at 128 x 128) and does 7 K V operations on it, in f32; all tokens of the call
// run before the state goes back.  k^T S and q^T S are summed in one pass over
// the decayed state, because
//     q^T (S + k u^T) = q^T S + (q.k) u,
// so a token costs one exchange between the warps.
//
// With few heads, latency counts: a CTA holds a block of a head's columns in
// registers, all of its loads in flight at once (32 states of 128 x 128: 15 us with
// the call, which the host bounds).  With many, bandwidth does: whole states pass through
// a ring of bulk copies (8192 states of 128 x 128: 171 us, 6.33 TB/s; loads,
// sums and stores of a CTA in turn, at two or three CTAs an SM, reached 5.0-5.2).
#include "delta_tmem.cuh"

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
// exp(g), 0 where it leaves f32's normal range.
__device__ __forceinline__ float decay_of(float g) { return g <= -87.f ? 0.f : exp_rounded(g); }
__device__ __forceinline__ void fma4(float4 &d, float a, const float4 &b) {
    d.x += a * b.x; d.y += a * b.y; d.z += a * b.z; d.w += a * b.w;
}

}  // namespace

// VT columns of the state per CTA: VT / 4 lanes hold a row's columns, four each.
template <typename T, int KP, int VT>
__global__ void __launch_bounds__(kStepThreads, 3) delta_step_kernel(const DeltaStepArgs a, const int vec4) {
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
        for (long long i = tid; i < (long long)(a.t - count) * VT; i += kStepThreads)
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
    for (unsigned t0 = 0; t0 < (unsigned)count; t0 += kStepTokens) {
        const int nt = min(kStepTokens, count - (int)t0);
        if (t0) __syncthreads();
        for (int i = tid; i < nt * KP; i += kStepThreads) {
            const int t = i / KP, k = i % KP;
            sk[t][k] = k < a.k ? to_f32<T>(row_ptr<T>(a.kk, none, seq, t0 + t, head_k)[k]) : 0.f;
            sq[t][k] = k < a.k ? to_f32<T>(row_ptr<T>(a.q, none, seq, t0 + t, head_k)[k]) : 0.f;
        }
        if (tid < nt) {
            const float g = row_ptr<float>(a.g, none, seq, t0 + tid, head)[0];
            sa[tid] = decay_of(g);
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

// ---- many large states: a ring of whole states in shared memory --------------------
// A CTA takes its share of the heads in turn.  A head's state is one run of
// bytes, so one thread moves it with one bulk copy each way: it stores the state that
// is done and loads the one that is next in its place, two others being on their way
// or at work meanwhile, so that reads and writes never pause for the sums.  Four warps
// bring the tokens' small inputs (a token each) ahead of them, eight warps compute.
// Smaller states take less of the SM, which then runs two or three such CTAs.

namespace {

constexpr int kRingStages = 3, kRingTokens = 4;
constexpr int kRingWarps = 8, kRingCompute = 32 * kRingWarps, kRingThreads = kRingCompute + 32 * (1 + kRingTokens);
// CTAs of an SM: as many as their shared memory and registers admit
constexpr int ring_ctas(int kp, int vp) { return kp * vp > 8192 ? 1 : kp * vp > 4096 ? 2 : 3; }

template <int KP, int VP>
struct RingTokens {
    float k[kRingTokens][KP], q[kRingTokens][KP], v[kRingTokens][VP];
    float decay[kRingTokens], beta[kRingTokens], qk[kRingTokens];
    int count;
    int pad[3];
};
template <int KP, int VP>
struct RingSmem {
    float state[kRingStages][KP * VP];
    RingTokens<KP, VP> in[kRingStages];
    float4 sum_k[2][kRingWarps][VP / 4], sum_q[2][kRingWarps][VP / 4];
    uint64_t state_full[kRingStages], in_full[kRingStages], done[kRingStages];
    int gave_up;
};
static_assert(sizeof(RingSmem<128, 128>) <= 227 * 1024, "too much shared memory");

// Whether any of the computing threads says so; all of them wait for one another.
__device__ __forceinline__ bool any_computing(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"((uint32_t)x), "n"(kRingCompute) : "memory");
    return r != 0;
}
// How many tokens of the sequence count; 0 where its page does not exist.
__device__ __forceinline__ int step_tokens(const DeltaStepArgs &a, long long seq, long long &page) {
    page = a.slots ? a.slots[seq] : seq;
    const int count = a.lengths ? a.lengths[seq] : a.t;
    return page < 0 || page >= a.pages || count < 0 ? 0 : count > a.t ? a.t : count;
}

}  // namespace

// VP / 4 lanes hold a row's columns, four each.
template <typename T, int KP, int VP>
__global__ void __launch_bounds__(kRingThreads, ring_ctas(KP, VP)) delta_step_ring_kernel(const DeltaStepArgs a) {
    constexpr int LPR = VP / 4, GROUPS = kRingCompute / LPR, ROWS = KP / GROUPS;
    extern __shared__ __align__(128) unsigned char ring_bytes[];
    RingSmem<KP, VP> &m = *reinterpret_cast<RingSmem<KP, VP> *>(ring_bytes);
    volatile int *gave_up = &m.gave_up;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long heads = a.seqs * a.hv;
    const int items = (int)((heads - blockIdx.x + gridDim.x - 1) / gridDim.x);
    auto item = [&](int i, long long &seq, int &head) {
        const long long x = blockIdx.x + (long long)i * gridDim.x;
        seq = x / a.hv;
        head = (int)(x % a.hv);
    };
    if (tid == 0) {
        for (int i = 0; i < kRingStages; ++i) {
            mbar_init(&m.state_full[i], 1);
            mbar_init(&m.in_full[i], kRingTokens);
            mbar_init(&m.done[i], kRingWarps);
        }
        m.gave_up = 0;
        mbar_init_done();
    }
    __syncthreads();

    if (warp == kRingWarps) {   // states
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(a.k * a.v) * 4;
            const size_t words = (size_t)a.k * a.v;
            float *at[kRingStages];   // where the stages' states belong; null where there is none
#pragma unroll
            for (int st = 0; st < kRingStages; ++st) at[st] = nullptr;
            int begun = 0;   // loads
            int i = 0;
            for (; i < items + kRingStages; i += kRingStages)
#pragma unroll
                for (int st = 0; st < kRingStages; ++st) {
                    const int now = i + st, before = now - kRingStages;
                    long long seq, page;
                    int head;
                    float *to = nullptr;
                    if (now < items) {
                        item(now, seq, head);
                        if (step_tokens(a, seq, page) > 0) to = a.state + (size_t)(page * a.hv + head) * words;
                    }
                    if (before >= 0 && before < items) {
                        wait_phase(&m.done[st], (before / kRingStages) & 1, gave_up);
                        if (!*gave_up && at[st] != nullptr) {
                            bulk_store(at[st], smem_u32(m.state[st]), bytes);
                            bulk_commit();
                            bulk_wait_read();
                        }
                    }
                    at[st] = to;
                    if (now >= items || *gave_up) continue;
                    begun = now + 1;
                    if (to != nullptr) {
                        mbar_arrive_expect_tx(&m.state_full[st], bytes);
                        bulk_load(m.state[st], to, bytes, &m.state_full[st]);
                    } else {
                        mbar_arrive(&m.state_full[st]);
                    }
                }
            bulk_wait();
            if (*gave_up)   // loads in flight
                for (int x = begun < kRingStages ? 0 : begun - kRingStages; x < begun; ++x)
                    wait_drained(&m.state_full[x % kRingStages], (x / kRingStages) & 1);
        }
    } else if (warp > kRingWarps) {   // a token's inputs
        const int t = warp - kRingWarps - 1;
        const Span none{};
        for (int i = 0; i < items; ++i) {
            const int st = i % kRingStages;
            long long seq, page;
            int head;
            item(i, seq, head);
            const int head_k = head / (a.hv / a.hk), count = step_tokens(a, seq, page);
            float k[KP / 32], q[KP / 32], v[VP / 32], g = 0.f, beta = 0.f, d = 0.f;
            if (t < count) {
#pragma unroll
                for (int j = 0; j < KP / 32; ++j) {
                    const int x = lane + 32 * j;
                    k[j] = x < a.k ? to_f32<T>(row_ptr<T>(a.kk, none, seq, t, head_k)[x]) : 0.f;
                    q[j] = x < a.k ? to_f32<T>(row_ptr<T>(a.q, none, seq, t, head_k)[x]) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < VP / 32; ++j) {
                    const int x = lane + 32 * j;
                    v[j] = x < a.v ? to_f32<T>(row_ptr<T>(a.vv, none, seq, t, head)[x]) : 0.f;
                }
                g = row_ptr<float>(a.g, none, seq, t, head)[0];
                beta = a.beta_f32 ? row_ptr<float>(a.beta, none, seq, t, head)[0] : to_f32<T>(row_ptr<T>(a.beta, none, seq, t, head)[0]);
#pragma unroll
                for (int j = 0; j < KP / 32; ++j) d += k[j] * q[j];
#pragma unroll
                for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
            }
            if (i >= kRingStages) wait_phase(&m.done[st], (i / kRingStages - 1) & 1, gave_up);
            if (__any_sync(0xffffffffu, *gave_up)) break;
            RingTokens<KP, VP> &in = m.in[st];
            if (t < count) {
#pragma unroll
                for (int j = 0; j < KP / 32; ++j) {
                    in.k[t][lane + 32 * j] = k[j];
                    in.q[t][lane + 32 * j] = q[j];
                }
#pragma unroll
                for (int j = 0; j < VP / 32; ++j) in.v[t][lane + 32 * j] = v[j];
                if (lane == 0) {
                    in.decay[t] = decay_of(g);
                    in.beta[t] = beta;
                    in.qk[t] = d;
                }
            }
            if (t == 0 && lane == 0) in.count = count;
            warp_arrive(&m.in_full[st], lane);
        }
    } else {
        const int col = tid % LPR, group = tid / LPR, c0 = 4 * col;
        const bool in_row = c0 < a.v;   // the columns come in fours
        const size_t ostride = (size_t)a.hv * a.v;
        int n = 0;   // tokens so far
        bool failed = false;
        for (int i = 0; i < items; ++i) {
            const int st = i % kRingStages;
            long long seq;
            int head;
            item(i, seq, head);
            wait_phase(&m.in_full[st], (i / kRingStages) & 1, gave_up);
            wait_phase(&m.state_full[st], (i / kRingStages) & 1, gave_up);
            failed = any_computing(*gave_up != 0);   // all eight warps leave together
            if (failed) break;
            const RingTokens<KP, VP> &in = m.in[st];
            T *out = static_cast<T *>(a.o) + ((size_t)seq * a.t * a.hv + head) * a.v;
            const int count = in.count;
            for (int x = tid; x < (a.t - count) * VP; x += kRingCompute)   // outputs of tokens that do not count
                if (x % VP < a.v) out[(count + x / VP) * ostride + x % VP] = from_f32<T>(0.f);
            if (count > 0) {
                float4 S[ROWS];
                float *state = m.state[st] + c0;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const int k = group + r * GROUPS;
                    S[r] = in_row && k < a.k ? *reinterpret_cast<const float4 *>(state + k * a.v) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                for (int t = 0; t < count; ++t, ++n) {
                    const float decay = in.decay[t], beta = in.beta[t];
                    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        // a forgotten state is 0 even where it held an infinity or a NaN
                        if (decay == 0.f) S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                        S[r].x *= decay; S[r].y *= decay; S[r].z *= decay; S[r].w *= decay;
                        fma4(pk, in.k[t][group + r * GROUPS], S[r]);
                        fma4(pq, in.q[t][group + r * GROUPS], S[r]);
                    }
#pragma unroll
                    for (int x = LPR; x < 32; x <<= 1) { pk = shfl_add(pk, x); pq = shfl_add(pq, x); }
                    if (lane < LPR) { m.sum_k[n & 1][warp][lane] = pk; m.sum_q[n & 1][warp][lane] = pq; }
                    any_computing(false);
                    pk = m.sum_k[n & 1][0][col];
#pragma unroll
                    for (int w = 1; w < kRingWarps; ++w) fma4(pk, 1.f, m.sum_k[n & 1][w][col]);
                    const float4 v = *reinterpret_cast<const float4 *>(in.v[t] + c0);
                    const float4 u = make_float4(beta * (v.x - pk.x), beta * (v.y - pk.y), beta * (v.z - pk.z), beta * (v.w - pk.w));
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) fma4(S[r], in.k[t][group + r * GROUPS], u);
                    if (warp == t && lane < LPR && in_row) {
                        pq = m.sum_q[n & 1][0][col];
#pragma unroll
                        for (int w = 1; w < kRingWarps; ++w) fma4(pq, 1.f, m.sum_q[n & 1][w][col]);
                        fma4(pq, in.qk[t], u);
                        T *op = out + t * ostride + c0;
                        op[0] = from_f32<T>(a.scale * pq.x);
                        op[1] = from_f32<T>(a.scale * pq.y);
                        op[2] = from_f32<T>(a.scale * pq.z);
                        op[3] = from_f32<T>(a.scale * pq.w);
                    }
                }
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const int k = group + r * GROUPS;
                    if (in_row && k < a.k) *reinterpret_cast<float4 *>(state + k * a.v) = S[r];
                }
                fence_async();
            }
            warp_arrive(&m.done[st], lane);
        }
        if (failed)   // the outputs are not what they should be: say so
            for (int i = 0; i < items; ++i) {
                long long seq;
                int head;
                item(i, seq, head);
                T *out = static_cast<T *>(a.o) + ((size_t)seq * a.t * a.hv + head) * a.v;
                for (int x = tid; x < a.t * VP; x += kRingCompute)
                    if (x % VP < a.v) out[x / VP * ostride + x % VP] = from_f32<T>(__int_as_float(0x7fc00000));
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
template <typename T, int KP, int VP>
cudaError_t step_ring(const DeltaStepArgs &a, cudaStream_t s) {
    constexpr int bytes = sizeof(RingSmem<KP, VP>);
    cudaError_t e = cudaFuncSetAttribute(delta_step_ring_kernel<T, KP, VP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    delta_step_ring_kernel<T, KP, VP><<<152 * ring_ctas(KP, VP), kRingThreads, bytes, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int KP>
cudaError_t step_for(const DeltaStepArgs &a, cudaStream_t s) {
    const long long heads = a.seqs * a.hv;
    const bool whole = a.v % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;   // as bulk copies want them
    // The ring against the states in registers, us of a token each (caches flushed before, bf16):
    //   128 x 128: 608 heads 23 / 25, 1024 33 / 37, 8192 173 / 238, four tokens 301 / 384
    //   64 x 64: 640 heads 13 / 14, 2048 21 / 29, 8192 50 / 89    64 x 128: 640 19 / 20, 8192 119 / 164
    //   128 x 64: 640 heads 19 / 17, 1280 27 / 25, 2048 35 / 38, 8192 103 / 126
    // Fewer heads leave the ring's CTAs with two or three states each.
    if (whole && a.v > 32 && a.v <= 128 && a.t <= kRingTokens && heads >= (KP == 128 && a.v <= 64 ? 12 : 4) * 152)
        return a.v <= 64 ? step_ring<T, KP, 64>(a, s) : step_ring<T, KP, 128>(a, s);
    // Blocks of 64 columns where there are CTAs enough for the machine, narrower ones where there are
    // not: more of the state's bytes are then in flight at once.
    if (a.v <= 32 || heads * ((a.v + 63) / 64) < 2 * 152) return step<T, KP, 32>(a, s);
    return step<T, KP, 64>(a, s);
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
