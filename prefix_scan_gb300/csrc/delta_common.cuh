// delta_common.cuh -- pieces shared by the gated delta rule's kernels: the
// split of 32-bit numbers into pairs of bf16, matrix products of 16-bit
// tiles (mma.sync) on swizzled shared-memory images, tile loads with
// zero-filled edges, and where a chunk's data lie in the workspace.
//
// Notation, for one value head of one sequence, cut into chunks of C = 64
// tokens: S is the K x V state at the chunk's start, G the running sum of
// the log decays g inside the chunk, and
//     D_ij = exp(G_i - G_j)          (j <= i)
//     N_ij = D_ij k_i.k_j            (j < i),   P_ij = scale D_ij q_i.k_j
//     T    = (I + diag(beta) N)^-1
//     R    = V - exp(G) K S          U = T diag(beta) R
//     O    = scale exp(G) Q S + P U
//     S'   = exp(G_C) S + sum_j exp(G_C - G_j) k_j u_j^T.
// These are the recurrence S <- e^g S, u = beta (v - k^T S), S <- S + k u^T,
// o = scale q^T S with the tokens of a chunk taken together.
//
// Precision.  States, T, P, N and every sum are 32-bit.  As operands of the
// matrix units they are pairs hi + lo of bf16 (16 significant bits, off by 2^-18.4
// of the number in the root mean square), so that states and the gradients of g
// come out to about 2^-18 and not to bf16's 2^-9.  bf16 inputs are exact with one
// number (NP = 1), f16 inputs with a pair (NP = 2); f32 inputs become pairs, and lose
// eight bits, where they meet a matrix unit: q, k and dO (v meets none).
// Why two parts: a third one would keep 24 bits, at half as many products again (three
// for two beside an exact input, six for four of two pairs) and half as many bytes of
// every image; and the chains would not fit, as the state of 128 columns, its operand in
// three parts (192), X and S^T Q^T (128) and the two other operands (96 each) take more
// than tensor memory's 512.  16-bit outputs are the rounding of what they would be anyway;
// f32 ones (states, gradients of states and of g, everything of f32 inputs) are off by
// 1.3e-6 to 5e-6 where f32 sums are by 1e-7 to 4e-7.  The single-step kernel is f32
// throughout, for whole prompts too.  Where a number goes into pairs:
//     q, k, dO of f32                 load_tile() here; dO of the chains in delta_chain_backward.cu
//     P, N, T's blocks, T - 1         delta_prepare.cu
//     S, beta R, exp(G_C - G) U, U    delta_chain.cu; a segment's M too
//     dS', Y, exp(G) dR, dU, scaled dO    delta_chain_backward.cu
//     a segment's state               delta_join.cu
//     S, U, dS', dU as they were left, F1, F2    delta_gradients.cu
// For bf16 inputs U^T P^T and X2, X3 of the gradients leave out the product of the two
// lower parts, 2^-19.6 of its terms: nothing in results that are rounded at 2^-9, and in
// the gradients of g, which are f32 always, a twentieth on top of the pairs' own errors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "delta_internal.h"

namespace ps {

// ---- warp-level matrix products ----------------------------------------------

// D (16x8, f32) += A (16x16, bf16, row) B (16x8, bf16, col).  Lane l holds, with
// r = l / 4 and c = 2 (l % 4): A rows r, r+8 at columns c.. and c+8..; B row
// pairs c.., c+8.. of column r; D rows r, r+8 at columns c, c+1.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---- pairs of bf16 -------------------------------------------------------------

__device__ __forceinline__ uint32_t pack_bf16(float lo_half, float hi_half) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi_half), "f"(lo_half));
    return r;
}
__device__ __forceinline__ float bf16_low(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_high(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
// (x, y) as a pair of packed bf16x2: x ~ low halves of hi + lo, y ~ high halves.
// (An infinity becomes a NaN: its rest is inf - inf.)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - bf16_low(hi), y - bf16_high(hi));
}
// Two accumulator tiles of a 16-column block (columns 0-7 and 8-15) as a left operand.
__device__ __forceinline__ void split_tiles(const float (&lo8)[4], const float (&hi8)[4], uint32_t (&f)[2][4]) {
    split2(lo8[0], lo8[1], f[0][0], f[1][0]);
    split2(lo8[2], lo8[3], f[0][1], f[1][1]);
    split2(hi8[0], hi8[1], f[0][2], f[1][2]);
    split2(hi8[2], hi8[3], f[0][3], f[1][3]);
}

// ---- swizzled images -----------------------------------------------------------
// A tile of 16-bit numbers in rows of 64 (128 bytes); the 16-byte piece p of row r sits at
// piece p ^ (r & 7), so that the eight rows of an ldmatrix matrix fall into eight different
// bank groups.  It is also the 128-byte swizzle of the tensor-memory products' operands, for
// which an image starts at a multiple of 1024 bytes.  Wider tiles are columns of such images:
// numbers 64 h .. 64 h + 63 of all rows lie HALF bytes after the 64 before them.
constexpr int kHalf = 128 * 128;   // 128 rows
template <int HALF = kHalf>
__device__ __forceinline__ uint32_t img(uint32_t base, int row, int piece) {
    return base + (uint32_t)((piece >> 3) * HALF + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}
// Operands by ldmatrix from an image whose rows are `row`s and whose pieces hold
// eight 16-bit columns.  r16, c16: the first row and the first column.
//   load_a    A fragment of the 16x16 block (A row = image row, A column = image column)
//   load_a_t  A fragment of the block's transpose (A row = image column)
//   load_b    B fragments of two 8-column tiles n = rows r16.., r16+8.. and k = columns
//             c16..c16+15 (B column = image row): b[0], b[1] and b[2], b[3]
//   load_b_t  the same with n = columns c16.., c16+8.. and k = rows r16..r16+15
template <int HALF = kHalf>
__device__ __forceinline__ void load_a(uint32_t (&a)[4], uint32_t base, int r16, int c16, int lane) {
    ldsm4(a, img<HALF>(base, r16 + (lane & 15), (c16 >> 3) + (lane >> 4)));
}
template <int HALF = kHalf>
__device__ __forceinline__ void load_a_t(uint32_t (&a)[4], uint32_t base, int r16, int c16, int lane) {
    // matrices: (rows 0-7, cols 0-7), (rows 0-7, cols 8-15), (rows 8-15, cols 0-7), (rows 8-15, cols 8-15)
    ldsm4_t(a, img<HALF>(base, r16 + (lane & 7) + ((lane >> 4) << 3), (c16 >> 3) + ((lane >> 3) & 1)));
}
template <int HALF = kHalf>
__device__ __forceinline__ void load_b(uint32_t (&b)[4], uint32_t base, int r16, int c16, int lane) {
    ldsm4(b, img<HALF>(base, r16 + (lane & 7) + ((lane >> 4) << 3), (c16 >> 3) + ((lane >> 3) & 1)));
}
template <int HALF = kHalf>
__device__ __forceinline__ void load_b_t(uint32_t (&b)[4], uint32_t base, int r16, int c16, int lane) {
    ldsm4_t(b, img<HALF>(base, r16 + (lane & 15), (c16 >> 3) + (lane >> 4)));
}

// ---- tile loads ------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
    const int n = take ? 16 : 0;   // 0: sixteen zero bytes, the source is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
// Two values as one word of 16-bit T.
template <typename T> __device__ __forceinline__ uint32_t pack2(float x, float y);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) { return pack_bf16(x, y); }
template <> __device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T> struct Planes { static constexpr int NP = 2; };
template <> struct Planes<__nv_bfloat16> { static constexpr int NP = 1; };

// One 64-row tile: rows `first`.. of a tensor whose row r starts at src + r * stride,
// columns [0, cols) of COLS; rows at and past `rows` and columns at and past
// `cols` are zero (they are not read).  bf16 goes over as it is, by asynchronous
// copies where `vec` says that every row is 16-byte aligned and cols a multiple
// of 8; other types become a pair of images hi, hi + plane.
template <typename T, int COLS>
__device__ __forceinline__ void load_tile(uint32_t hi, uint32_t plane, const T *src, long long stride, int rows,
                                          int cols, bool vec, int tid, int nthreads) {
    constexpr int PIECES = COLS / 8;
    for (int i = tid; i < kChunk * PIECES; i += nthreads) {
        const int r = i / PIECES, p = i % PIECES;
        const uint32_t dst = img(hi, r, p);
        const bool in = r < rows && p * 8 < cols;
        if constexpr (Planes<T>::NP == 1) {
            if (vec) {
                cp_async16(dst, in ? (const void *)(src + r * stride + p * 8) : (const void *)src, in);
                continue;
            }
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = p * 8 + 2 * j;
                const T z = from_f32<T>(0.f);
                const T x = r < rows && c < cols ? src[r * stride + c] : z;
                const T y = r < rows && c + 1 < cols ? src[r * stride + c + 1] : z;
                w[j] = (uint32_t)__bfloat16_as_ushort(x) | ((uint32_t)__bfloat16_as_ushort(y) << 16);
            }
            st_shared16(dst, make_uint4(w[0], w[1], w[2], w[3]));
        } else {
            float x[8];
            if (vec && in) {
                constexpr int NV = (int)sizeof(T) / 2;   // 16-byte loads for eight elements
                uint4 raw[NV];
#pragma unroll
                for (int j = 0; j < NV; ++j) raw[j] = reinterpret_cast<const uint4 *>(src + r * stride + p * 8)[j];
                const T *t = reinterpret_cast<const T *>(raw);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(t[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = r < rows && p * 8 + j < cols ? to_f32<T>(src[r * stride + p * 8 + j]) : 0.f;
            }
            uint32_t h[4], l[4];   // exact for f16; f32 keeps 16 bits (see above)
#pragma unroll
            for (int j = 0; j < 4; ++j) split2(x[2 * j], x[2 * j + 1], h[j], l[j]);
            st_shared16(dst, make_uint4(h[0], h[1], h[2], h[3]));
            st_shared16(dst + plane, make_uint4(l[0], l[1], l[2], l[3]));
        }
    }
}

// Copies BYTES (a multiple of 16) of an image as it stands in the workspace.
template <int BYTES, int THREADS>
__device__ __forceinline__ void load_image(uint32_t dst, const void *src, int tid) {
    const char *s = static_cast<const char *>(src) + tid * 16;
    dst += tid * 16;
#pragma unroll
    for (int i = 0; i < BYTES / (16 * THREADS); ++i) cp_async16(dst + i * THREADS * 16, s + i * THREADS * 16, true);
    constexpr int DONE = BYTES / (16 * THREADS) * 16 * THREADS;
    if (DONE < BYTES && DONE + tid * 16 < BYTES) cp_async16(dst + DONE, s + DONE, true);
}
// exp(x).  Errors of decays near 1 multiply up over the many tokens or chunks that such a state remembers, so there
// 1 + expm1(x), rounded once, takes the place of expf, whose errors of an ulp have one sign: with it 300 single steps of
// x = -0.00005 .. -0.05 leave outputs off by 1.3e-6, and 256 chunks of small x a state off by 3.7e-6.
__device__ __forceinline__ float exp_rounded(float x) { return x > -0.5f ? 1.f + expm1f(x) : expf(x); }

// ---- sequences and chunks ----------------------------------------------------------

// Where a sequence's tokens lie.  Offsets that leave [0, tokens] are clamped, each
// sequence by itself, so that wrong ones give wrong results and no access out of
// range.  Where they fall, sequences may share tokens and slots: a running maximum
// would keep them apart, at the price of another launch for every call.
struct Span {
    long long first;   // token of the whole input (outputs are stored by it)
    long long at;      // token offset to add to a tensor's base (0 where seq_stride is used)
    long long len;
    long long slot;    // its first chunk's slot in the workspace
};
__device__ __forceinline__ Span span_of(const DeltaShape &s, long long seq) {
    Span r;
    if (s.cu == nullptr) {
        r.first = seq * s.tokens;
        r.at = 0;
        r.len = s.tokens;
        r.slot = seq * ((s.tokens + kChunk - 1) / kChunk);
    } else {
        long long a = s.cu[seq], b = s.cu[seq + 1];
        a = a < 0 ? 0 : a > s.tokens ? s.tokens : a;
        b = b < a ? a : b > s.tokens ? s.tokens : b;
        r.first = r.at = a;
        r.len = b - a;
        r.slot = a / kChunk + seq;   // ceil(len / C) <= floor(b / C) - floor(a / C) + 1: slots never meet
    }
    return r;
}
// The sequence that chunk slot `slot` belongs to, or -1 if no chunk uses it.
__device__ __forceinline__ long long seq_of_slot(const DeltaShape &s, long long slot) {
    if (s.cu == nullptr) {
        const long long per = (s.tokens + kChunk - 1) / kChunk;
        return per ? slot / per : -1;
    }
    long long lo = 0, hi = s.seqs - 1;   // the last sequence whose first slot is <= slot
    while (lo < hi) {
        const long long mid = (lo + hi + 1) / 2;
        if (span_of(s, mid).slot <= slot) lo = mid; else hi = mid - 1;
    }
    const Span p = span_of(s, lo);
    return slot >= p.slot && slot - p.slot < (p.len + kChunk - 1) / kChunk ? lo : -1;
}
// A chain's work: the whole sequence, or one of the segments that it is cut into (span then is the
// segment's alone).
struct Chain {
    long long seq, slot;   // slot: of the segment
    bool first, last;      // first, last segment of its sequence
    Span span;
};
__device__ __forceinline__ long long first_segment(const DeltaArgs &a, long long seq) { return span_of(a.s, seq).slot / a.seg + seq; }
__device__ __forceinline__ bool chain_of(const DeltaArgs &a, long long index, Chain &c) {
    if (a.seg == 0) {
        if (a.order) index = a.order[index];
        c = Chain{index, 0, true, true, span_of(a.s, index)};
        return true;
    }
    long long lo = 0, hi = a.s.seqs - 1;   // the last sequence whose first segment is <= index
    while (lo < hi) {
        const long long mid = (lo + hi + 1) / 2;
        if (first_segment(a, mid) <= index) lo = mid; else hi = mid - 1;
    }
    const Span all = span_of(a.s, lo);
    const long long part = index - first_segment(a, lo), tokens = (long long)a.seg * kChunk;
    const long long parts = all.len > 0 ? (all.len + tokens - 1) / tokens : 1;
    if (part < 0 || part >= parts) return false;
    c = Chain{lo, index, part == 0, part == parts - 1, all};
    c.span.first += part * tokens;
    c.span.at += part * tokens;
    c.span.slot += part * a.seg;
    c.span.len = all.len - part * tokens < tokens ? all.len - part * tokens : tokens;
    return true;
}
template <typename T>
__device__ __forceinline__ const T *row_ptr(const DeltaTensor &t, const Span &sp, long long seq, long long tok, int head) {
    return static_cast<const T *>(t.p) + seq * t.seq + (sp.at + tok) * t.tok + (long long)head * t.head;
}

}  // namespace ps
