// delta_tmem.cuh -- tensor-memory primitives of the gated delta rule's chains
// (inline PTX, sm_103a): allocation, loads and stores of 32-bit columns, the
// 128-row matrix product with its left operand in tensor memory and its right
// one in shared memory, and bounded waits.
//
// Tensor memory is 128 lanes of 512 32-bit columns; an address is lane << 16 |
// column, and warp w of a group of four reaches lanes 32 (w % 4) .. + 31.  A
// 128-row accumulator of N columns takes N columns, row = lane; a 16-bit left
// operand packs columns 2 c and 2 c + 1 of its row into column c.
#pragma once

#include "delta_common.cuh"
#include "scan_pipeline.cuh"

namespace ps {

constexpr uint32_t kTmemColumns = 512;

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst) {   // one warp, all lanes
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_dst), "n"(kTmemColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr) {        // the same warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "n"(kTmemColumns) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of this warp's lanes (8 for the packed pairs).
__device__ __forceinline__ void tmem_get16(uint32_t (&u)[16], uint32_t addr) {   // usable after tmem_wait_ld()
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(float (&r)[16], uint32_t addr) {
    uint32_t u[16];
    tmem_get16(u, addr);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(u[i]);
}
// 16 columns at each of two addresses.
__device__ __forceinline__ void tmem_ld16(float (&r)[16], uint32_t addr, float (&q)[16], uint32_t addr2) {
    uint32_t u[16], w[16];
    tmem_get16(u, addr);
    tmem_get16(w, addr2);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        r[i] = __uint_as_float(u[i]);
        q[i] = __uint_as_float(w[i]);
    }
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const float (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :: "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])), "r"(__float_as_uint(r[3])),
           "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])), "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7])),
           "r"(__float_as_uint(r[8])), "r"(__float_as_uint(r[9])), "r"(__float_as_uint(r[10])), "r"(__float_as_uint(r[11])),
           "r"(__float_as_uint(r[12])), "r"(__float_as_uint(r[13])), "r"(__float_as_uint(r[14])), "r"(__float_as_uint(r[15])),
           "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&u)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 :: "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(addr)
                 : "memory");
}
// Two f32 at a time (one instruction on sm_103a).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// 16 numbers as pairs of bf16, packed two to a word: a left operand's 8 columns.
__device__ __forceinline__ void split16(const float (&x)[16], uint32_t (&hi)[8], uint32_t (&lo)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        const float2 r = fma2(make_float2(bf16_low(hi[i]), bf16_high(hi[i])), make_float2(-1.f, -1.f), make_float2(x[2 * i], x[2 * i + 1]));
        lo[i] = pack_bf16(r.x, r.y);
    }
}
__device__ __forceinline__ void scale16(float (&x)[16], float f) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float2 a = mul2(make_float2(f, f), make_float2(x[i], x[i + 1]));
        x[i] = a.x; x[i + 1] = a.y;
    }
}
// x[i] *= y[i], with y in shared memory
__device__ __forceinline__ void scale16(float (&x)[16], const float *y) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(y + i);
        const float2 a = mul2(make_float2(f.x, f.y), make_float2(x[i], x[i + 1]));
        const float2 b = mul2(make_float2(f.z, f.w), make_float2(x[i + 2], x[i + 3]));
        x[i] = a.x; x[i + 1] = a.y; x[i + 2] = b.x; x[i + 3] = b.y;
    }
}
// The row's 16 numbers from column 16 c16 on into an image and the one of their second parts `lower` bytes on.
__device__ __forceinline__ void keep16(uint32_t image, uint32_t lower, int row, int c16, const uint32_t (&hi)[8], const uint32_t (&lo)[8]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t at = img(image, row, 2 * c16 + p);
        st_shared16(at, make_uint4(hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]));
        st_shared16(at + lower, make_uint4(lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]));
    }
}

// ---- products --------------------------------------------------------------------
// Descriptor of a 16-bit operand in a 128-byte-swizzled image (rows of 64 numbers,
// eight rows to 1024 bytes; delta_common.cuh's img() is that swizzle).  by_rows: the rows
// are the product's columns n and their numbers run along its inner dimension; otherwise
// rows run along the inner dimension, numbers along n, and 64 numbers further on along n lie
// `half` bytes further on.
__device__ __forceinline__ uint64_t operand(uint32_t addr, bool by_rows, uint32_t half) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(by_rows ? 1u : half >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// The operand `bytes` (a multiple of 16) further on.
__device__ __forceinline__ uint64_t further(uint64_t operand, uint32_t bytes) { return operand + (bytes >> 4); }
// Shape word: f32 accumulator, bf16 operands, 128 rows, n columns.
constexpr uint32_t shape(int n, bool by_rows) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (by_rows ? 0u : 1u << 16) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
// One lane of the (converged) warp.  Only that lane's products and commits are issued, but the whole
// warp runs the code around them: in uniform control flow their operands stay in uniform registers,
// where the instruction wants them, instead of being moved there one by one.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Products run in the order of issue only where one adds to the accumulator of the one before it, at the
// same columns and of the same shape.  All else that shares columns of tensor memory (another shape, an
// accumulator where an operand was) waits for a commit in between.
// d (128 x n) = (add ? d : 0) + a (128 x 16) b (16 x n)
__device__ __forceinline__ void mma_tmem(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t shape_word, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b), "r"(shape_word), "r"((uint32_t)add), "r"(one) : "memory");
}
// The same with the left operand in shared memory: an image whose rows are the product's rows, or
// (shape_word | kLeftByColumns) run along its inner dimension.
constexpr uint32_t kLeftByColumns = 1u << 15;
__device__ __forceinline__ void mma_smem(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t shape_word, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(shape_word), "r"((uint32_t)add), "r"(one) : "memory");
}
// The barrier completes its phase when all products issued so far have.
__device__ __forceinline__ void mma_commit(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        :: "r"(smem_u32(bar)), "r"(one) : "memory");
}

// ---- barriers --------------------------------------------------------------------
__device__ __forceinline__ void mbar_init_done() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// Shared memory written by this thread becomes visible to bulk copies and products.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// This thread's arrival once the asynchronous 16-byte copies that it has issued have landed.
__device__ __forceinline__ void mbar_arrive_after_copies(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}
// A wait that ran out (which a correct launch never does) raises the CTA's flag; every later wait
// then returns at once, so that all warps run to the kernel's end.  Waiting threads sleep in the
// barrier; wait_busy() polls instead, which wakes sooner, for the few warps that hold up all others.
constexpr uint32_t kWaitNs = 10000;
static __device__ __noinline__ void wait_long(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    if (*gave_up) return;
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 0; i < kMbarSpinCap; ++i) {
        if (mbar_try_wait_for(bar, parity, kWaitNs)) return;
        if ((i & 15u) == 15u && (*gave_up || global_ns() - t0 > kMbarWaitLimitNs)) break;
    }
    *gave_up = 1;
}
__device__ __forceinline__ void wait_phase(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    if (mbar_try_wait_for(bar, parity, kWaitNs)) return;
    wait_long(bar, parity, gave_up);
}
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void wait_busy(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
#pragma unroll 1
    for (int i = 0; i < 4096; ++i)
        if (mbar_test(bar, parity)) return;
    wait_long(bar, parity, gave_up);
}
// A wait that does not go by the flag: for copies and products in flight when a CTA gives up.
__device__ __forceinline__ void wait_drained(uint64_t *bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 0; i < kMbarSpinCap; ++i)
        if (mbar_try_wait(bar, parity) || ((i & 63u) == 63u && global_ns() - t0 > kMbarWaitLimitNs)) return;
}
// This warp's arrival, after all its lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" :: "l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace ps
