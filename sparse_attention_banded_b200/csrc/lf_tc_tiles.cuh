// What the tensor-core kernels of the windowed attention share: tensor-memory
// loads and stores, MMAs with the A operand in tensor memory, tile layout
// helpers and the tensor maps of lf_heads views.
#pragma once

#include <cuda.h>

#include "lf_convert.cuh"
#include "lf_pair_math.cuh"
#include "lf_window.h"
#include "sm100.cuh"

namespace lf {
namespace sm100 {

template <typename T>
struct MmaFormat;
template <>
struct MmaFormat<__half> { static constexpr uint32_t fmt = 0; };
template <>
struct MmaFormat<__nv_bfloat16> { static constexpr uint32_t fmt = 1; };

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 32 lanes x 32 consecutive columns, into float registers.
__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}
// The same with 16 columns.
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16f(uint32_t taddr, const float (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]),
        "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The tensor-core instructions of a whole warp, issued by its elected lane.
// One asm block holds the four k-steps of a product: issued one by one from
// a lane's branch, each instruction's descriptors were moved to uniform
// registers again, about 120 cycles apiece (640 cycles for four MMAs and a
// commit of the attention kernel's issuing warp, 320 in this form).

// D[tmem] (+)= A B^T over 64 of K: A (128 rows) and B (64 rows) K-major in
// shared memory, 128-byte swizzle.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate = 0) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D0 (+)= A[:, :32] B[:32], D1 (+)= A[:, 32:] B[32:]: A (128 x 64, 16-bit) in
// tensor memory, its halves of 32 in 16 columns each, kApart columns apart;
// B 64 x 64, MN-major in shared memory.  D1 == D0 with accumulate_second: one sum.
template <int kApart = 32>
__device__ __forceinline__ void mma4_ts(uint32_t d0, uint32_t d1, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate, uint32_t accumulate_second) {
    asm volatile(
        "{\n\t.reg .pred e, p, q, r;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 r, %6, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "add.s32 a1, %2, 8;\n\tadd.s32 a2, %2, %7;\n\tadd.s32 a3, %2, %8;\n\t"
        "add.s64 b1, %3, 128;\n\tadd.s64 b2, %3, 256;\n\tadd.s64 b3, %3, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %3, %4, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [a2], b2, %4, r;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [a3], b3, %4, q;\n\t}" ::"r"(d0),
        "r"(d1), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(accumulate_second), "n"(kApart), "n"(kApart + 8)
        : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The whole warp waits; the result is warp-uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Half a row: 32 16-bit values from 32 floats.
template <typename T>
__device__ __forceinline__ void store_row32(T* p, const float* o) {
    uint4* d = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        d[c] = make_uint4(Pair<T>::pack(o[8 * c], o[8 * c + 1]), Pair<T>::pack(o[8 * c + 2], o[8 * c + 3]),
                          Pair<T>::pack(o[8 * c + 4], o[8 * c + 5]), Pair<T>::pack(o[8 * c + 6], o[8 * c + 7]));
}
template <typename T>
__device__ __forceinline__ void zero_row64(T* p) {
    uint4* d = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int c = 0; c < 8; ++c) d[c] = make_uint4(0u, 0u, 0u, 0u);
}

template <typename T>
__device__ __forceinline__ T* view_row(const lf_heads& v, int batch, int head, int token) {
    return static_cast<T*>(v.data) + batch * v.batch_stride + head * v.head_stride + token * v.token_stride;
}

}  // namespace sm100

// Tensor map of a 16-bit view: dims (64, heads, tokens, batches), box (64,
// box_heads, box_tokens, 1), 128-byte swizzle; rows of the box land in shared
// memory with the head inner.
bool make_heads_map(CUtensorMap* m, const lf_heads& v, int heads, int tokens, int batches, int box_heads,
                    int box_tokens);

}  // namespace lf
