// Products of a few queries with many short rows, for kernels that stream rows once
// and are bound by memory (pa_blocks_select, pa_weights_add): 16 rows against 8
// columns per mma.sync.m16n8k16 in bf16 (fp16 for e4m3 codes), accumulated in fp32.
//
// A sum over dimensions may run in any order, so long as rows and columns agree on it:
// the instruction's k slots are filled with what 16-byte loads bring, straight from
// global memory into registers.  Lane 4 g + t holds of rows g and g + 8 the chunks t, t
// + 4, t + 8, ... of 16 bytes; four lanes read 64 contiguous bytes of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_device.cuh"

namespace pa {

// c += A B of 16-bit values: bf16, or fp16 (F16).
template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-byte load of data that is read once.
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Two e4m3 codes (the low 16 bits) as two fp16 values, exactly (one cvt; to
// bf16 it takes four instructions, which then bound the kernels).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
    return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
}
__device__ __forceinline__ float2 f16x2_values(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
// Two fp32 values rounded to fp16, a in the low half.
__device__ __forceinline__ uint32_t to_f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A lane's chunk of 16 bytes as the operands of 16-bit MMAs: kVecs vectors of 4 words
// (8 values) each.
template <bool F8>
struct Chunk {
    static constexpr int kVecs = F8 ? 2 : 1;
};
template <bool F8>
__device__ __forceinline__ void widen(const uint4 &in, uint4 (&out)[Chunk<F8>::kVecs]) {
    if constexpr (F8) {
        out[0] = make_uint4(e4m3x2_to_f16x2(in.x & 0xffffu), e4m3x2_to_f16x2(in.x >> 16), e4m3x2_to_f16x2(in.y & 0xffffu),
                            e4m3x2_to_f16x2(in.y >> 16));
        out[1] = make_uint4(e4m3x2_to_f16x2(in.z & 0xffffu), e4m3x2_to_f16x2(in.z >> 16), e4m3x2_to_f16x2(in.w & 0xffffu),
                            e4m3x2_to_f16x2(in.w >> 16));
    } else {
        out[0] = in;
    }
}
// The first dimension of vector v of lane t of four (the chunks of a row in turn).
template <bool F8>
__host__ __device__ constexpr int vec_dim(int v, int t) {
    return F8 ? 16 * (t + 4 * (v >> 1)) + 8 * (v & 1) : 8 * (t + 4 * v);
}

}  // namespace pa
