// Device helpers of the paged 4-bit KV cache: number formats and addressing.
#pragma once

#include <cuda_fp16.h>

#include "df_internal.cuh"

namespace df {

// Four bytes of E2M1 pairs as FP16 pairs: byte i's low half is the low value of r[i].
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// Two E4M3 bytes (low byte first) as an FP16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

// x rounded to E2M1 (nearest even, at most 6), as 4 bits of a byte.
__device__ __forceinline__ uint32_t f32_to_e2m1(float x) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(x));
    return r & 0xfu;
}
// Four values rounded to E2M1, the first in the lowest 4 bits of 16.
__device__ __forceinline__ uint32_t f32x4_to_e2m1(float x0, float x1, float x2, float x3) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, z;\n\tmov.b32 {z, z, z, z}, 0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b, z, z};\n\t}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
}

// (lo, hi) rounded to E4M3 (nearest even, at most 448): lo in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
    const uint32_t h = e4m3x2_to_f16(byte);
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

// Index of cache row `row` of sequence b, KV head h, in rows of the pools; -1 (with the status
// written) for a row past the page table or a page id outside the pool.
__device__ __forceinline__ long long paged_row(const df_paged_kv &c, int b, int h, long long row,
                                               int32_t *status) {
    if (row < 0 || row >= (long long)c.max_pages * c.page_size) {
        set_status(status, DF_ECAPACITY);
        return -1;
    }
    const int shift = 31 - __clz(c.page_size);
    const int page = c.page_table[(size_t)b * c.max_pages + (int)(row >> shift)];
    if (page < 0 || page >= c.n_pages) {
        set_status(status, DF_EINVAL);
        return -1;
    }
    return (((long long)page * c.n_kv_heads + h) << shift) + (row & (c.page_size - 1));
}

}  // namespace df
