// The paged key-value cache's formats as the kernels see them, and what the kernels around the linears share.
#pragma once

#include <cstdint>

#include "nf4_device.cuh"
#include "nf4_internal.h"

namespace nf4 {

// Bytes of one stored vector of D values, and of its scales.
__host__ __device__ constexpr int kv_vector_bytes(int format, int D) {
    return format == kKvBf16 ? 2 * D : format == kKvFp8 ? D : D / 2;
}
__host__ __device__ constexpr int kv_scale_bytes(int format, int D) {
    return format == kKvBf16 ? 0 : format == kKvFp8 ? 4 : D / 64 * 2;
}

constexpr float kFp8Max = 448.0f;  // the largest e4m3 value

// Two e4m3 codes (low byte first) -> two halves; exact (e4m3 is a subset of binary16).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t d;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(d) : "r"(codes));
    return d;
}

// Two floats -> two e4m3 codes (lo in the low byte), round to nearest even, saturated at +-448.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float2 bf16x2_to_f32x2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// A launch that may begin before the previous kernel of the stream has ended (its kernels wait before they read).
inline cudaLaunchConfig_t pdl_config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace nf4
