// kvc8_codes.cuh -- int8 codes as exact 16-bit floating-point pairs, and the small
// arithmetic that the shared-prefix attention's kernels (and the rotation's) have in common.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace kvc8 {

__device__ __forceinline__ float ex2(float x) {  // 2^x, -inf gives 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_fp16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_fp16(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The power of two at or below x > 0, from 2^-100 to 2^100, where it and its reciprocal are
// normal (divided by it, a value of 2^116 or more passes the range of fp16).
__device__ __forceinline__ int power_of(float x) {
    return min(100, max(-100, (int)(__float_as_uint(x) >> 23) - 127));
}

// Byte c of a word beside 0x43 is, with the low seven bits alone, 128 + them, and with
// the sign bit alone 128 or 256 (the exponent's lowest bit is the sign's place); the
// difference is c, exact in bf16.  x: codes in bytes 0 and 2.
__device__ __forceinline__ uint32_t bf16_of(uint32_t x) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((x & 0x007F007Fu) | 0x43004300u), "r"((x & 0x00800080u) | 0x43004300u));
    return r;
}
// c + 128 beside 0x64 is 1024 + c + 128.  x: 0x64 and c + 128, twice.
__device__ __forceinline__ uint32_t fp16_of(uint32_t x) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
    return r;
}
// Two neighbouring codes of a word with every sign bit flipped (select 0x4140: the first two,
// 0x4342: the others).
__device__ __forceinline__ uint32_t codes_fp16(uint32_t biased, uint32_t select) {
    return fp16_of(__byte_perm(biased, 0x64646464u, select));
}
// The same byte of two words, whose places are nibbles 0 and 2 of select.
template <bool HALF>
__device__ __forceinline__ uint32_t codes_of_two(uint32_t a, uint32_t b, uint32_t select) {
    const uint32_t x = __byte_perm(a, b, select);
    return HALF ? fp16_of((x & 0x00FF00FFu) ^ 0x64806480u) : bf16_of(x);
}

// Launch that may start when every block of the kernel before it in the stream has started.
template <typename... A>
cudaError_t launch_dependent(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace kvc8
