// The numbers of a cache held in 8 bits: e4m3, and whole numbers.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace colibri {

// kMost = kMant * 2^kExp: the largest code.
struct E4M3 {
    static constexpr float kMost = 448.f, kMant = 1.75f;
    static constexpr int kExp = 8;
    // 4 numbers to codes, nearest even
    static __device__ __forceinline__ uint32_t encode4(const float* v) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
    static __device__ __forceinline__ void decode4(uint32_t c, float* v) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3));
            const float2 f = __half22float2(h);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
};
struct I8 {
    static constexpr float kMost = 127.f, kMant = 1.984375f;
    static constexpr int kExp = 6;
    static __device__ __forceinline__ uint32_t encode4(const float* v) {
        uint32_t hi, d;
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(__float2int_rn(v[3])), "r"(__float2int_rn(v[2])), "r"(0));
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(__float2int_rn(v[1])), "r"(__float2int_rn(v[0])), "r"(hi));
        return d;
    }
    static __device__ __forceinline__ void decode4(uint32_t c, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(c >> (8 * i));
    }
};

// The smallest power of two 2^e, e >= -100, with most <= largest code * 2^e; NaN for
// what is not finite.
template <typename Code>
__device__ __forceinline__ float fitting_scale(uint32_t most_bits) {
    if (most_bits >= 0x7f800000u) return __int_as_float(0x7fc00000);
    // most = 1.m 2^(field - 127)
    const int e = (int)(most_bits >> 23) - 127 - Code::kExp +
                  ((most_bits & 0x7fffffu) > (__float_as_uint(Code::kMant) & 0x7fffffu));
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

}  // namespace colibri
