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
    // codes 0, 1 and 2, 3 as f16 pairs
    static __device__ __forceinline__ void halves(uint32_t c, uint32_t& lo, uint32_t& hi) {
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(c));
    }
    // codes 0, 2 and 1, 3
    static __device__ __forceinline__ void evens_odds(uint32_t c, uint32_t& even, uint32_t& odd) {
        halves(__byte_perm(c, 0, 0x3120), even, odd);
    }
    // codes 0, 1 and 2, 3 as bf16 pairs: the code's bits moved to bf16's places are the
    // number times 2^-120, subnormal numbers included.  (A byte with its sign above it,
    // four bits to the left: the sign, copies of it that go, the other seven bits.)
    static __device__ __forceinline__ void pairs(uint32_t c, uint32_t& lo, uint32_t& hi) {
        asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(c));
        asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(hi) : "r"(c));
        lo = scaled(lo << 4 & 0x87f087f0u), hi = scaled(hi << 4 & 0x87f087f0u);
    }
    static __device__ __forceinline__ uint32_t scaled(uint32_t p) {
        uint32_t r;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(0x7b807b80u));   // 2^120
        return r;
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
    // codes 0, 1 and 2, 3 as f16 pairs: 1024 + (code + 128), less 1152
    static __device__ __forceinline__ void halves(uint32_t c, uint32_t& lo, uint32_t& hi) {
        const uint32_t u = c ^ 0x80808080u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
    }
    // codes 0, 2 and 1, 3
    static __device__ __forceinline__ void evens_odds(uint32_t c, uint32_t& even, uint32_t& odd) {
        const uint32_t u = c ^ 0x80808080u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(__byte_perm(u, 0x64646464u, 0x4240)), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(__byte_perm(u, 0x64646464u, 0x4341)), "r"(0x64806480u));
    }
    // codes 0, 1 and 2, 3 as bf16 pairs
    static __device__ __forceinline__ void pairs(uint32_t c, uint32_t& lo, uint32_t& hi) {
        lo = widen(__byte_perm(c, 0x43434343u, 0x4140)), hi = widen(__byte_perm(c, 0x43434343u, 0x4342));
    }
    // 128 + (the lower seven bits), less 128 + 128 (the sign bit)
    static __device__ __forceinline__ uint32_t widen(uint32_t p) {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p & 0xff7fff7fu), "r"(p & 0xff80ff80u));
        return r;
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
