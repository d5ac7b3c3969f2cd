// Attention of single bf16 rows over a paged cache of 8-bit codes with a scale for
// each block of tokens and key head: the decode step.
//
// The frame, its equal shares and its rings are attn_decode.cu's (attn_share.cuh); a
// step of 8 KB holds twice the keys.  What is added is the way from codes to operands:
//   s_j = (q . code_j) (scale_k c / 2^e)       c = scale * log2(e)
//   o   = sum_j (2^(s_j - m) scale_v) code_j,  l = sum_j 2^(s_j - m)
// so codes enter the products as they are, exact in 16 bits, and a scale costs one
// product per score and one per weight instead of one per element.
//
// Keys become f16, because that takes the fewest instructions (e4m3: one conversion
// per two codes; whole numbers: 5 instructions per 4), and the query row becomes f16
// with them: multiplied by a power of two 2^e that puts its largest element in
// [2^14, 2^15), it is exact but for elements 2^-29 below that one, whose error, 2^-39
// of it, is below that of the f32 sums.  Values become bf16, so that the weights,
// rounded once to the operand's type, keep f32's range whatever the scales are.
//
// Which element of a head stands at which place of the product's inner dimension is
// free as long as both operands agree: a lane takes 16 neighbouring codes of a key in
// one load and holds the same 16 elements of q.  Values come by ldmatrix.trans as
// 16-bit pairs of neighbouring codes of two keys, and the byte permutation that widens
// a pair also parts even columns from odd ones.
#include <cuda_runtime.h>

#include "attn_share.cuh"
#include "codes.cuh"

namespace colibri {
namespace {

__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Up to 16 MT rows of a group.
template <typename Code, int D, int MT>
struct CodeRows {
    using T = uint8_t;
    using Out = __nv_bfloat16;
    static constexpr int kD = D, kRows = 16 * MT, KS = kStepKeys<T, D>, kScratch = 0;
    uint32_t qf[MT][D / 16][4];
    float o[MT][D / 8][4], m[MT][2], l[MT][2];
    float c[MT][2];                                                // scale * log2(e) / 2^e

    template <bool kEarly>
    __device__ __forceinline__ void begin(const AttnArgs& a, int b, int h, int r0) {
        const int lane = threadIdx.x & 31;
        // row lane / 4 (+ 8); of each 64 columns the 16 from 16 (lane % 4) on
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int g = r0 + 16 * t + 8 * half + (lane >> 2);
                const uint4* q = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.q_stride + (int64_t)(h * a.group + g) * D);
                uint32_t w[D / 64][8], top = 0;
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 v = g < a.group ? ld_early<kEarly>(q + y * 8 + (lane & 3) * 2 + i) : make_uint4(0u, 0u, 0u, 0u);
                        w[y][4 * i] = v.x, w[y][4 * i + 1] = v.y, w[y][4 * i + 2] = v.z, w[y][4 * i + 3] = v.w;
                    }
                // (magnitudes as whole numbers: NaN and infinity on top)
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, max(w[y][i] & 0x7fffu, w[y][i] >> 16 & 0x7fffu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t up = min(268u - (top >> 7), 240u);    // 2^e's exponent field
                const float by = __uint_as_float(up << 23);
                c[t][half] = a.scale_log2 * __uint_as_float((254u - up) << 23);
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __half2 f = __floats2half2_rn(__uint_as_float(w[y][i] << 16) * by,
                                                            __uint_as_float(w[y][i] & 0xffff0000u) * by);
                        qf[t][4 * y + i / 2][half + 2 * (i & 1)] = *reinterpret_cast<const uint32_t*>(&f);
                    }
            }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
        }
    }
    // K and V of `keys` keys at ks and vs; scale: lane 4 kind + s has that of keys 16 s ..
    __device__ __forceinline__ void step(const AttnArgs& a, uint32_t ks, uint32_t vs, int keys, float scale) {
        const int lane = threadIdx.x & 31;
        const auto at = [](int key, int chunk) {
            return key * D + (D == 64 ? (chunk ^ (key >> 1 & 3)) << 4 : (chunk ^ code_turn(key)) << 4);
        };
        float s[MT][KS / 8][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < KS / 8; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
        for (int n = 0; n < KS / 8; ++n)
#pragma unroll
            for (int y = 0; y < D / 64; ++y) {
                const uint4 v = lds16(ks + at(n * 8 + (lane >> 2), 4 * y + (lane & 3)));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b0, b1;
                    Code::halves(w[i], b0, b1);
#pragma unroll
                    for (int t = 0; t < MT; ++t) mma16816_f16(s[t][n], qf[t][4 * y + i], b0, b1);
                }
            }
        uint32_t pf[MT][KS / 16][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < KS / 16; ++n) {
                const float sk = __shfl_sync(0xffffffffu, scale, n);
                const float f[2] = {sk * c[t][0], sk * c[t][1]};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float& x = s[t][2 * n + e / 4][e % 4];
                    x *= f[e % 4 >> 1];
                    if (keys < KS && n * 16 + e / 4 * 8 + 2 * (lane & 3) + (e & 1) >= keys) x = -INFINITY;
                    top[e % 4 >> 1] = fmaxf(top[e % 4 >> 1], x);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            }
            // the reference maximum moves only when a row's has grown by
            // more than 2^8 (weights below 2^8 are held as exactly)
            if (__any_sync(0xffffffffu, top[0] > m[t][0] + 8.f || top[1] > m[t][1] + 8.f)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool grow = top[r] > m[t][r];
                    const float keep = grow ? ex2(m[t][r] - top[r]) : 1.f;
                    if (grow) m[t][r] = top[r];
                    l[t][r] *= keep;
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) o[t][x][2 * r] *= keep, o[t][x][2 * r + 1] *= keep;
                }
            }
            const float ref[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
            for (int n = 0; n < KS / 16; ++n) {
                const float sv = __shfl_sync(0xffffffffu, scale, 4 + n);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float& x = s[t][2 * n + e / 4][e % 4];
                    x = ex2(x - ref[e % 4 >> 1]);
                    l[t][e % 4 >> 1] += x;
                    x *= sv;
                }
                pf[t][n][0] = bf16x2(s[t][2 * n][0], s[t][2 * n][1]);
                pf[t][n][1] = bf16x2(s[t][2 * n][2], s[t][2 * n][3]);
                pf[t][n][2] = bf16x2(s[t][2 * n + 1][0], s[t][2 * n + 1][1]);
                pf[t][n][3] = bf16x2(s[t][2 * n + 1][2], s[t][2 * n + 1][3]);
            }
        }
#pragma unroll
        for (int n = 0; n < KS / 16; ++n)
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                // keys 0 - 7 and 8 - 15 of codes 32 x .. + 15, then of the 16 after them
                uint32_t v[4];
                ldm4t(vs + at(n * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), 2 * x + (lane >> 4)), v);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t e0, e1, d0, d1;
                    Code::evens_odds(v[2 * i], e0, d0);
                    Code::evens_odds(v[2 * i + 1], e1, d1);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma16816(o[t][4 * x + 2 * i], pf[t][n], e0, e1);
                        mma16816(o[t][4 * x + 2 * i + 1], pf[t][n], d0, d1);
                    }
                }
            }
    }
    // as TensorRows::end; a lane has columns 16 x + 4 (lane % 4) .. + 3
    template <typename Put>
    __device__ __forceinline__ void end(Put put) {
        const int lane = threadIdx.x & 31, col = 4 * (lane & 3);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[t][r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                put(16 * t + 8 * r + (lane >> 2), m[t][r], sum, col == 0, [&](auto* out, float inv) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const float *e = o[t][2 * x] + 2 * r, *d = o[t][2 * x + 1] + 2 * r;
                        const float u[4] = {e[0] * inv, d[0] * inv, e[1] * inv, d[1] * inv};
                        if constexpr (sizeof(*out) == 2)
                            *reinterpret_cast<uint2*>(out + x * 16 + col) = make_uint2(bf16x2(u[0], u[1]), bf16x2(u[2], u[3]));
                        else
                            *reinterpret_cast<float4*>(out + x * 16 + col) = make_float4(u[0], u[1], u[2], u[3]);
                    }
                });
            }
    }
};

template <int D>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
    if (a.int8) return a.group <= 16 ? launch<CodeRows<I8, D, 1>>(a, s) : launch<CodeRows<I8, D, 2>>(a, s);
    return a.group <= 16 ? launch<CodeRows<E4M3, D, 1>>(a, s) : launch<CodeRows<E4M3, D, 2>>(a, s);
}

}  // namespace

cudaError_t launch_attn_decode8(int d, const AttnArgs& a, cudaStream_t s) {
    return d == 64 ? launch_rows<64>(a, s) : launch_rows<128>(a, s);
}

}  // namespace colibri
