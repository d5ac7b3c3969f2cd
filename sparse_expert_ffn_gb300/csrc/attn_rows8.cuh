// Attention of single bf16 rows, and of the few rows of a draft, over a paged cache of
// 8-bit codes with a scale for each block of tokens and key head.
//
// The frame, its equal shares and its rings are attn_decode.cu's (attn_share.cuh); a
// step of 8 KB holds twice the keys.  Bound by HBM as there: from 131072 to 262144 keys
// of 8 heads the time grows at 7.0 TB/s, above some 15 us for two launches; 64
// sequences of 100 - 8000 keys take 89 us, 5.4 TB/s.  What is added is the way from codes to operands:
//   s_j = (q . code_j) (scale_k c / 2^e)       c = scale * log2(e)
//   o   = sum_j (2^(s_j - m) scale_v) code_j,  l = sum_j 2^(s_j - m)
// so codes enter the products as they are, exact in 16 bits, and a scale costs one
// product per score and one per weight instead of one per element.
//
// The products are formed with the keys as the rows of mma.sync m16n8k16 and a group's
// query rows as its 8 columns, or two times 8: S^T = K Q^T and O^T = V^T P^T.  A group
// of 4 then fills half of an MMA instead of a quarter, O takes half the registers, and
// three CTAs fit an SM (rows of the group as the MMA's rows and values as bf16: 103
// instead of 87 us for the 64 sequences).  P^T, which lies as the first product leaves
// it, key by key, is turned by movmatrix.  More rows are further tiles, which read the
// keys again: 32 rows at once spill, and take 95 us for one sequence of 65421 keys and
// groups of 32 where two tiles of 16 take less.
//
// Codes become f16, because that takes the fewest instructions (e4m3: one conversion per
// two codes; whole numbers: 5 instructions per 4).  The query row becomes f16 with
// them: multiplied by a power of two 2^e that puts its largest element in
// [2^14, 2^15), it is exact but for elements 2^-29 below that one, whose error, 2^-39
// of it, is below that of the f32 sums.  A weight times its value scale is rounded to
// f16 once.  What is kept below f16's range is that product, not the weight: the
// reference m moves so that the largest 2^(s_j - m) scale_v of a row is between 2^6 and
// 2^15, and what is lost is a part 2^-31 of the row's largest term.
//
// Which element of a head stands at which place of the product's inner dimension is
// free as long as both operands agree: a lane takes 16 neighbouring codes of a key in
// one load and holds the same 16 elements of q.  Values come by ldmatrix.trans as
// 16-bit pairs of neighbouring codes of two keys, and the byte permutation that widens
// a pair also parts even columns from odd ones.
#pragma once

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

// An 8 x 8 matrix of 16-bit elements, one row per four lanes, turned.
__device__ __forceinline__ uint32_t turned8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

constexpr float kHigh = 15.f, kSet = 6.f;      // log2 of a row's largest weight: at most, and once set

// Up to 8 NT rows of a group, or (kTokens) of several tokens times a group.  g = lane / 4,
// c = lane % 4.
template <typename Code, int D, int NT, bool kTokens>
struct CodeRows {
    static constexpr bool kMany = kTokens;
    using T = uint8_t;
    using Out = __nv_bfloat16;
    static constexpr int kD = D, kRows = 8 * NT, KS = kStepKeys<T, D>, kScratch = 0;
    static constexpr int kCtas = share_ctas<T>(kRows), kStages = kCtas == 3 ? 2 : 3;
    uint32_t qf[NT][D / 16][2];                                    // row g
    // rows 2 c and 2 c + 1; o: columns 16 x + 2 g of both, then 16 x + 2 g + 1
    float o[NT][D / 16][4], m[NT][2], l[NT][2], f[NT][2];          // f: scale * log2(e) / 2^e
    int limit[NT][2], least;                                       // keys that the rows see, and all of them

    template <bool kEarly>
    __device__ __forceinline__ void begin(const AttnArgs& a, const AttnSeq& q_rows, int h, int r0) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            // of each 64 columns of row g the 16 from 16 c on
            const int row = r0 + 8 * t + (lane >> 2), token = kTokens ? row / a.group : 0;
            const bool there = row < q_rows.n * a.group;
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                            (int64_t)(q_rows.row0 + token) * a.q_stride +
                                                            (int64_t)(h * a.group + row - token * a.group) * D);
            if constexpr (kTokens) {
                const int sees = there ? attn_limit(a, q_rows, token) : q_rows.kv;
#pragma unroll
                for (int j = 0; j < 2; ++j) limit[t][j] = __shfl_sync(0xffffffffu, sees, 4 * (2 * (lane & 3) + j));
                least = t == 0 ? sees : min(least, sees);
                least = __reduce_min_sync(0xffffffffu, least);
            }
            uint32_t w[D / 64][8], top = 0;
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = there ? ld_early<kEarly>(q + y * 8 + (lane & 3) * 2 + i) : make_uint4(0u, 0u, 0u, 0u);
                    w[y][4 * i] = v.x, w[y][4 * i + 1] = v.y, w[y][4 * i + 2] = v.z, w[y][4 * i + 3] = v.w;
                }
            // (magnitudes as whole numbers: NaN and infinity on top)
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, max(w[y][i] & 0x7fffu, w[y][i] >> 16 & 0x7fffu));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t up = min(268u - (top >> 7), 240u);        // 2^e's exponent field
            const float by = __uint_as_float(up << 23), back = a.scale_log2 * __uint_as_float((254u - up) << 23);
#pragma unroll
            for (int j = 0; j < 2; ++j) f[t][j] = __shfl_sync(0xffffffffu, back, 4 * (2 * (lane & 3) + j));
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const __half2 v = __floats2half2_rn(__uint_as_float(w[y][i] << 16) * by,
                                                        __uint_as_float(w[y][i] & 0xffff0000u) * by);
                    qf[t][4 * y + i / 2][i & 1] = *reinterpret_cast<const uint32_t*>(&v);
                }
            m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
        }
    }
    // K and V of keys key0 .. hi - 1 (KS of them at most) at ks and vs; scale: lane
    // 4 kind + s has that of keys 16 s ..
    __device__ __forceinline__ void step(const AttnArgs& a, uint32_t ks, uint32_t vs, int hi, int key0, float scale) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        const auto at = [](int key, int chunk) {
            return key * D + (D == 64 ? (chunk ^ (key >> 1 & 3)) << 4 : (chunk ^ code_turn(key)) << 4);
        };
        float s[NT][KS / 16][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < KS / 16; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
        for (int n = 0; n < KS / 16; ++n)
#pragma unroll
            for (int y = 0; y < D / 64; ++y) {
                const uint4 u = lds16(ks + at(n * 16 + g, 4 * y + (lane & 3)));
                const uint4 w = lds16(ks + at(n * 16 + 8 + g, 4 * y + (lane & 3)));
                const uint32_t k[2][4] = {{u.x, u.y, u.z, u.w}, {w.x, w.y, w.z, w.w}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t r[4];
                    Code::halves(k[0][i], r[0], r[2]);
                    Code::halves(k[1][i], r[1], r[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816_f16(s[t][n], r, qf[t][4 * y + i][0], qf[t][4 * y + i][1]);
                }
            }
        // log2 of the value scales, so that no value scale is below 2^-64 for the reference
        const float log_scale = fmaxf(__log2f(fabsf(scale)), -64.f);
        float sk[KS / 16], sv[KS / 16], lv[KS / 16];
#pragma unroll
        for (int n = 0; n < KS / 16; ++n) {
            sk[n] = __shfl_sync(0xffffffffu, scale, n);
            sv[n] = __shfl_sync(0xffffffffu, scale, 4 + n);
            lv[n] = __shfl_sync(0xffffffffu, log_scale, 4 + n);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < KS / 16; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float by = sk[n] * f[t][j];
                    s[t][n][j] *= by, s[t][n][j + 2] *= by;
                }
        if ((kTokens ? min(hi, least) : hi) - key0 < KS) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int n = 0; n < KS / 16; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + n * 16 + (e >> 1) * 8 + g >= (kTokens ? min(hi, limit[t][e & 1]) : hi)) s[t][n][e] = -INFINITY;
        }
        uint32_t pf[NT][KS / 16][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < KS / 16; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) top[j] = fmaxf(top[j], fmaxf(s[t][n][j], s[t][n][j + 2]) + lv[n]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], off));
            if (__any_sync(0xffffffffu, top[0] > m[t][0] + kHigh || top[1] > m[t][1] + kHigh)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float to = top[j] - kSet;
                    const bool grow = to > m[t][j];
                    const float keep = grow ? ex2(m[t][j] - to) : 1.f;
                    if (grow) m[t][j] = to;
                    l[t][j] *= keep;
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) o[t][x][j] *= keep, o[t][x][j + 2] *= keep;
                }
            }
            const float ref[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
            for (int n = 0; n < KS / 16; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = ex2(s[t][n][e] - ref[e & 1]);
                    l[t][e & 1] += p;
                    s[t][n][e] = p * sv[n];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 p = __floats2half2_rn(s[t][n][2 * i], s[t][n][2 * i + 1]);
                    pf[t][n][i] = turned8x8(*reinterpret_cast<const uint32_t*>(&p));
                }
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
                    uint32_t r[4];
                    Code::evens_odds(v[2 * i], r[0], r[1]);
                    Code::evens_odds(v[2 * i + 1], r[2], r[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816_f16(o[t][2 * x + i], r, pf[t][n][0], pf[t][n][1]);
                }
            }
    }
    // as TensorRows::end
    template <typename Put>
    __device__ __forceinline__ void end(Put put) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sum = l[t][j];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                put(8 * t + 2 * (lane & 3) + j, m[t][j], sum, g == 0, [&](auto* out, float inv) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const float u = o[t][x][j] * inv, w = o[t][x][j + 2] * inv;
                        if constexpr (sizeof(*out) == 2) *reinterpret_cast<uint32_t*>(out + x * 16 + 2 * g) = bf16x2(u, w);
                        else *reinterpret_cast<float2*>(out + x * 16 + 2 * g) = make_float2(u, w);
                    }
                });
            }
    }
};

}  // namespace
}  // namespace colibri
