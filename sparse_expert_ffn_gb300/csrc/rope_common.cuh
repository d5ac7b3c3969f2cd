// What the kernels that ready projection rows for attention share: vectors of 8
// elements, a row's place, its angles, the norm and rotation of a head.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace colibri {

// 8 consecutive elements (not read through the read-only path: q_out may be q).
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a, reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <>
struct Vec8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Position and sequence of a row; called by a whole warp.  seq < 0: the row
// belongs to no sequence.
__device__ __forceinline__ void row_place(const AppendArgs& a, int row, int* seq, int* pos) {
    const int lane = threadIdx.x & 31;
    if (!a.seq_start) {
        *seq = row < a.n_seqs ? row : -1;
        *pos = *seq >= 0 && a.kv_len ? max(__ldg(a.kv_len + row), 0) - 1 : 0;
        return;
    }
    *seq = -1, *pos = 0;
    for (int base = 0; base < a.n_seqs; base += 32) {
        const int b = base + lane;
        int s0 = 0, s1 = 0;
        if (b < a.n_seqs) s0 = max(__ldg(a.seq_start + b), 0), s1 = min(__ldg(a.seq_start + b + 1), a.n_rows);
        const unsigned hit = __ballot_sync(0xffffffffu, row >= s0 && row < s1);
        if (hit) {
            const int src = __ffs(hit) - 1;
            s0 = __shfl_sync(0xffffffffu, s0, src);
            s1 = __shfl_sync(0xffffffffu, s1, src);
            *seq = base + src;
            const int total = a.kv_len ? max(__ldg(a.kv_len + *seq), 0) : s1 - s0;
            *pos = total - (s1 - row);
            return;
        }
    }
}

// Pair `pair`'s fraction of a turn per position, 2^64 to the turn (formed in double:
// freq / 2 pi is rounded once, at 2^-53 of itself).  Once per CTA: f64 is slow.
__device__ __forceinline__ uint64_t pair_unit(const AppendArgs& a, int pair) {
    const double t = __ldg(a.freq + pair) * 0.15915494309189533577;
    return __double2ull_rd((t - floor(t)) * 18446744073709551616.0);
}

// (mscale cos, mscale sin) of pair `pair`, of pair_unit `unit`, of a row at position pos.
// kFine: the float32 that the angle is rounded to is that of the distance to the nearest
// quarter turn, so that it is off by 2^-28 turn at most, instead of 2^-26.  Rounded to 8
// bits, an element that is off in the last bit of float32 may land on the other code.
template <bool kFine = false>
__device__ __forceinline__ float2 row_turn(const AppendArgs& a, int64_t row, int pos, int pair, uint64_t unit) {
    if (a.positions && row < a.n_rows) {
        const int axis = a.axis ? min((int)__ldg(a.axis + pair), a.n_axes - 1) : 0;
        pos = __ldg(a.positions + axis * a.axis_stride + row);
    }
    const int32_t top = (int32_t)((unit * (uint64_t)(int64_t)pos) >> 32);
    float sn, cs;
    if constexpr (kFine) {
        const uint32_t quarter = ((uint32_t)top + (1u << 29)) >> 30;
        sincospif((float)(int32_t)((uint32_t)top - (quarter << 30)) * 4.656612873077392578125e-10f, &sn, &cs);
        const float c = quarter & 1 ? sn : cs, s = quarter & 1 ? cs : sn;
        return make_float2((quarter == 1 || quarter == 2 ? -c : c) * a.mscale, (quarter & 2 ? -s : s) * a.mscale);
    }
    sincospif((float)top * 4.656612873077392578125e-10f, &sn, &cs);   // 2^-31: half turns
    return make_float2(cs * a.mscale, sn * a.mscale);
}

// Heads h0, h0 + step, ... of one kind (query or key) of a row: loaded, normalised,
// rotated and stored.  Element order in a lane: c0 .. c0 + 7, c1 .. c1 + 7.
template <typename T, int D, bool kInterleaved>
struct Heads {
    static constexpr int kLanes = D / 16;
    // (u, w) -> (u m[0] - w m[1], w m[2] + u m[3]): rotation and norm weights.  A lane
    // whose elements are not rotated leaves the second products out: 0 times an
    // infinite neighbour would not be 0.
    float m[8][4];
    bool norm, turns;
    float eps;

    // (kFine: norm weights u, w, cosine and sine as they are, for turned<true>)
    template <bool kFine = false>
    __device__ __forceinline__ void prepare(const T* weight, float e, const float2* turn, int lane, bool rotated, int c0,
                                            int c1) {
        norm = weight != nullptr, eps = e, turns = rotated;
        float g[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = 1.f;
        if (norm) {
            Vec8<T> v;
            float f[8];
            v.load(weight + c0);
            v.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = f[i];
            v.load(weight + c1);
            v.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[8 + i] = f[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = turns ? turn[8 * lane + i] : make_float2(1.f, 0.f);
            const float gu = g[kInterleaved ? 2 * i : i], gw = g[kInterleaved ? 2 * i + 1 : i + 8];
            if (kFine) m[i][0] = gu, m[i][1] = gw, m[i][2] = t.x, m[i][3] = t.y;
            else m[i][0] = gu * t.x, m[i][1] = gw * t.y, m[i][2] = gw * t.x, m[i][3] = gu * t.y;
        }
    }
    __device__ __forceinline__ void apply(Vec8<T> (&x)[2]) const {
        float y[2][8];
        turned(x, y);
        x[0].set(y[0]);
        x[1].set(y[1]);
    }
    // the same before it is rounded to T; kFine (after prepare<true>): with fewer roundings,
    // the products of elements and norm weights being exact where T has 8 bits, and the
    // norm's factor, rounded to nearest, multiplied to what is turned
    template <bool kFine = false>
    __device__ __forceinline__ void turned(const Vec8<T> (&x)[2], float (&y)[2][8]) const {
        float p[16];
        {
            float f[8];
            x[0].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = f[i];
            x[1].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[8 + i] = f[i];
        }
        float inv = 1.f;
        if (norm) {
            float ss = 0.f, st = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(p[i], p[i], ss), st = fmaf(p[8 + i], p[8 + i], st);
            ss += st;
            // (the lanes of the head only: other groups of the warp may have fewer heads)
            const uint32_t mine = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mine, ss, o);
            inv = kFine ? __frsqrt_rn(fmaf(ss, 1.f / D, eps)) : rsqrtf(fmaf(ss, 1.f / D, eps));
        }
        const auto products = [&](auto second) {                   // second(): with the second products
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = p[kInterleaved ? 2 * i : i] * (kFine ? m[i][0] : inv);
                const float w = p[kInterleaved ? 2 * i + 1 : i + 8] * (kFine ? m[i][1] : inv);
                float yu = u * m[i][kFine ? 2 : 0], yw = w * m[i][2];
                if (second()) yu -= w * m[i][kFine ? 3 : 1], yw += u * m[i][3];
                if (kFine) yu *= inv, yw *= inv;
                if (kInterleaved) y[i / 4][i % 4 * 2] = yu, y[i / 4][i % 4 * 2 + 1] = yw;
                else y[0][i] = yu, y[1][i] = yw;
            }
        };
        // (one branch or a select per element: bf16 15373 rows 66 or 64 us, float32
        // 1852 rows 15.7 or 16.2 us, by the registers that they take)
        if (sizeof(T) == 2) products([&] { return turns; });
        else if (turns) products([] { return true; });
        else products([] { return false; });
    }
};

}  // namespace colibri
