// Rows of a q/k/v projection made ready for attention, in one pass: RMSNorm of
// every query and key head, rotation to the row's position, keys and values
// placed in the pages of a cache (or key rows of a tensor).
//
// Mathematics, per head x of a row at position t:
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> mscale (a cos t f_i - b sin t f_i, b cos t f_i + a sin t f_i)
// for the pairs (a, b) of y; float32, rounded once at the end.
//
// The angle: f_i / 2 pi as a 64-bit fraction of a turn; t times it, wrapped by
// the integer product itself, is exact to 2^-33 turn at any int32 position,
// where a float32 product would be off by 2^-24 of t f_i radians.  sin and cos
// of the top 32 bits are then good to float32 rounding.  One set of angles
// serves every head of a row.
//
// Bound by HBM: each element is read once and written once.  A head is held by
// head_dim / 8 lanes, 8 consecutive elements each (one 16-byte vector of bf16,
// two of float32); its norm is a butterfly over those lanes, its rotation in
// the half layout one shuffle from the lane that holds the partner elements.
#include <cuda_runtime.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kThreads = 256;

// 8 consecutive elements of a row (not read through the read-only path: q_out
// may be q).
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <>
struct Vec8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(h[i]);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
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

// One CTA per (row, slice of the row's heads); heads are q's, then k's, then
// v's.  The loads of a lane group's heads are issued before the row's place
// and angles are known.
template <typename T, int D, int HEADS>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
    constexpr int kLanes = D / 8;                  // lanes of a head
    constexpr int kGroups = kThreads / kLanes;     // heads in flight per pass
    __shared__ float2 turn[D / 2];                 // mscale * (cos, sin)
    __shared__ int place[2];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes;
    const int row = blockIdx.x;
    const int heads = a.hq + (a.v_out ? 2 : 1) * a.hkv;
    const int h0 = (blockIdx.y * HEADS) * kGroups + grp;

    Vec8<T> x[HEADS];
#pragma unroll
    for (int c = 0; c < HEADS; ++c) {
        const int h = h0 + c * kGroups;
        if (h < a.hq)
            x[c].load(static_cast<const T*>(a.q) + row * a.q_stride + (int64_t)h * D + lane * 8);
        else if (h < a.hq + a.hkv)
            x[c].load(static_cast<const T*>(a.k) + row * a.k_stride + (int64_t)(h - a.hq) * D + lane * 8);
        else if (h < heads)
            x[c].load(static_cast<const T*>(a.v) + row * a.v_stride + (int64_t)(h - a.hq - a.hkv) * D + lane * 8);
    }
    if (tid < 32) {
        int seq, pos;
        row_place(a, row, &seq, &pos);
        if (tid == 0) place[0] = seq, place[1] = pos;
    }
    const int pairs = a.freq ? a.rot_dim >> 1 : 0;
    // a frequency's fraction of a turn, 2^64 to the turn (formed in double:
    // freq / 2 pi is rounded once, at 2^-53 of itself)
    uint64_t step = 0;
    if (tid < pairs) {
        const double t = __ldg(a.freq + tid) * 0.15915494309189533577;
        step = __double2ull_rd((t - floor(t)) * 18446744073709551616.0);
    }
    __syncthreads();
    const int seq = place[0], pos = place[1];
    if (seq < 0) return;
    if (tid < pairs) {
        const int32_t top = (int32_t)((step * (uint64_t)(int64_t)pos) >> 32);
        float sn, cs;
        sincospif((float)top * 4.656612873077392578125e-10f, &sn, &cs);   // 2^-31: half turns
        turn[tid] = make_float2(cs * a.mscale, sn * a.mscale);
    }
    __syncthreads();

    // the row's place in the cache
    int64_t at = -1;
    if (a.v_out) {
        if (pos >= 0 && (pos >> a.page_shift) < a.table_stride) {
            const int id = __ldg(a.table + (int64_t)seq * a.table_stride + (pos >> a.page_shift));
            if ((unsigned)id < (unsigned)a.num_pages)
                at = (int64_t)id * a.page_stride + (int64_t)(pos & ((1 << a.page_shift) - 1)) * a.row_stride;
        }
    } else {
        at = (int64_t)row * a.row_stride;
    }
    const int half = a.rot_dim >> 4;               // lanes of half the rotated part
#pragma unroll
    for (int c = 0; c < HEADS; ++c) {
        const int h = h0 + c * kGroups;
        // (the lane groups of a warp may hold different kinds of heads: the
        // shuffles below are over the whole warp, outside the branches)
        const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
        const void* w = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
        float y[8];
        x[c].get(y);
        if (a.q_norm || a.k_norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w) {
                const float inv = 1.0f / sqrtf(ss / (float)D + a.eps);
                Vec8<T> wv;
                float g[8];
                wv.load(static_cast<const T*>(w) + lane * 8);
                wv.get(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * g[e];
            }
        }
        if (pairs) {
            if (a.interleaved) {
                if (lane * 8 < a.rot_dim && (is_q || is_k)) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 t = turn[lane * 4 + e / 2];
                        const float p = y[e], r = y[e + 1];
                        y[e] = p * t.x - r * t.y;
                        y[e + 1] = r * t.x + p * t.y;
                    }
                }
            } else {
                const bool low = lane < half;
                const int src = (tid & 31) - lane + (low ? lane + half : lane < 2 * half ? lane - half : lane);
                float z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(0xffffffffu, y[e], src);
                if (lane < 2 * half && (is_q || is_k)) {
                    const float sign = low ? -1.f : 1.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = turn[(low ? lane : lane - half) * 8 + e];
                        y[e] = fmaf(y[e], t.x, sign * z[e] * t.y);
                    }
                }
            }
        }
        if (h >= heads) continue;
        if (is_q || is_k) x[c].set(y);            // v's bits are copied
        if (is_q)
            x[c].store(static_cast<T*>(a.q_out) + row * a.q_out_stride + (int64_t)h * D + lane * 8);
        else if (at >= 0) {
            const int hk = is_k ? h - a.hq : h - a.hq - a.hkv;
            x[c].store(static_cast<T*>(is_k ? a.k_out : a.v_out) + at + (int64_t)hk * a.head_stride + lane * 8);
        }
    }
}

template <typename T, int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    constexpr int kGroups = kThreads / (D / 8);
    const int heads = a.hq + (a.v_out ? 2 : 1) * a.hkv;
    const int passes = (heads + kGroups - 1) / kGroups;
    // a few rows are bound by latency: one pass per CTA; otherwise one CTA
    // takes up to four passes of a row, so that their loads overlap and the
    // angles are formed once
    const int per = a.n_rows < 152 ? 1 : passes < 4 ? passes : 4;
    const dim3 grid(a.n_rows, (passes + per - 1) / per), block(kThreads);
    switch (per) {
        case 1: return launch_pdl(append_kernel<T, D, 1>, grid, block, 0, s, a);
        case 2: return launch_pdl(append_kernel<T, D, 2>, grid, block, 0, s, a);
        case 3: return launch_pdl(append_kernel<T, D, 3>, grid, block, 0, s, a);
        default: return launch_pdl(append_kernel<T, D, 4>, grid, block, 0, s, a);
    }
}

}  // namespace

cudaError_t launch_append(DType dt, int d, const AppendArgs& a, cudaStream_t s) {
    if (a.n_rows <= 0) return cudaSuccess;
    if (dt == DType::F32) return d == 64 ? launch<float, 64>(a, s) : launch<float, 128>(a, s);
    return d == 64 ? launch<__nv_bfloat16, 64>(a, s) : launch<__nv_bfloat16, 128>(a, s);
}

}  // namespace colibri
