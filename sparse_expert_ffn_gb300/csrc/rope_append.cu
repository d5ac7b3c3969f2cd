// Rows of a q/k/v projection made ready for attention, in one pass: RMSNorm of
// every query and key head, rotation to the row's position, keys and values
// placed in the pages of a cache (or key rows of a tensor).
//
// Mathematics, per head x of a row at position t:
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> mscale (a cos t f_i - b sin t f_i, b cos t f_i + a sin t f_i)
// for the pairs (a, b) of y; float32, rounded once at the end.
//
// The angle: f_i / 2 pi, formed in double, as a 64-bit fraction of a turn; t times
// it, wrapped by the integer product itself, of which the top 32 bits are taken:
// off by at most 2^-32 turn and t (f_i 2^-55 + 2^-64) turns (the double product and
// its constant, and the fraction's end).  That is 2^-32 turn at positions that
// contexts have and 2^-24 at 2^31, where a float32 product would be off by 2^-24 of
// t f_i radians.  sin and cos of it are good to float32 rounding.  One set of
// angles serves every head of a row.
//
// Bound by HBM (each element is read once and written once), and close to it by
// instruction issue, so the work per element is kept small: a head is held by
// head_dim / 16 lanes, each with the first elements of eight pairs and their
// second ones, so that the rotation needs no exchange; the norm is a butterfly
// over those lanes; and a lane group takes several heads of one row, whose
// cosines and sines, times the norm weights, stay in registers.
#include <cuda_runtime.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kThreads = 256;

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

// heads of a lane group in flight (64 bytes per lane)
template <typename T> constexpr int kBatch = sizeof(T) == 2 ? 2 : 1;
// float32: the first key and value heads are loaded during the kind before them
// (1852 rows of 48 heads 17.3 -> 15.5 us).  For bf16 the registers that this takes
// cost more (15373 rows 71 -> 78 us); its heads are fetched into L2 two batches
// ahead, which takes none (71 -> 64 us; all of a row at once: 71).
template <typename T> constexpr bool kAhead = sizeof(T) == 4;
template <typename T> using Vecs = Vec8<T>[kBatch<T>][2];

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
            m[i][0] = gu * t.x, m[i][1] = gw * t.y, m[i][2] = gw * t.x, m[i][3] = gu * t.y;
        }
    }
    __device__ __forceinline__ void apply(Vec8<T> (&x)[2]) const {
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
            inv = rsqrtf(fmaf(ss, 1.f / D, eps));
        }
        float y[2][8];
        const auto products = [&](auto second) {                   // second(): with the second products
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = p[kInterleaved ? 2 * i : i] * inv, w = p[kInterleaved ? 2 * i + 1 : i + 8] * inv;
                float yu = u * m[i][0], yw = w * m[i][2];
                if (second()) yu -= w * m[i][1], yw += u * m[i][3];
                if (kInterleaved) y[i / 4][i % 4 * 2] = yu, y[i / 4][i % 4 * 2 + 1] = yw;
                else y[0][i] = yu, y[1][i] = yw;
            }
        };
        // (one branch or a select per element: bf16 15373 rows 66 or 64 us, float32
        // 1852 rows 15.7 or 16.2 us, by the registers that they take)
        if (sizeof(T) == 2) products([&] { return turns; });
        else if (turns) products([] { return true; });
        else products([] { return false; });
        x[0].set(y[0]);
        x[1].set(y[1]);
    }
};

// A CTA takes kGroups / per_row rows, `per_row` lane groups each (a power of two);
// group `sub` of a row takes heads sub, sub + step, ... of q's, of k's and of v's
// (step: per_row times the CTAs that share the row).
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ AppendArgs a, int per_row) {
    constexpr int kLanes = D / 16;                 // lanes of a head
    constexpr int kGroups = kThreads / kLanes;
    __shared__ float2 turn[2 * kThreads];          // rows x pairs: mscale * (cos, sin)
    __shared__ int place[16][2];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes;
    const int rows = kGroups / per_row, r = grp / per_row;
    const int64_t row0 = (int64_t)blockIdx.x * rows, row = row0 + r;
    const int sub = grp % per_row + per_row * blockIdx.y, step = per_row * gridDim.y;
    const int pairs = a.freq ? a.rot_dim >> 1 : 0;
    // this lane's elements.  Half layout: the first and second elements of eight
    // pairs, then the elements that are not rotated; interleaved: sixteen neighbours.
    int c0 = 16 * lane, c1 = 16 * lane + 8;
    const bool turns = 16 * lane < 2 * pairs;
    if (!kInterleaved && turns) c0 = 8 * lane, c1 = pairs + 8 * lane;

    // the first heads are loaded before the row's place and angles are known
    const T* q = static_cast<const T*>(a.q) + row * a.q_stride;
    Vecs<T> x, ahead;
    Vecs<T>& y = *(kAhead<T> ? &ahead : &x);
    const auto load = [&](Vecs<T>& x, const T* p, int h, int heads) {
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c)
            if (h + c * step < heads) {
                x[c][0].load(p + (int64_t)(h + c * step) * D + c0);
                x[c][1].load(p + (int64_t)(h + c * step) * D + c1);
            }
    };
    // a batch fetched into L2 ahead of its load
    const auto touch = [&](const T* p, int h, int heads) {
        if (kAhead<T>) return;
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c)
            if (h + c * step < heads) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (int64_t)(h + c * step) * D + c0));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (int64_t)(h + c * step) * D + c1));
            }
    };
    if (row < a.n_rows) load(x, q, sub, a.hq);
    if (row < a.n_rows) touch(q, sub + kBatch<T> * step, a.hq);
    for (int w = tid >> 5; w < rows; w += kThreads / 32) {
        int seq = -1, pos = 0;
        if (row0 + w < a.n_rows) row_place(a, (int)(row0 + w), &seq, &pos);
        if ((tid & 31) == 0) place[w][0] = seq, place[w][1] = pos;
    }
    __syncthreads();
    for (int e = tid; e < rows * pairs; e += kThreads) {
        // a frequency's fraction of a turn, 2^64 to the turn (formed in double:
        // freq / 2 pi is rounded once, at 2^-53 of itself)
        const double t = __ldg(a.freq + e % pairs) * 0.15915494309189533577;
        const uint64_t unit = __double2ull_rd((t - floor(t)) * 18446744073709551616.0);
        const int32_t top = (int32_t)((unit * (uint64_t)(int64_t)place[e / pairs][1]) >> 32);
        float sn, cs;
        sincospif((float)top * 4.656612873077392578125e-10f, &sn, &cs);   // 2^-31: half turns
        turn[e] = make_float2(cs * a.mscale, sn * a.mscale);
    }
    __syncthreads();
    const int seq = place[r][0], pos = place[r][1];
    if (seq < 0) return;

    // the row's place in the cache
    int64_t at = -1;
    if (a.v_out) {
        if (pos >= 0 && (pos >> a.page_shift) < a.table_stride) {
            const int id = __ldg(a.table + (int64_t)seq * a.table_stride + (pos >> a.page_shift));
            if ((unsigned)id < (unsigned)a.num_pages)
                at = (int64_t)id * a.page_stride + (int64_t)(pos & ((1 << a.page_shift) - 1)) * a.row_stride;
        }
    } else {
        at = row * a.row_stride;
    }
    Heads<T, D, kInterleaved> hd;
    hd.prepare(static_cast<const T*>(a.q_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
    T* q_out = static_cast<T*>(a.q_out) + row * a.q_out_stride;
    const T* k = static_cast<const T*>(a.k) + row * a.k_stride;
    if (kAhead<T> && at >= 0) load(y, k, sub, a.hkv);
    for (int h = sub; h < a.hq; h += kBatch<T> * step) {
        if (h != sub) load(x, q, h, a.hq);
        if (h + 2 * kBatch<T> * step < a.hq) touch(q, h + 2 * kBatch<T> * step, a.hq);
        else if (h + kBatch<T> * step < a.hq) touch(k, sub, a.hkv);
        else if (a.v_out) touch(static_cast<const T*>(a.v) + row * a.v_stride, sub, a.hkv);
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c) {
            if (h + c * step >= a.hq) break;
            hd.apply(x[c]);
            x[c][0].store(q_out + (int64_t)(h + c * step) * D + c0);
            x[c][1].store(q_out + (int64_t)(h + c * step) * D + c1);
        }
    }
    if (at < 0) return;
    const T* v = static_cast<const T*>(a.v) + row * a.v_stride;
    if (kAhead<T> && a.v_out) load(x, v, sub, a.hkv);
    T* k_out = static_cast<T*>(a.k_out) + at;
    if (sub < a.hkv) hd.prepare(static_cast<const T*>(a.k_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
    for (int h = sub; h < a.hkv; h += kBatch<T> * step) {
        if (!kAhead<T> || h != sub) load(y, k, h, a.hkv);
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c) {
            if (h + c * step >= a.hkv) break;
            hd.apply(y[c]);
            y[c][0].store(k_out + (int64_t)(h + c * step) * a.head_stride + c0);
            y[c][1].store(k_out + (int64_t)(h + c * step) * a.head_stride + c1);
        }
    }
    if (!a.v_out) return;
    T* v_out = static_cast<T*>(a.v_out) + at;
    for (int h = sub; h < a.hkv; h += kBatch<T> * step) {
        if (!kAhead<T> || h != sub) load(x, v, h, a.hkv);
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c) {
            if (h + c * step >= a.hkv) break;
            x[c][0].store(v_out + (int64_t)(h + c * step) * a.head_stride + c0);
            x[c][1].store(v_out + (int64_t)(h + c * step) * a.head_stride + c1);
        }
    }
}

template <typename T, int D, bool kInterleaved>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    constexpr int kGroups = kThreads / (D / 16);
    auto kern = append_kernel<T, D, kInterleaved>;
    // four groups per row while that gives three CTAs per SM; fewer rows are
    // spread over more groups, and a few over as many CTAs as give every group
    // one head (they are bound by latency)
    int per_row = 4;
    while (per_row < kGroups && (int64_t)a.n_rows * per_row < (int64_t)3 * 152 * kGroups) per_row *= 2;
    const int rows = kGroups / per_row;
    const int slices = rows == 1 && a.n_rows < 3 * 152 ? (a.hq + kGroups - 1) / kGroups : 1;
    return launch_pdl(kern, dim3((unsigned)(((int64_t)a.n_rows + rows - 1) / rows), slices), dim3(kThreads), 0, s, a,
                      per_row);
}

}  // namespace

cudaError_t launch_append(DType dt, int d, const AppendArgs& a, cudaStream_t s) {
    if (a.n_rows <= 0) return cudaSuccess;
    const bool il = a.freq && a.interleaved;
    if (dt == DType::F32)
        return d == 64 ? (il ? launch<float, 64, true>(a, s) : launch<float, 64, false>(a, s))
                       : (il ? launch<float, 128, true>(a, s) : launch<float, 128, false>(a, s));
    return d == 64 ? (il ? launch<__nv_bfloat16, 64, true>(a, s) : launch<__nv_bfloat16, 64, false>(a, s))
                   : (il ? launch<__nv_bfloat16, 128, true>(a, s) : launch<__nv_bfloat16, 128, false>(a, s));
}

}  // namespace colibri
