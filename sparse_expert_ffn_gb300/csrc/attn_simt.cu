// Attention on CUDA cores, float32 arithmetic throughout: float32 layers.
//
// One CTA takes a tile of ROWS (row, head of the group) rows of one sequence
// and key head and walks its keys 64 at a time:
//   s = scale q k^T,  m' = max(m, max s),  p = 2^(s - m'),
//   l = l 2^(m - m') + sum p,  o = o 2^(m - m') + p v
// (scores in units of log2, so that 2^x is one instruction), o / l at the end.
// The rows of a group share every key and value read.  FFMA-bound for prompts
// (64 rows: 16 FMA per shared-memory vector read), bound by shared-memory
// reads for the 16-row tiles of single tokens.
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;

template <int ROWS, int D>
struct SimtSmem {
    float q[ROWS][D];
    float k[kKeys][D + 4];
    float v[kKeys][D];
    float p[ROWS][kKeys + 4];
    int item[2];
};

// 4 consecutive elements as floats.
__device__ __forceinline__ float4 load4(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

template <typename T, int ROWS, int D>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(AttnArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    auto& sm = *reinterpret_cast<SimtSmem<ROWS, D>*>(raw);
    pdl_enter();
    const int tid = threadIdx.x;
    if (tid < 32) {
        int b = 0, tile = 0;
        const bool ok = attn_item(a, blockIdx.x, a.group, ROWS, &b, &tile);
        if (tid == 0) sm.item[0] = ok ? b : -1, sm.item[1] = tile;
    }
    __syncthreads();
    const int b = sm.item[0];
    if (b < 0) return;
    const AttnSeq sq = attn_seq(a, b);
    const int h = blockIdx.y, sp = blockIdx.z;
    const int r0 = sm.item[1] * ROWS, rows = min(ROWS, sq.n * a.group - r0);
    if (rows <= 0) return;

    constexpr int kRPT = ROWS / 16;          // rows per thread
    constexpr int kCPT = D / 64;             // float4 output columns per thread
    const int ty = tid >> 4, tx = tid & 15;
    const T* q = static_cast<const T*>(a.q);
    for (int e = tid; e < ROWS * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int i = (r0 + r) / a.group, g = (r0 + r) % a.group;
            v = load4(q + (int64_t)(sq.row0 + i) * a.q_stride + (int64_t)(h * a.group + g) * D + c);
        }
        *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
    }
    int lim[kRPT];
    float m[kRPT], l[kRPT];
    float4 o[kRPT][kCPT];
#pragma unroll
    for (int x = 0; x < kRPT; ++x) {
        const int r = ty * kRPT + x;
        lim[x] = r < rows ? attn_limit(a, sq, (r0 + r) / a.group) : 0;
        m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
        for (int c = 0; c < kCPT; ++c) o[x][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int lo, hi;
    attn_split(a, sp, kKeys, sq.kv0, attn_limit_max(a, sq, (r0 + rows - 1) / a.group + 1), &lo, &hi);

    const T* kp = static_cast<const T*>(a.k);
    const T* vp = static_cast<const T*>(a.v);
    for (int j0 = lo; j0 < hi; j0 += kKeys) {
        __syncthreads();
        for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
            const int j = e / (D / 4), c = (e % (D / 4)) * 4, key = j0 + j;
            float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
            if (key < hi) {
                int64_t at = -1;
                if (a.table) {
                    const int id = attn_page(a, b, key >> a.page_shift);
                    if (id >= 0)
                        at = (int64_t)id * a.page_stride +
                             (int64_t)(key & (a.page_size - 1)) * a.row_stride;
                } else {
                    at = (int64_t)(sq.row0 + key) * a.row_stride;
                }
                if (at >= 0) {
                    at += (int64_t)h * a.head_stride + c;
                    kv = load4(kp + at);
                    vv = load4(vp + at);
                }
            }
            *reinterpret_cast<float4*>(&sm.k[j][c]) = kv;
            *reinterpret_cast<float4*>(&sm.v[j][c]) = vv;
        }
        __syncthreads();
        float s[kRPT][4];
#pragma unroll
        for (int x = 0; x < kRPT; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 qv[kRPT], kv[4];
#pragma unroll
            for (int x = 0; x < kRPT; ++x) qv[x] = *reinterpret_cast<const float4*>(&sm.q[ty * kRPT + x][c]);
#pragma unroll
            for (int y = 0; y < 4; ++y) kv[y] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * y][c]);
#pragma unroll
            for (int x = 0; x < kRPT; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s[x][y] = fmaf(qv[x].x, kv[y].x, s[x][y]);
                    s[x][y] = fmaf(qv[x].y, kv[y].y, s[x][y]);
                    s[x][y] = fmaf(qv[x].z, kv[y].z, s[x][y]);
                    s[x][y] = fmaf(qv[x].w, kv[y].w, s[x][y]);
                }
        }
#pragma unroll
        for (int x = 0; x < kRPT; ++x) {
            // a row's 64 scores lie in 16 lanes, 4 each
            float top = -INFINITY;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int key = j0 + tx + 16 * y;
                s[x][y] = key < min(lim[x], hi) ? s[x][y] * a.scale_log2 : -INFINITY;
                top = fmaxf(top, s[x][y]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float mn = fmaxf(m[x], top), ref = mn == -INFINITY ? 0.f : mn;
            const float keep = ex2(m[x] - ref);
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float p = ex2(s[x][y] - ref);
                sm.p[ty * kRPT + x][tx + 16 * y] = p;
                sum += p;
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[x] = l[x] * keep + sum;
            m[x] = mn;
#pragma unroll
            for (int c = 0; c < kCPT; ++c)
                o[x][c].x *= keep, o[x][c].y *= keep, o[x][c].z *= keep, o[x][c].w *= keep;
        }
        __syncwarp();    // a row's weights are read by the half warp that wrote them
#pragma unroll 2
        for (int j = 0; j < kKeys; j += 4) {
            float4 p[kRPT];
#pragma unroll
            for (int x = 0; x < kRPT; ++x) p[x] = *reinterpret_cast<const float4*>(&sm.p[ty * kRPT + x][j]);
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int c = 0; c < kCPT; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(&sm.v[j + y][tx * 4 + 64 * c]);
#pragma unroll
                    for (int x = 0; x < kRPT; ++x) {
                        const float w = y == 0 ? p[x].x : y == 1 ? p[x].y : y == 2 ? p[x].z : p[x].w;
                        o[x][c].x = fmaf(w, v.x, o[x][c].x);
                        o[x][c].y = fmaf(w, v.y, o[x][c].y);
                        o[x][c].z = fmaf(w, v.z, o[x][c].z);
                        o[x][c].w = fmaf(w, v.w, o[x][c].w);
                    }
                }
        }
    }
#pragma unroll
    for (int x = 0; x < kRPT; ++x) {
        const int r = ty * kRPT + x;
        if (r >= rows) continue;
        const int row = sq.row0 + (r0 + r) / a.group, head = h * a.group + (r0 + r) % a.group;
        const float inv = l[x] > 0.f ? 1.f / l[x] : l[x] == 0.f ? 0.f : l[x];   // NaN stays NaN
        const float lse2 = l[x] == 0.f ? -INFINITY : m[x] + log2f(l[x]);
        const int64_t flat = (int64_t)row * a.hq + head;
        if (a.part_o) {
            const int64_t at = (int64_t)(a.part_slot + sp) * a.n_rows * a.hq + flat;
            if (tx == 0) a.part_lse[at] = lse2;
#pragma unroll
            for (int c = 0; c < kCPT; ++c)
                store4(a.part_o + at * D + tx * 4 + 64 * c,
                       make_float4(o[x][c].x * inv, o[x][c].y * inv, o[x][c].z * inv, o[x][c].w * inv));
        } else {
            if (tx == 0 && a.lse) a.lse[flat] = lse2 * kLn2;
            T* out = static_cast<T*>(a.o) + (int64_t)row * a.o_stride + (int64_t)head * D;
#pragma unroll
            for (int c = 0; c < kCPT; ++c)
                store4(out + tx * 4 + 64 * c,
                       make_float4(o[x][c].x * inv, o[x][c].y * inv, o[x][c].z * inv, o[x][c].w * inv));
        }
    }
}

template <typename T, int ROWS, int D>
cudaError_t launch_simt(const AttnArgs& a, cudaStream_t s) {
    auto kern = attn_simt_kernel<T, ROWS, D>;
    const int bytes = (int)sizeof(SimtSmem<ROWS, D>);
    cudaError_t e = smem_attr((const void*)kern, bytes);
    if (e != cudaSuccess) return e;
    // at most this many tiles: a sequence's last one may be partial
    int64_t items;
    if (a.mode == kAttnPrompt) items = (int64_t)a.n_rows * a.group / ROWS + a.n_seqs;
    else if (a.mode == kAttnPrefix) items = ((int64_t)a.n_seqs * a.group + ROWS - 1) / ROWS;
    else items = (int64_t)a.n_seqs * ((a.group + ROWS - 1) / ROWS);
    if (items <= 0) return cudaSuccess;
    return launch_pdl(kern, dim3((unsigned)items, a.hkv, a.splits), dim3(kThreads), bytes, s, a);
}

}  // namespace

// Tiles of 16 rows for single tokens (a group of at most 16 heads), 64 rows
// otherwise: a 64-row tile of 4 live rows spends 16 times the products.
int attn_simt_rows(const AttnArgs& a) { return a.mode == kAttnSuffix && a.group <= 16 ? 16 : 64; }

cudaError_t launch_attn_simt(DType dt, int d, const AttnArgs& a, cudaStream_t s) {
    const bool few = attn_simt_rows(a) == 16;
    if (dt == DType::F32) {
        if (d == 64) return few ? launch_simt<float, 16, 64>(a, s) : launch_simt<float, 64, 64>(a, s);
        return few ? launch_simt<float, 16, 128>(a, s) : launch_simt<float, 64, 128>(a, s);
    }
    if (d == 64)
        return few ? launch_simt<__nv_bfloat16, 16, 64>(a, s) : launch_simt<__nv_bfloat16, 64, 64>(a, s);
    return few ? launch_simt<__nv_bfloat16, 16, 128>(a, s) : launch_simt<__nv_bfloat16, 64, 128>(a, s);
}

}  // namespace colibri
