// Attention on CUDA cores for float32 layers, float32 arithmetic throughout.
//
// One CTA takes a tile of ROWS (row, head of the group) rows of one sequence
// and key head and walks its keys 64 at a time:
//   s = c q k^T,  m' = max(m, max s),  p = 2^(s - m'),
//   l = l 2^(m - m') + sum p,  o = o 2^(m - m') + p v
// with c = scale * log2(e), o / l at the end.  The rows of a group share every
// key and value read.  Each thread holds ROWS / 16 rows x 4 keys of s and
// ROWS / 16 rows x d / 16 columns of o; products are packed two to an
// instruction, along d in s and along the columns in o, because one product per
// instruction leaves no issue slots for the shared-memory reads; the next keys
// are copied during the products.  Prompts are bound by the f32 pipes and the
// shared-memory reads that feed them (4 x 4 products per thread, 256 threads:
// 1721 rows of 16 heads of 64 take 126 us, of 128 188 us; 8 x 4, 128 threads, 132 us at
// d 64: too few warps).
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
    float k[2][kKeys][D + 4];
    float v[2][kKeys][D];
    float p[ROWS][kKeys + 4];
    int item[3];
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// two packed pairs
__device__ __forceinline__ ulonglong2 load2x2(const float* p) { return *reinterpret_cast<const ulonglong2*>(p); }

template <int ROWS, int D>
__device__ __forceinline__ void simt_tile(const AttnArgs& a, SimtSmem<ROWS, D>& sm) {
    const int tid = threadIdx.x;
    if (tid < 32) {
        int b = 0, tile = 0;
        // (in order of length from two CTAs per SM on, like the plan of the ranges: attn_host.cu)
        const bool ok = attn_item(a, blockIdx.x / a.hkv, a.group, ROWS, gridDim.x * gridDim.y > 304, &b, &tile);
        int end = 0;
        if (ok && a.mode == kAttnPrefix)
            end = attn_limit_max(a, attn_seq(a, b), tile * ROWS / a.group,
                                 (min((tile + 1) * ROWS, a.n_seqs * a.group) - 1) / a.group + 1);
        if (tid == 0) sm.item[0] = ok ? b : -1, sm.item[1] = tile, sm.item[2] = end;
    }
    __syncthreads();
    const int b = sm.item[0];
    if (b < 0) return;
    const AttnSeq sq = attn_seq(a, b);
    const int h = blockIdx.x % a.hkv, sp = blockIdx.y;
    const int r0 = sm.item[1] * ROWS, rows = min(ROWS, sq.n * a.group - r0);
    if (rows <= 0) return;

    constexpr int kRPT = ROWS / 16;          // rows per thread
    constexpr int kCPT = D / 64;             // groups of 4 output columns per thread
    constexpr int kChunks = D / 4;           // 16-byte chunks of a row
    constexpr int kPasses = kKeys * kChunks / kThreads;
    const int ty = tid >> 4, tx = tid & 15;
    int lo, hi;
    attn_split(a, sp, kKeys, sq.kv0, a.mode == kAttnPrefix ? sm.item[2] : attn_limit(a, sq, (r0 + rows - 1) / a.group), &lo, &hi);

    // copies of a 64-key tile; the page ids of the tile after it are read ahead
    const int row_in = tid / kChunks, chunk = tid % kChunks;
    const float* kp = static_cast<const float*>(a.k) + (int64_t)h * a.head_stride + chunk * 4;
    const float* vp = static_cast<const float*>(a.v) + (int64_t)h * a.head_stride + chunk * 4;
    int page[kPasses];
    const auto look = [&](int j0) {
        if (!a.table) return;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int key = j0 + row_in + i * (kThreads / kChunks);
            page[i] = key < hi ? attn_page(a, b, key >> a.page_shift) : -1;
        }
    };
    const auto copy = [&](int j0, int buf) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = row_in + i * (kThreads / kChunks), key = j0 + r;
            const bool there = key < hi && (!a.table || page[i] >= 0);
            const int64_t at = !there    ? 0
                               : a.table ? (int64_t)page[i] * a.page_stride + (int64_t)(key & (a.page_size - 1)) * a.row_stride
                                         : (int64_t)(sq.row0 + key) * a.row_stride;
            cp16((uint32_t)__cvta_generic_to_shared(&sm.k[buf][r][chunk * 4]), kp + at, there);
            cp16((uint32_t)__cvta_generic_to_shared(&sm.v[buf][r][chunk * 4]), vp + at, there);
        }
    };
    look(lo);
    if (lo < hi) copy(lo, 0);
    cp_commit();
    look(lo + kKeys);

    const float* q = static_cast<const float*>(a.q);
    for (int e = tid; e < ROWS * kChunks; e += kThreads) {
        const int r = e / kChunks, c = (e % kChunks) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int i = (r0 + r) / a.group, g = (r0 + r) % a.group;
            v = load4(q + (int64_t)(sq.row0 + i) * a.q_stride + (int64_t)(h * a.group + g) * D + c);
        }
        *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
    }
    int lim[kRPT];
    float m[kRPT], l[kRPT];
    uint64_t o[kRPT][kCPT][2];
#pragma unroll
    for (int x = 0; x < kRPT; ++x) {
        const int r = ty * kRPT + x;
        lim[x] = min(hi, r < rows ? attn_limit(a, sq, (r0 + r) / a.group) : 0);
        m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
        for (int c = 0; c < kCPT; ++c) o[x][c][0] = o[x][c][1] = 0;
    }
    int buf = 0;
    for (int j0 = lo; j0 < hi; j0 += kKeys, buf ^= 1) {
        if (j0 + kKeys < hi) copy(j0 + kKeys, buf ^ 1);
        cp_commit();
        look(j0 + 2 * kKeys);
        cp_wait<1>();
        __syncthreads();
        uint64_t s2[kRPT][4];
#pragma unroll
        for (int x = 0; x < kRPT; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) s2[x][y] = 0;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            ulonglong2 qv[kRPT], kv[4];
#pragma unroll
            for (int x = 0; x < kRPT; ++x) qv[x] = load2x2(&sm.q[ty * kRPT + x][c]);
#pragma unroll
            for (int y = 0; y < 4; ++y) kv[y] = load2x2(&sm.k[buf][tx + 16 * y][c]);
#pragma unroll
            for (int x = 0; x < kRPT; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s2[x][y] = fma2(qv[x].x, kv[y].x, s2[x][y]);
                    s2[x][y] = fma2(qv[x].y, kv[y].y, s2[x][y]);
                }
        }
#pragma unroll
        for (int x = 0; x < kRPT; ++x) {
            // a row's 64 scores lie in 16 lanes, 4 each
            float s[4], top = -INFINITY;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float2 half = unpack2(s2[x][y]);
                s[y] = j0 + tx + 16 * y < lim[x] ? (half.x + half.y) * a.scale_log2 : -INFINITY;
                top = fmaxf(top, s[y]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float mn = fmaxf(m[x], top), ref = mn == -INFINITY ? 0.f : mn;
            const float keep = ex2(m[x] - ref);
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float p = ex2(s[y] - ref);
                sm.p[ty * kRPT + x][tx + 16 * y] = p;
                sum += p;
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[x] = l[x] * keep + sum;
            m[x] = mn;
            const uint64_t keep2 = pack2(keep, keep);
#pragma unroll
            for (int c = 0; c < kCPT; ++c) o[x][c][0] = mul2(o[x][c][0], keep2), o[x][c][1] = mul2(o[x][c][1], keep2);
        }
        __syncwarp();    // a row's weights are read by the half warp that wrote them
#pragma unroll 2
        for (int j = 0; j < kKeys; j += 4) {
            float4 p[kRPT];
#pragma unroll
            for (int x = 0; x < kRPT; ++x) p[x] = load4(&sm.p[ty * kRPT + x][j]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint64_t w2[kRPT];
#pragma unroll
                for (int x = 0; x < kRPT; ++x) {
                    const float w = y == 0 ? p[x].x : y == 1 ? p[x].y : y == 2 ? p[x].z : p[x].w;
                    w2[x] = pack2(w, w);
                }
#pragma unroll
                for (int c = 0; c < kCPT; ++c) {
                    const ulonglong2 v = load2x2(&sm.v[buf][j + y][tx * 4 + 64 * c]);
#pragma unroll
                    for (int x = 0; x < kRPT; ++x) {
                        o[x][c][0] = fma2(w2[x], v.x, o[x][c][0]);
                        o[x][c][1] = fma2(w2[x], v.y, o[x][c][1]);
                    }
                }
            }
        }
        __syncthreads();
    }
    cp_wait<0>();
#pragma unroll
    for (int x = 0; x < kRPT; ++x) {
        const int r = ty * kRPT + x;
        if (r >= rows) continue;
        const int row = sq.row0 + (r0 + r) / a.group, head = h * a.group + (r0 + r) % a.group;
        const float inv = l[x] > 0.f ? 1.f / l[x] : l[x];              // no key: 0; NaN stays
        const float lse2 = l[x] == 0.f ? -INFINITY : m[x] + log2f(l[x]);
        const int64_t flat = (int64_t)row * a.hq + head;
        const int64_t at = (int64_t)(a.part_slot + sp) * a.n_rows * a.hq + flat;
        float* out = a.part_o ? a.part_o + at * D : static_cast<float*>(a.o) + (int64_t)row * a.o_stride + (int64_t)head * D;
        if (tx == 0) {
            if (a.part_o) a.part_lse[at] = lse2;
            else if (a.lse) a.lse[flat] = lse2 * kLn2;
        }
#pragma unroll
        for (int c = 0; c < kCPT; ++c) {
            const float2 u = unpack2(o[x][c][0]), w = unpack2(o[x][c][1]);
            *reinterpret_cast<float4*>(out + tx * 4 + 64 * c) = make_float4(u.x * inv, u.y * inv, w.x * inv, w.y * inv);
        }
    }
}

template <int ROWS, int D>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    pdl_enter();
    simt_tile(a, *reinterpret_cast<SimtSmem<ROWS, D>*>(raw));
}

template <int ROWS, int D>
cudaError_t launch_simt(const AttnArgs& a, cudaStream_t s) {
    auto kern = attn_simt_kernel<ROWS, D>;
    const int bytes = (int)sizeof(SimtSmem<ROWS, D>);
    cudaError_t e = smem_attr((const void*)kern, bytes);
    if (e != cudaSuccess) return e;
    const int64_t items = attn_simt_items(a);
    if (items <= 0) return cudaSuccess;
    return launch_pdl(kern, dim3((unsigned)(items * a.hkv), a.splits), dim3(kThreads), bytes, s, a);
}

// Tiles of 64 rows, and of 16 for few rows over a prefix.  Those are latency as
// long as their CTAs are few, and 16-row tiles have a quarter of a step's products
// (512 keys of d 128 with 4 key heads: 32 rows 17 us instead of 24, 64 rows 19
// instead of 27); once they fill the GPU, 64-row tiles read less shared memory per
// product (4096 keys, 64 rows: 40 us instead of 67).
int tile_rows(const AttnArgs& a) {
    const int64_t rows = (int64_t)a.n_seqs * a.group;
    const bool few = rows <= 16 || (rows + 15) / 16 * a.hkv * (((int64_t)a.prefix_len + 127) / 128) <= 76;
    return a.mode == kAttnPrefix && few ? 16 : 64;
}

}  // namespace

int64_t attn_simt_items(const AttnArgs& a) {
    const int rows = tile_rows(a);
    // (a prompt's sequences end in a partial tile each, at most)
    if (a.mode == kAttnPrompt) return (int64_t)a.n_rows * a.group / rows + a.n_seqs;
    if (a.mode == kAttnPrefix) return ((int64_t)a.n_seqs * a.group + rows - 1) / rows;
    return (int64_t)a.n_seqs * ((a.group + rows - 1) / rows);
}

cudaError_t launch_attn_simt(int d, const AttnArgs& a, cudaStream_t s) {
    const bool few = tile_rows(a) == 16;
    if (d == 64) return few ? launch_simt<16, 64>(a, s) : launch_simt<64, 64>(a, s);
    return few ? launch_simt<16, 128>(a, s) : launch_simt<64, 128>(a, s);
}

}  // namespace colibri
